"""What importing the package needs: libkvpack.so.  torch, and the extension next to it, are for the calls that use them."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "rank_compressed_kv_b200"


def _python(code, cwd=ROOT):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=cwd, timeout=300)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


OTHERS = """
import rank_compressed_kv_b200 as kv
d = kv.Dims(batch=1, n_q_heads=8, n_kv_heads=8, T_vis=64, L_text_cap=16)
p = kv.PagedDims(1, 8, 8, 16, 4, 4)
assert kv.decode_workspace(d, 1) > 0 and kv.paged_decode_workspace(p, 1) > 0 and kv.decode_paged_workspace(d, p, 1) > 0
assert kv.footprint(d, 1, 16)[0] > 0 and callable(kv.decode_attn) and kv.Rope(n_axes=3).n_axes == 3
try:
    kv.decode_attn(d, 1, *[0] * 9, 0, 0, 1.0, 0, 0, None, stream=0)
except kv.KvpackError as e:
    assert e.status == 1                          # addresses as integers go to the library
"""
LOADS = """
for name in ("rope", "paged_append", "paged_decode_attn"):
    try:
        getattr(kv, name)
    except ImportError as e:
        assert %r in str(e), e
    else:
        raise AssertionError(name)
print("done")
"""


def test_without_torch():
    r = _python("import sys; sys.modules['torch'] = None\n" + OTHERS + LOADS % "torch")
    assert r.stdout.strip() == "done", r.stderr


@pytest.mark.parametrize("there,text", [(None, "build.py"), (b"\x7fELF not one", "_call.so")])
def test_without_the_extension(tmp_path, there, text):
    """None, or one that does not load."""
    shutil.copytree(os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE, ignore=shutil.ignore_patterns("_call*.so*", "csrc", "__pycache__"))
    if there is not None:
        (tmp_path / PACKAGE / "_call.so").write_bytes(there)
    r = _python(OTHERS + LOADS % text, tmp_path)
    assert r.stdout.strip() == "done", r.stderr


def test_with_both_and_what_is_loaded_when():
    r = _python("import sys\n" + OTHERS + """
assert "torch" not in sys.modules and {"rope", "paged_append", "paged_decode_attn"} <= set(dir(kv))
from rank_compressed_kv_b200 import paged_append, rope
assert rope is kv.rope and "rope" in vars(kv) and rope.__doc__.startswith("Rotate q") and kv.paged_decode_attn.__name__ == "paged_decode_attn"
try:
    kv.nothing
except AttributeError:
    print("done")
""")
    assert r.stdout.strip() == "done", r.stderr
    r = _python("from rank_compressed_kv_b200 import *\nprint(rope.__name__, decode_attn.__name__, PagedDims.__name__)")
    assert r.stdout.split() == ["rope", "decode_attn", "PagedDims"], r.stderr


def _build_module():
    import __graft_entry__
    return __graft_entry__._build_module()


def test_the_extension_is_rebuilt_for_another_torch_or_python(tmp_path, monkeypatch):
    b = _build_module()
    assert b.call_is_fresh()
    for name in ("CALL", "CALL_FOR"):
        shutil.copy(getattr(b, name), tmp_path)
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    os.utime(b.CALL)
    assert b.call_is_fresh()
    now, at = b.call_for(), b._torch()[0]
    monkeypatch.setattr(b, "_torch", lambda: (at, "9.9.9"))
    assert not b.call_is_fresh()
    monkeypatch.undo()
    for name in ("CALL", "CALL_FOR"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    with open(b.CALL_FOR, "w") as f:
        f.write(now.replace("cpython-3", "cpython-2"))
    assert not b.call_is_fresh()
    os.remove(b.CALL_FOR)                     # one of which nothing is known
    assert not b.call_is_fresh()


def test_an_extension_for_another_torch_is_not_loaded():
    r = _python("import torch\nhave = torch.__version__\ntorch.__version__ = type(have)('9.9.9')\n" + OTHERS + """
for _ in range(2):
    try:
        kv.rope
    except ImportError as e:
        assert "built for torch " + have in str(e) and "9.9.9" in str(e), e
    else:
        raise AssertionError
print("done")
""")
    assert r.stdout.strip() == "done", r.stderr
