"""Copies and pickles of Rope and PagedDims stand for themselves, and neither is taken for the other (no GPU is needed:
tensors on the CPU are refused after everything that reads the shape objects)."""
import copy
import ctypes
import gc
import os
import pickle
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    import rank_compressed_kv_b200 as kv
    return kv


WAYS = {"deepcopy": copy.deepcopy, "copy": copy.copy, "pickle": lambda x: pickle.loads(pickle.dumps(x)),
        "pickle 2": lambda x: pickle.loads(pickle.dumps(x, 2))}


def _dims(kv, batch=3):
    return kv.PagedDims(batch=batch, n_q_heads=16, n_kv_heads=8, page_size=64, n_pages=10, max_pages=500)


def _rope_of_three_axes(kv, spec):
    """What the extension answers: it reads n_axes from the structure, then refuses the device."""
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    kv.rope(spec, torch.zeros(spec.rotary_dim // 2, dtype=torch.float64), torch.zeros(3, 3, dtype=torch.int32), x, x)


@pytest.mark.parametrize("way", WAYS)
def test_a_copy_outlives_its_original(kv, way):
    want = kv.paged_decode_workspace(_dims(kv), 2)
    assert want > 256
    dims = [WAYS[way](_dims(kv)) for _ in range(100)]
    specs = [WAYS[way](kv.Rope(96, 3, axis_of_pair=[p % 3 for p in range(48)], adjacent=True)) for _ in range(100)]
    gc.collect()
    others = [(kv.Rope(64, 1), kv.PagedDims(0, 1, 1, 1, 1, 1)) for _ in range(400)]     # what lies where the originals lay
    for d in dims:
        assert d == _dims(kv) and kv.paged_decode_workspace(d, 2) == want
        assert d._at == ctypes.addressof(d._c)
    for s in specs:
        assert (s.rotary_dim, s.n_axes, s.adjacent, s.axis_of_pair) == (96, 3, True, (0, 1, 2) * 16)
        assert s._at == ctypes.addressof(s._c)
        assert (s._c.rotary_dim, s._c.n_axes, s._c.adjacent, tuple(s._c.axis)[:48]) == (96, 3, 1, (0, 1, 2) * 16)
        with pytest.raises(ValueError, match="is not on the current CUDA device"):
            _rope_of_three_axes(kv, s)
    assert len(others) == 400


def test_another_process_takes_a_pickle(kv):
    code = ("import pickle, sys, rank_compressed_kv_b200 as kv\n"
            "d, s = pickle.load(sys.stdin.buffer)\n"
            "print(kv.paged_decode_workspace(d, 2), s._c.n_axes, s._c.rotary_dim)\n")
    got = subprocess.run([sys.executable, "-c", code], input=pickle.dumps((_dims(kv), kv.Rope(64, 2))), capture_output=True,
                         cwd=ROOT, check=True, timeout=300).stdout.split()
    assert [int(x) for x in got] == [kv.paged_decode_workspace(_dims(kv), 2), 2, 64]


def test_neither_is_taken_for_the_other(kv):
    d, s = _dims(kv), kv.Rope()

    class Other:
        _at = s._at
        _c = s._c

    class Bytes:
        _at = 0
        _c = bytes(200)

    x = torch.zeros(3, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    for bad in (d, Bytes(), 5, None, s._c):
        with pytest.raises(TypeError, match="spec is not a Rope"):
            kv.rope(bad, torch.zeros(64, dtype=torch.float64), torch.zeros(1, 3, dtype=torch.int32), x, x)
    for bad in (s, Other(), Bytes(), 5, None):
        with pytest.raises(TypeError, match="dims is not a PagedDims"):
            kv.paged_append(bad, 1, None, None, None, None, x, x, None, i, i, None, x, x)
        with pytest.raises(TypeError, match="dims is not a PagedDims"):
            kv.paged_decode_attn(bad, 1, x, x, x, i, i, 1.0, x, None, x)
        with pytest.raises(TypeError, match="not a PagedDims"):
            kv.paged_decode_workspace(bad, 1)
        with pytest.raises(TypeError, match="not a PagedDims"):
            kv.decode_paged_workspace(kv.Dims(3, 16, 8, 100, 0), bad, 1)
    pool = torch.zeros(1, 10, 8, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="spec is not a Rope"):
        kv.paged_append(_dims(kv), 1, d, torch.zeros(64, dtype=torch.float64), torch.zeros(1, 3, dtype=torch.int32), None,
                        x[:, :8], x[:, :8], None, i, torch.zeros(3, 500, dtype=torch.int32), None, pool, pool)

def test_a_rotation_is_not_changed_in_place(kv):
    s = kv.Rope()
    for name, value in (("rotary_dim", 64), ("n_axes", 2), ("adjacent", True), ("axis_of_pair", (0,) * 64)):
        with pytest.raises(AttributeError):
            setattr(s, name, value)
    assert (s.rotary_dim, s.n_axes, s.adjacent) == (128, 1, False)
    s.freq = 1                                        # other attributes are the user's own
    assert s.freq == 1
