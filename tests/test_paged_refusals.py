"""Refusals of the position and paged-cache entry points: bad arguments are answered before anything is
launched (no GPU is needed), by the C ABI with its statuses and by the binding with ValueError."""
import ctypes

import pytest
import torch

P = 0x10000   # never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    import rank_compressed_kv_b200 as kv
    return kv


def _pd(kv, **over):
    base = dict(batch=3, n_q_heads=16, n_kv_heads=8, page_size=64, n_pages=10, max_pages=5)
    return kv.PagedDims(**{**base, **over})


class _CHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("outer", ctypes.c_int64), ("row", ctypes.c_int64), ("group", ctypes.c_int64)]


def _heads(kv, data=P, strides=(0, 4096, 512)):
    return ctypes.pointer(_CHeads(data, *strides))


def _rope(kv, spec=None, rows=4, n_q=2, n_k=0, outer=1, freq=P, pos=P, q=None, q_out=None, raw=None):
    c = ctypes.byref((spec or kv.Rope())._c if raw is None else raw)
    q = q or _heads(kv)
    return _L(kv).kvpack_rope(c, freq, pos, outer, rows, n_q, q, q_out or _heads(kv, 2 * P), n_k, None, None, 0, None)


def test_rope_refusals(kv):
    R = kv._paged._CRopeSpec
    none = (ctypes.c_uint8 * 64)()
    assert _rope(kv, raw=R(0, 1, 0, none)) == 1
    assert _rope(kv, raw=R(128, 0, 0, none)) == 1
    assert _rope(kv, raw=R(128, 1, 2, none)) == 1
    assert _rope(kv, raw=R(24, 1, 0, none)) == 3
    assert _rope(kv, raw=R(144, 1, 0, none)) == 3
    assert _rope(kv, raw=R(128, 5, 0, none)) == 3
    assert _rope(kv, raw=R(128, 2, 0, (ctypes.c_uint8 * 64)(*([0] * 63 + [2])))) == 1
    assert _rope(kv, rows=-1) == 1
    assert _rope(kv, outer=0) == 1
    assert _rope(kv, n_q=0) == 1
    assert _rope(kv, n_k=1) == 1                                   # no k
    assert _rope(kv, n_q=1025) == 3
    assert _rope(kv, freq=None) == 1
    assert _rope(kv, pos=P + 4) == 2
    assert _rope(kv, q=_heads(kv, None)) == 1
    assert _rope(kv, q=_heads(kv, P + 2)) == 2
    assert _rope(kv, q=_heads(kv, P, (0, 4097, 512))) == 2
    assert _rope(kv, q=_heads(kv), q_out=_heads(kv, P, (0, 8192, 512))) == 1   # in place with other strides
    assert _rope(kv, q_out=_heads(kv, 2 * P, (0, 0, 512))) == 1    # rows of an output share memory
    assert _rope(kv, outer=2, q_out=_heads(kv, 2 * P, (0, 4096, 512))) == 1
    assert _rope(kv, n_q=5, q_out=_heads(kv, 2 * P, (0, 4096, 0))) == 1
    assert _rope(kv, n_q=2 ** 31 - 1, n_k=2 ** 31 - 1) == 3
    assert _rope(kv, rows=0, freq=None) == 0                       # nothing to do


def test_rope_spec_refusals(kv):
    for bad in (dict(rotary_dim=24), dict(rotary_dim=144), dict(n_axes=0), dict(n_axes=5), dict(sections=(64,), axis_of_pair=[0] * 64),
                dict(n_axes=2, sections=(10, 10)), dict(axis_of_pair=[0] * 63 + [1])):
        with pytest.raises(ValueError):
            kv.Rope(**bad)
    assert kv.Rope(n_axes=3, sections=(16, 24, 24)).axis_of_pair == (0,) * 16 + (1,) * 24 + (2,) * 24


def _L(kv):
    """The C entry points with untyped pointers."""
    L, vp, i32 = ctypes.CDLL(kv.library_path()), ctypes.c_void_p, ctypes.c_int32
    L.kvpack_rope.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, i32, vp]
    L.kvpack_paged_append.argtypes = [vp, i32, vp, vp, vp, i32, *([vp] * 10)]
    L.kvpack_paged_decode_attn.argtypes = [vp, i32, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]
    return L


def _attend(kv, d, n_layers=1, q=P, table=P, lens=P, scale=1.0, out=P, lse=P, ws=P, ws_bytes=None):
    n = kv.paged_decode_workspace(d, n_layers) if ws_bytes is None else ws_bytes
    return _L(kv).kvpack_paged_decode_attn(d._at, n_layers, q, P, P, table, lens, scale, out, lse, ws, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), 1), (dict(n_q_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(page_size=0), 1), (dict(n_pages=0), 1),
    (dict(max_pages=0), 1), (dict(head_dim=64), 3), (dict(n_q_heads=12), 3), (dict(n_q_heads=72), 3),
    (dict(batch=4097), 3), (dict(page_size=8), 3), (dict(page_size=48), 3), (dict(page_size=512), 3),
    (dict(page_size=256, max_pages=65537), 3), (dict(n_kv_heads=2048, n_q_heads=2048), 3)])
def test_paged_shape_refusals(kv, over, status):
    d = _pd(kv, **over)
    assert kv.paged_decode_workspace(d, 1) == 0
    assert _attend(kv, d, ws_bytes=1 << 40) == status
    h = _heads(kv)
    assert _L(kv).kvpack_paged_append(d._at, 1, None, None, None, d.batch, None, h, h, None, P, P, None, P, P, None) == status


def test_paged_decode_refusals(kv):
    d = _pd(kv)
    assert _attend(kv, d, n_layers=0, ws_bytes=1 << 40) == 1
    assert _attend(kv, d, q=None) == 1
    assert _attend(kv, d, out=None) == 1
    assert _attend(kv, d, table=None) == 1
    assert _attend(kv, d, lens=P + 4) == 2
    assert _attend(kv, d, lse=P + 4) == 2
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(kv, d, scale=scale) == 1
    assert _attend(kv, d, ws=None) == 4
    assert _attend(kv, d, ws_bytes=kv.paged_decode_workspace(d, 1) - 1) == 4


def test_paged_append_refusals(kv):
    d, h = _pd(kv), _heads(kv)

    def call(spec=None, freq=None, pos=None, rows=3, q=None, k=h, v=h, off=None, lens=P, table=P, q_out=None, K=P, L=1):
        return _L(kv).kvpack_paged_append(d._at, L, spec, freq, pos, rows, q, k, v, off, lens, table, q_out, K, P, None)

    assert call(L=0) == 1
    assert call(rows=4) == 1                       # one row per sequence without offsets
    assert call(rows=-1, off=P) == 1
    assert call(k=None) == 1
    assert call(v=_heads(kv, P, (0, 4, 512))) == 2
    assert call(q=h) == 1                          # q without q_out
    assert call(q=h, q_out=_heads(kv, P, (0, 8192, 512))) == 1
    assert call(spec=kv.Rope()._at, pos=P) == 1     # no frequencies
    assert call(spec=kv.Rope()._at, freq=P, pos=P + 8) == 2
    assert call(off=P + 4) == 2
    assert call(lens=None) == 1
    assert call(K=P + 8) == 2
    assert call(rows=0, off=P) == 0


def test_decode_attn_paged_refusals(kv):
    d = kv.Dims(batch=3, n_q_heads=16, n_kv_heads=8, T_vis=100, L_text_cap=0)
    pd = _pd(kv)
    n = kv.decode_paged_workspace(d, pd, 2)
    assert n > kv.decode_workspace(d, 2)

    def call(dd=d, pp=pd, table=P, ws_bytes=n, scale=1.0):
        return kv.lib().kvpack_decode_attn_paged(ctypes.byref(dd.c()), pp._at, 2, *([P] * 9), table, P, P, scale, P, P, P,
                                                 ws_bytes, None)

    assert call(pp=_pd(kv, batch=4)) == 1
    assert call(pp=_pd(kv, n_q_heads=32)) == 1
    assert call(pp=_pd(kv, page_size=8)) == 3
    assert call(table=None) == 1
    assert call(table=P + 4) == 2
    assert call(ws_bytes=n - 1) == 4
    assert call(scale=0.0) == 1
    assert kv.decode_paged_workspace(d, _pd(kv, page_size=8), 2) == 0


# The binding compares devices last: tensors on the CPU that pass every other check are refused there, so that all of
# them can be seen without a GPU.

def _ok(kv):
    """Arguments that only their device speaks against."""
    d, spec = _pd(kv), kv.Rope()
    x = torch.zeros(3, 32, 128, dtype=torch.bfloat16)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    rope = dict(spec=spec, freq=spec.frequencies(device="cpu"), pos=torch.zeros(1, 3, dtype=torch.int32), q=x[:, :16],
                q_out=z(3, 16, 128), k=x[:, 16:24], k_out=z(3, 8, 128))
    pool = dict(K_pages=z(1, 10, 8, 64, 128), V_pages=z(1, 10, 8, 64, 128), block_table=torch.zeros(3, 5, dtype=torch.int32),
                seq_lens=torch.zeros(3, dtype=torch.int32))
    append = dict(dims=d, n_layers=1, **rope, v=x[:, 24:], row_offsets=None, **pool)
    del append["k_out"]
    attend = dict(dims=d, n_layers=1, q=z(3, 16, 128), **pool, scale=1.0, out=z(3, 16, 128), lse=torch.zeros(3, 16),
                  ws=torch.zeros(100, dtype=torch.uint8))
    return {"rope": rope, "paged_append": append, "paged_decode_attn": attend}


BF = torch.bfloat16
BAD = [
    ("rope", dict(spec=3), TypeError, "Rope"),
    ("rope", dict(q=None), ValueError, "an input and its output"),
    ("rope", dict(q=None, q_out=None, k=None, k_out=None), ValueError, "an input and its output"),
    ("rope", dict(q=7), TypeError, "q is not a tensor"),
    ("rope", dict(pos=torch.zeros(1, 3)), ValueError, "pos is Float"),
    ("rope", dict(pos=torch.zeros(2, 3, dtype=torch.int32)), ValueError, "pos has shape"),
    ("rope", dict(pos=torch.zeros(3, dtype=torch.int32)), ValueError, "pos has shape"),
    ("rope", dict(pos=torch.zeros(3, 1, dtype=torch.int32).expand(3, 3)[:1, :].T.contiguous()), ValueError, "pos has shape"),
    ("rope", dict(freq=torch.zeros(64)), ValueError, "freq is Float"),
    ("rope", dict(freq=torch.zeros(32, dtype=torch.float64)), ValueError, "freq has shape"),
    ("rope", dict(q=torch.zeros(4, 16, 128, dtype=BF)), ValueError, "q has shape"),
    ("rope", dict(q_out=torch.zeros(3, 8, 128, dtype=BF)), ValueError, "q_out has shape"),
    ("rope", dict(q=torch.zeros(3, 16, 64, dtype=BF)), ValueError, "q has shape"),
    ("rope", dict(q=torch.zeros(16, 128, dtype=BF)), ValueError, "q has shape"),
    ("rope", dict(q=torch.zeros(3, 16, 128, dtype=torch.float16)), ValueError, "q is Half"),
    ("rope", dict(q=torch.zeros(3, 32, 128, dtype=BF)[:, ::2]), ValueError, "side by side"),
    ("rope", dict(k=torch.zeros(3, 8, 256, dtype=BF)[..., ::2]), ValueError, "side by side"),
    ("rope", dict(nothing=1), TypeError, "unexpected"),
    ("paged_append", dict(dims=None), TypeError, "PagedDims"),
    ("paged_append", dict(n_layers=2), ValueError, "k has shape"),
    ("paged_append", dict(n_layers=2 ** 40), ValueError, "n_layers"),
    ("paged_append", dict(k=torch.zeros(4, 8, 128, dtype=BF)), ValueError, "one row per sequence"),
    ("paged_append", dict(v=torch.zeros(3, 7, 128, dtype=BF)), ValueError, "v has shape"),
    ("paged_append", dict(q_out=None), ValueError, "q and q_out"),
    ("paged_append", dict(row_offsets=torch.zeros(3, dtype=torch.int32)), ValueError, "row_offsets has shape"),
    ("paged_append", dict(seq_lens=torch.zeros(3, dtype=torch.int64)), ValueError, "seq_lens is Long"),
    ("paged_append", dict(K_pages=torch.zeros(1, 9, 8, 64, 128, dtype=BF)), ValueError, "K_pages has shape"),
    ("paged_append", dict(pos=torch.zeros(3, 3, dtype=torch.int32)), ValueError, "pos has shape"),
    ("paged_decode_attn", dict(q=torch.zeros(3, 8, 128, dtype=BF)), ValueError, "q has shape"),
    ("paged_decode_attn", dict(q=torch.zeros(3, 32, 128, dtype=BF)[:, :16]), ValueError, "contiguous"),
    ("paged_decode_attn", dict(lse=torch.zeros(3, 16, dtype=BF)), ValueError, "lse is BFloat16"),
    ("paged_decode_attn", dict(block_table=torch.zeros(5, 3, dtype=torch.int32).T), ValueError, "contiguous"),
    ("paged_decode_attn", dict(block_table=torch.zeros(3, 6, dtype=torch.int32)), ValueError, "block_table has shape"),
    ("paged_decode_attn", dict(V_pages=torch.zeros(1, 10, 8, 64, 128)), ValueError, "V_pages is Float"),
    ("paged_decode_attn", dict(ws=torch.zeros(100)), ValueError, "ws is Float"),
    ("paged_decode_attn", dict(scale="x"), TypeError, "real number"),
]


@pytest.mark.parametrize("call", ["rope", "paged_append", "paged_decode_attn"])
def test_the_binding_refuses_tensors_that_are_not_on_the_current_device(kv, call):
    with pytest.raises(ValueError, match="is not on the current CUDA device"):
        getattr(kv, call)(**_ok(kv)[call])


@pytest.mark.parametrize("call,over,error,text", BAD)
def test_the_binding_refuses(kv, call, over, error, text):
    args = {**_ok(kv)[call], **over}
    with pytest.raises(error, match=text):
        getattr(kv, call)(**args)


def test_the_binding_takes_arguments_once(kv):
    a = _ok(kv)["rope"]
    with pytest.raises(TypeError, match="twice"):
        kv.rope(a["spec"], spec=a["spec"])
    with pytest.raises(TypeError, match="needs"):
        kv.rope(a["spec"])
    with pytest.raises(TypeError, match="at most"):
        kv.rope(*range(10))
