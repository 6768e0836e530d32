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


def _heads(kv, data=P, strides=(0, 4096, 512)):
    return kv._lib._CHeads(data, *strides)


def _rope(kv, spec=None, rows=4, n_q=2, n_k=0, outer=1, freq=P, pos=P, q=None, q_out=None, raw=None):
    c = (spec or kv.Rope())._c if raw is None else raw
    q = q or _heads(kv)
    return kv.lib().kvpack_rope(c, freq, pos, outer, rows, n_q, q, q_out or _heads(kv, 2 * P), n_k, None, None, 0, None)


def test_rope_refusals(kv):
    R = kv._lib._CRopeSpec
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
    assert _rope(kv, rows=0, freq=None) == 0                       # nothing to do


def test_rope_spec_refusals(kv):
    for bad in (dict(rotary_dim=24), dict(rotary_dim=144), dict(n_axes=0), dict(n_axes=5), dict(sections=(64,), axis_of_pair=[0] * 64),
                dict(n_axes=2, sections=(10, 10)), dict(axis_of_pair=[0] * 63 + [1])):
        with pytest.raises(ValueError):
            kv.Rope(**bad)
    assert kv.Rope(n_axes=3, sections=(16, 24, 24)).axis_of_pair == (0,) * 16 + (1,) * 24 + (2,) * 24


def _attend(kv, d, n_layers=1, q=P, table=P, lens=P, scale=1.0, out=P, lse=P, ws=P, ws_bytes=None):
    n = kv.paged_decode_workspace(d, n_layers) if ws_bytes is None else ws_bytes
    return kv.lib().kvpack_paged_decode_attn(d.c(), n_layers, q, P, P, table, lens, scale, out, lse, ws, n, None)


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
    assert kv.lib().kvpack_paged_append(d.c(), 1, None, None, None, d.batch, None, h, h, None, P, P, None, P, P, None) == status


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
        return kv.lib().kvpack_paged_append(d.c(), L, spec, freq, pos, rows, q, k, v, off, lens, table, q_out, K, P, None)

    assert call(L=0) == 1
    assert call(rows=4) == 1                       # one row per sequence without offsets
    assert call(rows=-1, off=P) == 1
    assert call(k=None) == 1
    assert call(v=_heads(kv, P, (0, 4, 512))) == 2
    assert call(q=h) == 1                          # q without q_out
    assert call(q=h, q_out=_heads(kv, P, (0, 8192, 512))) == 1
    assert call(spec=kv.Rope()._c, pos=P) == 1     # no frequencies
    assert call(spec=kv.Rope()._c, freq=P, pos=P + 8) == 2
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
        return kv.lib().kvpack_decode_attn_paged(ctypes.byref(dd.c()), pp.c(), 2, *([P] * 9), table, P, P, scale, P, P, P,
                                                 ws_bytes, None)

    assert call(pp=_pd(kv, batch=4)) == 1
    assert call(pp=_pd(kv, n_q_heads=32)) == 1
    assert call(pp=_pd(kv, page_size=8)) == 3
    assert call(table=None) == 1
    assert call(table=P + 4) == 2
    assert call(ws_bytes=n - 1) == 4
    assert call(scale=0.0) == 1
    assert kv.decode_paged_workspace(d, _pd(kv, page_size=8), 2) == 0


def test_the_binding_refuses_tensors_that_are_not_on_the_current_device(kv, monkeypatch):
    monkeypatch.setattr(kv._lib, "_device", lambda: 0)
    d, spec = _pd(kv), kv.Rope()
    x = torch.zeros(3, 16, 128, dtype=torch.bfloat16)
    lens, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int32)
    pool = torch.zeros(1, 10, 8, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        kv.rope(spec, spec.frequencies(device="cpu"), torch.zeros(1, 3, dtype=torch.int32), x, x)
    with pytest.raises(ValueError, match="device"):
        kv.paged_append(d, 1, None, None, None, None, x[:, :8], x[:, 8:], None, lens, table, None, pool, pool)
    with pytest.raises(ValueError, match="device"):
        kv.paged_decode_attn(d, 1, x, pool, pool, table, lens, 1.0, x, None, pool)


class _Fake:
    """A tensor's outside, as the binding's checks see it."""

    def __init__(self, *shape, dtype="torch.bfloat16", device=0, stride=None):
        t = torch.empty(shape, device="meta")
        self.shape, self.dtype, self._d, self._s = t.shape, dtype, device, stride or t.stride()
        self._c = stride is None

    def get_device(self): return self._d
    def stride(self): return self._s
    def dim(self): return len(self.shape)
    def numel(self): return self.shape.numel()
    def is_contiguous(self): return self._c
    def data_ptr(self): return P


def test_the_binding_refuses_shapes_types_and_strides(kv):
    L = kv._lib
    with pytest.raises(ValueError, match="shape"):
        L._want(_Fake(3, 4), 0, "x", ("torch.bfloat16",), shape=(3, 5))
    with pytest.raises(ValueError, match="is torch.float32"):
        L._want(_Fake(3, 4, dtype="torch.float32"), 0, "x", ("torch.bfloat16",), shape=(3, 4))
    with pytest.raises(ValueError, match="contiguous"):
        L._want(_Fake(3, 4, stride=(8, 1)), 0, "x", ("torch.bfloat16",), shape=(3, 4))
    with pytest.raises(ValueError, match="device"):
        L._want(_Fake(3, 4, device=1), 0, "x", ("torch.bfloat16",), shape=(3, 4))
    ok = L._heads(_Fake(7, 6, 128), 0, "x", 1, 7, 6)
    assert (ok.row_stride, ok.group_stride) == (768, 512)
    ok = L._heads(_Fake(2, 3, 7, 4, 128), 0, "x", 2, 7, 12)
    assert (ok.outer_stride, ok.row_stride, ok.group_stride) == (3 * 7 * 512, 512, 7 * 512)
    for bad in (_Fake(7, 6, 64), _Fake(8, 6, 128), _Fake(2, 7, 6, 128), _Fake(7, 6, 128, stride=(768, 256, 1)),
                _Fake(7, 6, 128, stride=(1536, 128, 2)), _Fake(1, 2, 7, 3, 128)):
        with pytest.raises(ValueError):
            L._heads(bad, 0, "x", 1, 7, 6)
