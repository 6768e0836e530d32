"""ctypes front end of libkvpack.so: argument marshalling only."""
import ctypes
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libkvpack.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libkvpack.so not found at {_LIB_PATH}; build it with `python rank_compressed_kv_b200/build.py` "
        "(there is no CPU fallback)")

_L = ctypes.CDLL(_LIB_PATH)

STATUS_NAMES = {
    0: "KVPACK_OK", 1: "KVPACK_ERR_INVALID_ARG", 2: "KVPACK_ERR_ALIGNMENT", 3: "KVPACK_ERR_UNSUPPORTED",
    4: "KVPACK_ERR_WORKSPACE", 5: "KVPACK_ERR_CUDA", 6: "KVPACK_ERR_NOCONVERGE", 7: "KVPACK_ERR_TIMEOUT",
    8: "KVPACK_ERR_PAGE",
}


class KvpackError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class _CDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "n_q_heads", "n_kv_heads", "group", "head_dim", "T_vis", "L_text_cap", "rank", "rank_lo")]


@dataclass(frozen=True)
class Dims:
    batch: int
    n_q_heads: int
    n_kv_heads: int
    T_vis: int
    L_text_cap: int
    group: int = 4
    head_dim: int = 128
    rank: int = 64
    rank_lo: int = 16

    @property
    def groups(self) -> int:
        return self.n_kv_heads // self.group

    @property
    def Hg(self) -> int:
        return (self.n_q_heads // self.n_kv_heads) * self.group

    def units(self, n_layers: int) -> int:
        return n_layers * self.batch * self.groups

    def c(self) -> _CDims:
        return _CDims(self.batch, self.n_q_heads, self.n_kv_heads, self.group, self.head_dim, self.T_vis,
                      self.L_text_cap, self.rank, self.rank_lo)


_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t
_dims_p = ctypes.POINTER(_CDims)

_L.kvpack_version.restype = _i32
_L.kvpack_status_string.argtypes = [ctypes.c_int]
_L.kvpack_status_string.restype = ctypes.c_char_p
_L.kvpack_last_device_status.argtypes = [_vp]
_L.kvpack_last_device_status.restype = ctypes.c_int
_L.kvpack_footprint.argtypes = [_dims_p, _i32, _i32, ctypes.POINTER(ctypes.c_uint64)]
_L.kvpack_footprint.restype = ctypes.c_int
_L.kvpack_compress_workspace.argtypes = [_dims_p, _i32]
_L.kvpack_compress_workspace.restype = _sz
_L.kvpack_compress.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_compress.restype = ctypes.c_int
_L.kvpack_decode_workspace.argtypes = [_dims_p, _i32]
_L.kvpack_decode_workspace.restype = _sz
_L.kvpack_decode_attn.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                  ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_decode_attn.restype = ctypes.c_int
_L.kvpack_decode_attn_noalloc.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                          _vp, ctypes.c_float, _vp, _vp, _vp]
_L.kvpack_decode_attn_noalloc.restype = ctypes.c_int
_L.kvpack_noalloc_scratch_bytes.restype = _sz


class _CTextBasis(ctypes.Structure):
    _fields_ = [("CK_lo", _vp), ("CK_hi", _vp), ("BK", _vp), ("CV_lo", _vp), ("CV_hi", _vp), ("BV", _vp),
                ("L_c", _i32)]


_L.kvpack_quantize4.argtypes = [_dims_p, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
_L.kvpack_quantize4.restype = ctypes.c_int
_L.kvpack_decode_attn_q4.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                     ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_decode_attn_q4.restype = ctypes.c_int
_L.kvpack_decode_tb_workspace.argtypes = [_dims_p, _i32, _i32]
_L.kvpack_decode_tb_workspace.restype = _sz
_L.kvpack_decode_attn_tb.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_CTextBasis),
                                     _vp, _vp, _i32, _vp, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_decode_attn_tb.restype = ctypes.c_int
_L.kvpack_dense_decode_workspace.argtypes = [_dims_p, _i32, _i32]
_L.kvpack_dense_decode_workspace.restype = _sz
_L.kvpack_dense_decode_attn.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _i32, _i32, ctypes.c_float, _vp, _vp, _sz, _vp]
_L.kvpack_dense_decode_attn.restype = ctypes.c_int
_L.kvpack_decompress.argtypes = [_dims_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp]
_L.kvpack_decompress.restype = ctypes.c_int
_L.kvpack_selftest_bounded_wait.argtypes = [ctypes.c_int64, _vp]
_L.kvpack_selftest_bounded_wait.restype = ctypes.c_int
_L.kvpack_select.argtypes = [_dims_p, _i32, _vp, _vp, ctypes.c_float, _i32, _vp, _vp]
_L.kvpack_select.restype = ctypes.c_int


def lib():
    return _L


def library_path() -> str:
    return _LIB_PATH


def version() -> int:
    return int(_L.kvpack_version())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("kvpack takes contiguous tensors")
    return t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(status: int, what: str):
    if status != 0:
        raise KvpackError(status, what)


def footprint(dims: Dims, n_layers: int, L_text: int):
    """(dense bytes, compressed coefficients + text bytes, basis bytes) of the cache."""
    out = (ctypes.c_uint64 * 3)()
    _check(_L.kvpack_footprint(ctypes.byref(dims.c()), n_layers, L_text, out), "kvpack_footprint")
    return int(out[0]), int(out[1]), int(out[2])


def compress_workspace(dims: Dims, n_layers: int) -> int:
    return int(_L.kvpack_compress_workspace(ctypes.byref(dims.c()), n_layers))


def decode_workspace(dims: Dims, n_layers: int) -> int:
    return int(_L.kvpack_decode_workspace(ctypes.byref(dims.c()), n_layers))


def compress(dims: Dims, n_layers: int, X, C_lo, C_hi, B, sigma, ws, stream=None):
    _check(_L.kvpack_compress(ctypes.byref(dims.c()), n_layers, _ptr(X), _ptr(C_lo), _ptr(C_hi), _ptr(B),
                              _ptr(sigma), _ptr(ws), _nbytes(ws), _stream(stream)), "kvpack_compress")


def decode_attn(dims: Dims, n_layers: int, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, K_text, V_text, L_text: int,
                mask, scale: float, out, mass, ws, stream=None):
    _check(_L.kvpack_decode_attn(ctypes.byref(dims.c()), n_layers, _ptr(q), _ptr(CK_lo), _ptr(CK_hi), _ptr(BK),
                                 _ptr(CV_lo), _ptr(CV_hi), _ptr(BV), _ptr(K_text), _ptr(V_text), L_text,
                                 _ptr(mask), float(scale), _ptr(out), _ptr(mass), _ptr(ws), _nbytes(ws),
                                 _stream(stream)), "kvpack_decode_attn")


def decode_attn_noalloc(dims: Dims, n_layers: int, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, K_text, V_text,
                        L_text: int, mask, scale: float, out, mass, stream=None):
    """decode_attn with the library's built-in scratch, for callers that cannot allocate device memory."""
    _check(_L.kvpack_decode_attn_noalloc(ctypes.byref(dims.c()), n_layers, _ptr(q), _ptr(CK_lo), _ptr(CK_hi),
                                         _ptr(BK), _ptr(CV_lo), _ptr(CV_hi), _ptr(BV), _ptr(K_text), _ptr(V_text),
                                         L_text, _ptr(mask), float(scale), _ptr(out), _ptr(mass), _stream(stream)),
           "kvpack_decode_attn_noalloc")


NOALLOC_SCRATCH_BYTES = int(_L.kvpack_noalloc_scratch_bytes())


def quantize4(dims: Dims, n_layers: int, T: int, C_lo, C_hi, Q_lo, Q_hi, E, stream=None):
    """4-bit codes (uint8, two per byte) and int8 exponents of the 16-bit coefficient planes."""
    _check(_L.kvpack_quantize4(ctypes.byref(dims.c()), n_layers, int(T), _ptr(C_lo), _ptr(C_hi), _ptr(Q_lo),
                               _ptr(Q_hi), _ptr(E), _stream(stream)), "kvpack_quantize4")


def decode_attn_q4(dims: Dims, n_layers: int, q, QK_lo, QK_hi, EK, BK, QV_lo, QV_hi, EV, BV, K_text, V_text,
                   L_text: int, mask, scale: float, out, mass, ws, stream=None):
    """decode_attn over 4-bit visual coefficients, dequantized inside the decode."""
    _check(_L.kvpack_decode_attn_q4(ctypes.byref(dims.c()), n_layers, _ptr(q), _ptr(QK_lo), _ptr(QK_hi), _ptr(EK),
                                    _ptr(BK), _ptr(QV_lo), _ptr(QV_hi), _ptr(EV), _ptr(BV), _ptr(K_text),
                                    _ptr(V_text), L_text, _ptr(mask), float(scale), _ptr(out), _ptr(mass),
                                    _ptr(ws), _nbytes(ws), _stream(stream)), "kvpack_decode_attn_q4")


def decode_tb_workspace(dims: Dims, n_layers: int, L_c: int) -> int:
    return int(_L.kvpack_decode_tb_workspace(ctypes.byref(dims.c()), n_layers, int(L_c)))


def decode_attn_tb(dims: Dims, n_layers: int, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, text_basis, K_text, V_text,
                   L_text: int, mask, scale: float, out, mass, ws, stream=None):
    """decode_attn with the text tokens compressed by a basis of their own: text_basis =
    (CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, L_c) in the visual planes' layouts with L_c tokens."""
    tk_lo, tk_hi, tbk, tv_lo, tv_hi, tbv, L_c = text_basis
    tb = _CTextBasis(_ptr(tk_lo), _ptr(tk_hi), _ptr(tbk), _ptr(tv_lo), _ptr(tv_hi), _ptr(tbv), int(L_c))
    _check(_L.kvpack_decode_attn_tb(ctypes.byref(dims.c()), n_layers, _ptr(q), _ptr(CK_lo), _ptr(CK_hi), _ptr(BK),
                                    _ptr(CV_lo), _ptr(CV_hi), _ptr(BV), ctypes.byref(tb), _ptr(K_text),
                                    _ptr(V_text), L_text, _ptr(mask), float(scale), _ptr(out), _ptr(mass), _ptr(ws),
                                    _nbytes(ws), _stream(stream)), "kvpack_decode_attn_tb")


def select(dims: Dims, n_layers: int, mass, score, alpha: float, k_hi: int, mask_out, stream=None):
    _check(_L.kvpack_select(ctypes.byref(dims.c()), n_layers, _ptr(mass), _ptr(score), float(alpha), int(k_hi),
                            _ptr(mask_out), _stream(stream)), "kvpack_select")


def dense_decode_workspace(dims: Dims, n_layers: int, L_cap: int) -> int:
    return int(_L.kvpack_dense_decode_workspace(ctypes.byref(dims.c()), n_layers, L_cap))


def dense_decode_attn(dims: Dims, n_layers: int, q, K, V, L_cap: int, L: int, scale: float, out, ws, stream=None):
    """Standard attention over an uncompressed bf16 cache [units][L_cap][4][128] (the baseline)."""
    _check(_L.kvpack_dense_decode_attn(ctypes.byref(dims.c()), n_layers, _ptr(q), _ptr(K), _ptr(V), L_cap, L,
                                       float(scale), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
           "kvpack_dense_decode_attn")


def decompress(dims: Dims, n_layers: int, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, mask, K_out, V_out, L_cap: int,
               stream=None):
    """Every visual token decompressed at its rank into rows 0..T-1 of K_out, V_out [units][L_cap][4][128]."""
    _check(_L.kvpack_decompress(ctypes.byref(dims.c()), n_layers, _ptr(CK_lo), _ptr(CK_hi), _ptr(BK), _ptr(CV_lo),
                                _ptr(CV_hi), _ptr(BV), _ptr(mask), _ptr(K_out), _ptr(V_out), L_cap, _stream(stream)),
           "kvpack_decompress")


# ------------------------------------------------------------------ positions and the paged cache

class _CHeads(ctypes.Structure):
    _fields_ = [("data", _vp), ("outer_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("group_stride", ctypes.c_int64)]


class _CRopeSpec(ctypes.Structure):
    _fields_ = [("rotary_dim", _i32), ("n_axes", _i32), ("adjacent", _i32), ("axis", ctypes.c_uint8 * 64)]


class _CPagedDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("batch", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_pages")]


_heads_p = ctypes.POINTER(_CHeads)
_spec_p = ctypes.POINTER(_CRopeSpec)
_paged_p = ctypes.POINTER(_CPagedDims)
_L.kvpack_rope.argtypes = [_spec_p, _vp, _vp, _i32, _i32, _i32, _heads_p, _heads_p, _i32, _heads_p, _heads_p, _i32, _vp]
_L.kvpack_rope.restype = ctypes.c_int
_L.kvpack_paged_append.argtypes = [_paged_p, _i32, _spec_p, _vp, _vp, _i32, _heads_p, _heads_p, _heads_p, _vp, _vp, _vp,
                                   _heads_p, _vp, _vp, _vp]
_L.kvpack_paged_append.restype = ctypes.c_int
_L.kvpack_paged_decode_workspace.argtypes = [_paged_p, _i32]
_L.kvpack_paged_decode_workspace.restype = _sz
_L.kvpack_paged_decode_attn.argtypes = [_paged_p, _i32, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_paged_decode_attn.restype = ctypes.c_int
_L.kvpack_decode_paged_workspace.argtypes = [_dims_p, _paged_p, _i32]
_L.kvpack_decode_paged_workspace.restype = _sz
_L.kvpack_decode_attn_paged.argtypes = [_dims_p, _paged_p, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_decode_attn_paged.restype = ctypes.c_int


class Rope:
    """A rotation: the first rotary_dim entries of a head in pairs, each turned by one of n_axes positions.

    axis_of_pair gives the axis of each of the rotary_dim / 2 pairs; by default sections (how many
    consecutive pairs each axis has) or, without them, pair p has axis p * n_axes // (rotary_dim / 2).
    Pairs are (p, p + rotary_dim / 2), or with adjacent (2p, 2p + 1).
    """

    def __init__(self, rotary_dim: int = 128, n_axes: int = 1, sections=None, axis_of_pair=None, adjacent: bool = False):
        n = rotary_dim // 2
        if rotary_dim % 16 != 0 or not 16 <= rotary_dim <= 128:
            raise ValueError("rotary_dim is a multiple of 16 up to 128")
        if not 1 <= n_axes <= 4:
            raise ValueError("n_axes is 1 to 4")
        if sections is not None:
            if axis_of_pair is not None:
                raise ValueError("give sections or axis_of_pair, not both")
            axis_of_pair = [a for a, k in enumerate(sections) for _ in range(k)]
        elif axis_of_pair is None:
            axis_of_pair = [p * n_axes // n for p in range(n)]
        axis_of_pair = tuple(int(a) for a in axis_of_pair)
        if len(axis_of_pair) != n or any(not 0 <= a < n_axes for a in axis_of_pair):
            raise ValueError(f"{n} pairs need an axis each, below {n_axes}")
        self.rotary_dim, self.n_axes, self.axis_of_pair, self.adjacent = rotary_dim, n_axes, axis_of_pair, bool(adjacent)
        self._c = _CRopeSpec(rotary_dim, n_axes, int(self.adjacent), (ctypes.c_uint8 * 64)(*axis_of_pair))

    def frequencies(self, theta: float = 10000.0, device="cuda"):
        """theta^(-2p / rotary_dim) of each pair p: float64, the freq argument of rope and paged_append."""
        import torch
        p = torch.arange(self.rotary_dim // 2, dtype=torch.float64, device=device)
        return theta ** (-2.0 * p / self.rotary_dim)


@dataclass(frozen=True)
class PagedDims:
    batch: int
    n_q_heads: int
    n_kv_heads: int
    page_size: int
    n_pages: int
    max_pages: int
    head_dim: int = 128

    def __post_init__(self):
        object.__setattr__(self, "_c", _CPagedDims(self.batch, self.n_q_heads, self.n_kv_heads, self.head_dim,
                                                   self.page_size, self.n_pages, self.max_pages))

    def c(self) -> _CPagedDims:
        return self._c


def _device():
    import torch
    return torch.cuda.current_device()


def _want(t, dev: int, what: str, dtypes, shape=None, numel=None):
    """The address of a contiguous tensor on the current device, of one of these types (itemsizes) and this shape."""
    if t.get_device() != dev:
        raise ValueError(f"{what} is not on the current CUDA device")
    if str(t.dtype) not in dtypes:
        raise ValueError(f"{what} is {t.dtype}, not {' or '.join(dtypes)}")
    if (shape is not None and tuple(t.shape) != shape) or (numel is not None and t.numel() != numel):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape if shape is not None else (numel,)}")
    return _ptr(t)


_BF16 = ("torch.bfloat16", "torch.int16")
_I32 = ("torch.int32",)


def _heads(t, dev: int, what: str, outer: int, rows: int, heads: int):
    """kvpack_heads of a tensor [rows][heads][128], [outer][rows][heads][128] or, in the compression's
    input layout, [outer][heads / 4][rows][4][128], with any strides that the structure can hold."""
    if t.get_device() != dev:
        raise ValueError(f"{what} is not on the current CUDA device")
    if str(t.dtype) not in _BF16:
        raise ValueError(f"{what} is {t.dtype}, not bf16")
    shape, st, nd = tuple(t.shape), t.stride(), t.dim()
    if nd == 5 and shape == (outer, heads // 4, rows, 4, 128) and heads % 4 == 0:
        so, sg, sr, sh, s1 = st
    elif nd == 4 and shape == (outer, rows, heads, 128):
        (so, sr, sh, s1), sg = st, 512
    elif nd == 3 and outer == 1 and shape == (rows, heads, 128):
        (sr, sh, s1), so, sg = st, 0, 512
    else:
        raise ValueError(f"{what} has shape {shape}: {outer} x {rows} rows of {heads} heads of 128 are wanted")
    if s1 != 1 or (sh != 128 and heads > 1):
        raise ValueError(f"{what}: a head's entries and the heads of a row (of four) lie side by side")
    return _CHeads(t.data_ptr(), so, sr, sg)


def rope(spec: Rope, freq, pos, q, q_out, k=None, k_out=None, inverse: bool = False, stream=None):
    """Rotate q into q_out and k into k_out (either pair may be None; an output may be its input).

    Rows are [batch][T][heads][128], [T][heads][128], or [batch][heads / 4][T][4][128] (what compress
    takes); pos is int32 [n_axes][batch][T] ([n_axes][T] for one batch row); freq float64 [rotary_dim / 2]
    (spec.frequencies).  inverse turns back: the gradient with respect to the input is
    rope(..., grad, grad_in, inverse=True).
    """
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("an input and its output, of q, of k or of both")
    dev = _device()
    if pos.dim() not in (2, 3) or pos.shape[0] != spec.n_axes:
        raise ValueError(f"pos has shape {tuple(pos.shape)}: [{spec.n_axes}][batch][T] is wanted")
    outer, rows = (pos.shape[1] if pos.dim() == 3 else 1), pos.shape[-1]
    if outer == 0 or rows == 0:
        return
    pp = _want(pos, dev, "pos", _I32)
    fp = _want(freq, dev, "freq", ("torch.float64",), numel=spec.rotary_dim // 2)

    def n_heads(t):
        return t.shape[1] * t.shape[3] if t.dim() == 5 else t.shape[-2]

    cq = cqo = ck = cko = None
    n_q = n_k = 0
    if q is not None:
        n_q = n_heads(q)
        cq, cqo = _heads(q, dev, "q", outer, rows, n_q), _heads(q_out, dev, "q_out", outer, rows, n_q)
    if k is not None:
        n_k = n_heads(k)
        ck, cko = _heads(k, dev, "k", outer, rows, n_k), _heads(k_out, dev, "k_out", outer, rows, n_k)
    _check(_L.kvpack_rope(spec._c, fp, pp, outer, rows, n_q, cq, cqo, n_k, ck, cko, int(bool(inverse)), _stream(stream)),
           "kvpack_rope")


def _pool(dims: PagedDims, n_layers: int, K_pages, V_pages, block_table, seq_lens, dev: int):
    n = n_layers * dims.n_pages * dims.n_kv_heads * dims.page_size * dims.head_dim
    return (_want(K_pages, dev, "K_pages", _BF16, numel=n), _want(V_pages, dev, "V_pages", _BF16, numel=n),
            _want(block_table, dev, "block_table", _I32, shape=(dims.batch, dims.max_pages)),
            _want(seq_lens, dev, "seq_lens", _I32, shape=(dims.batch,)))


def paged_append(dims: PagedDims, n_layers: int, spec, freq, pos, q, k, v, row_offsets, seq_lens, block_table, q_out,
                 K_pages, V_pages, stream=None):
    """New tokens into their pages: k rotated, v as it is; q rotated into q_out (both may be None).

    q, k, v: [rows][heads][128] (n_layers 1) or [n_layers][rows][heads][128]; row_offsets int32 [batch + 1], or
    None for one row per sequence; seq_lens with the new tokens counted; spec None: no rotation.
    """
    dev = _device()
    rows = k.shape[-3]
    if row_offsets is None and rows != dims.batch:
        raise ValueError("without row_offsets there is one row per sequence")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out, or neither")
    ck, cv = _heads(k, dev, "k", n_layers, rows, dims.n_kv_heads), _heads(v, dev, "v", n_layers, rows, dims.n_kv_heads)
    cq = cqo = sc = fp = pp = None
    if q is not None:
        cq = _heads(q, dev, "q", n_layers, rows, dims.n_q_heads)
        cqo = _heads(q_out, dev, "q_out", n_layers, rows, dims.n_q_heads)
    Kp, Vp, tp, lp = _pool(dims, n_layers, K_pages, V_pages, block_table, seq_lens, dev)
    op = None if row_offsets is None else _want(row_offsets, dev, "row_offsets", _I32, shape=(dims.batch + 1,))
    if spec is not None:
        sc = spec._c
        fp = _want(freq, dev, "freq", ("torch.float64",), numel=spec.rotary_dim // 2)
        pp = _want(pos, dev, "pos", _I32, shape=(spec.n_axes, rows))
    if rows == 0:
        return
    _check(_L.kvpack_paged_append(dims.c(), n_layers, sc, fp, pp, rows, cq, ck, cv, op, lp, tp, cqo, Kp, Vp,
                                  _stream(stream)), "kvpack_paged_append")


def paged_decode_workspace(dims: PagedDims, n_layers: int) -> int:
    return int(_L.kvpack_paged_decode_workspace(dims.c(), n_layers))


def paged_decode_attn(dims: PagedDims, n_layers: int, q, K_pages, V_pages, block_table, seq_lens, scale: float, out, lse,
                      ws, stream=None):
    """One query per sequence over its pages: out [n_layers * batch][n_q][128] bf16, lse [..][n_q] fp32 or None."""
    dev = _device()
    rows = (n_layers * dims.batch, dims.n_q_heads, 128)
    Kp, Vp, tp, lp = _pool(dims, n_layers, K_pages, V_pages, block_table, seq_lens, dev)
    _check(_L.kvpack_paged_decode_attn(
        dims.c(), n_layers, _want(q, dev, "q", _BF16, shape=rows), Kp, Vp, tp, lp, scale,
        _want(out, dev, "out", _BF16, shape=rows),
        None if lse is None else _want(lse, dev, "lse", ("torch.float32",), shape=rows[:2]),
        _want(ws, dev, "ws", ("torch.uint8",)), ws.numel(), _stream(stream)), "kvpack_paged_decode_attn")


def decode_paged_workspace(dims: Dims, pdims: PagedDims, n_layers: int) -> int:
    return int(_L.kvpack_decode_paged_workspace(ctypes.byref(dims.c()), pdims.c(), n_layers))


def decode_attn_paged(dims: Dims, pdims: PagedDims, n_layers: int, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, K_pages,
                      V_pages, block_table, seq_lens, mask, scale: float, out, mass, ws, stream=None):
    """decode_attn with the text tail in pages: batch row b has seq_lens[b] text tokens."""
    dev = _device()
    Kp, Vp, tp, lp = _pool(pdims, n_layers, K_pages, V_pages, block_table, seq_lens, dev)
    _check(_L.kvpack_decode_attn_paged(ctypes.byref(dims.c()), pdims.c(), n_layers, _ptr(q), _ptr(CK_lo), _ptr(CK_hi),
                                       _ptr(BK), _ptr(CV_lo), _ptr(CV_hi), _ptr(BV), Kp, Vp, tp, lp, _ptr(mask),
                                       float(scale), _ptr(out), _ptr(mass), _ptr(ws), _nbytes(ws), _stream(stream)),
           "kvpack_decode_attn_paged")


def selftest_bounded_wait(cycles: int, stream=None):
    """Run the bounded-wait self-test (a wait that nothing completes; expect KVPACK_ERR_TIMEOUT next)."""
    _check(_L.kvpack_selftest_bounded_wait(int(cycles), _stream(stream)), "kvpack_selftest_bounded_wait")


def last_device_status(stream=None) -> int:
    return int(_L.kvpack_last_device_status(_stream(stream)))
