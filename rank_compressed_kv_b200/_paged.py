"""Positions and the paged cache: the shapes' classes, and the calls.

rope, paged_append and paged_decode_attn are marshalled by the native extension _call
(csrc/binding.cpp): a step of a small batch takes a few microseconds on the GPU, less than a call
over ctypes.  The extension, and torch with it, is loaded when one of the three is first asked for:
what goes over ctypes, as in _lib, needs neither.
"""
import ctypes
import math
import os
from dataclasses import dataclass

from ._lib import Dims, _L, _check, _dims_p, _i32, _nbytes, _ptr, _stream, _sz, _vp

_CALL_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_call.so")
NATIVE = ("rope", "paged_append", "paged_decode_attn")


def __getattr__(name):
    if name not in NATIVE:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    if not os.path.exists(_CALL_PATH):
        raise ImportError(f"_call.so not found at {_CALL_PATH}; build it with `python rank_compressed_kv_b200/build.py`")
    import torch  # noqa: F401  (its libraries, before the extension that needs them)

    from . import _call
    _call.structures(_CRopeSpec, _CPagedDims)
    globals().update({n: getattr(_call, n) for n in NATIVE})
    return globals()[name]


class _CRopeSpec(ctypes.Structure):
    _fields_ = [("rotary_dim", _i32), ("n_axes", _i32), ("adjacent", _i32), ("axis", ctypes.c_uint8 * 64)]


class _CPagedDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("batch", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_pages")]


_L.kvpack_paged_decode_workspace.argtypes = [_vp, _i32]
_L.kvpack_paged_decode_workspace.restype = _sz
_L.kvpack_decode_paged_workspace.argtypes = [_dims_p, _vp, _i32]
_L.kvpack_decode_paged_workspace.restype = _sz
_L.kvpack_decode_attn_paged.argtypes = [_dims_p, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_L.kvpack_decode_attn_paged.restype = ctypes.c_int


class Rope:
    """A rotation: the first rotary_dim entries of a head in pairs, each turned by one of n_axes positions.

    axis_of_pair gives the axis of each of the rotary_dim / 2 pairs; by default sections (how many
    consecutive pairs each axis has) or, without them, pair p has axis p * n_axes // (rotary_dim / 2).
    Pairs are (p, p + rotary_dim / 2), or with adjacent (2p, 2p + 1).  These stay as they are made.
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
        vars(self).update(rotary_dim=rotary_dim, n_axes=n_axes, axis_of_pair=axis_of_pair, adjacent=bool(adjacent),
                          _c=_CRopeSpec(rotary_dim, n_axes, int(bool(adjacent)), (ctypes.c_uint8 * 64)(*axis_of_pair)))

    def __setattr__(self, name, value):
        if name in ("rotary_dim", "n_axes", "axis_of_pair", "adjacent", "_c"):
            raise AttributeError(f"a Rope's {name} is not changed in place")   # the calls read _c, made in __init__
        object.__setattr__(self, name, value)

    @property
    def _at(self):
        return ctypes.addressof(self._c)              # of this object's own structure, in copies too

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
        c = _CPagedDims(self.batch, self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size, self.n_pages,
                        self.max_pages)
        object.__setattr__(self, "_c", c)

    @property
    def _at(self):
        return ctypes.addressof(self._c)              # of this object's own structure, in copies too

    def c(self) -> _CPagedDims:
        return self._c


def _dims_at(dims) -> int:
    if not isinstance(dims, PagedDims):
        raise TypeError(f"{type(dims).__name__} is not a PagedDims")
    return dims._at


def paged_decode_workspace(dims: PagedDims, n_layers: int) -> int:
    return int(_L.kvpack_paged_decode_workspace(_dims_at(dims), n_layers))


def decode_paged_workspace(dims: Dims, pdims: PagedDims, n_layers: int) -> int:
    return int(_L.kvpack_decode_paged_workspace(ctypes.byref(dims.c()), _dims_at(pdims), n_layers))


def decode_attn_paged(dims: Dims, pdims: PagedDims, n_layers: int, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, K_pages,
                      V_pages, block_table, seq_lens, mask, scale: float, out, mass, ws, stream=None):
    """decode_attn with the text tail in pages: batch row b has seq_lens[b] text tokens."""
    import torch
    at = _dims_at(pdims)
    # the checks of paged_decode_attn: pools by their number of elements, the others by shape, devices last
    pool = (n_layers, pdims.n_pages, pdims.n_kv_heads, pdims.page_size, pdims.head_dim)
    cache = ((K_pages, "K_pages", torch.bfloat16, pool), (V_pages, "V_pages", torch.bfloat16, pool),
             (block_table, "block_table", torch.int32, (pdims.batch, pdims.max_pages)),
             (seq_lens, "seq_lens", torch.int32, (pdims.batch,)))
    for t, what, dtype, shape in cache:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} is not a tensor")
        if t.dtype != dtype and not (dtype == torch.bfloat16 and t.dtype == torch.int16):
            raise ValueError(f"{what} is {t.dtype}, not {dtype}")
        if t.numel() != math.prod(shape) or (shape is not pool and tuple(t.shape) != shape):
            raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: kvpack takes contiguous tensors")
    for t, what, _, _ in cache:
        if not t.is_cuda or t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{what} is not on the current CUDA device")
    _check(_L.kvpack_decode_attn_paged(ctypes.byref(dims.c()), at, n_layers, _ptr(q), _ptr(CK_lo), _ptr(CK_hi),
                                       _ptr(BK), _ptr(CV_lo), _ptr(CV_hi), _ptr(BV), _ptr(K_pages), _ptr(V_pages),
                                       _ptr(block_table), _ptr(seq_lens), _ptr(mask), float(scale), _ptr(out),
                                       _ptr(mass), _ptr(ws), _nbytes(ws), _stream(stream)), "kvpack_decode_attn_paged")
