"""The value product of the paged attention, against fp64: values that nearly cancel, and long sums."""
import math

import pytest
import torch

from gpu_util import DEV
from paged_util import D, normal, pages_for

pytestmark = pytest.mark.gpu


def _run(kv, lens, n_q, n_kv, page, q, K, V, table, scale):
    dims = kv.PagedDims(len(lens), n_q, n_kv, page, K.shape[1], table.shape[1])
    d = [t.to(DEV) for t in (q, K, V, table, torch.tensor(lens, dtype=torch.int32))]
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 5.0, dtype=torch.float32, device=DEV)
    ws = torch.full((kv.paged_decode_workspace(dims, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    kv.paged_decode_attn(dims, 1, *d, scale, out, lse, ws)
    assert kv.last_device_status() == 0
    return out.cpu(), lse.cpu()


def _two_terms(p):
    """p as the nearest bf16 and the nearest bf16 of what that leaves, and what the two leave."""
    hi = p.bfloat16().double()
    lo = (p - hi).bfloat16().double()
    return hi, lo, p - hi - lo


# batch, spare columns of the table: a cluster of blocks per unit, a warp per unit, runs over all units
FORMS = [(1, 2), (80, 0), (1, 4200)]


@pytest.mark.parametrize("batch,wide", FORMS)
def test_values_that_nearly_cancel(batch, wide):
    """Weights 1, 1 and p of values -hi, -lo and 1, where hi + lo are the 16 upper bits of p: what is left is below them.

    Tolerance: the weight p is a logit of two fp32 roundings and an exp2 (2^-22 of p in all, 2^-22 of the exp2 more); the
    sums of a few terms of at most 1 in fp32, 2^-22; one rounding of the output."""
    import rank_compressed_kv_b200 as kv
    x = -torch.arange(1, 256).double() / 256                       # all of them bf16
    p = torch.exp(x)
    rest = _two_terms(p)[2]
    order = rest.abs().argsort(descending=True)[:8]
    page, n_kv = 16, 4
    length = 64 if wide == 0 else 1500
    g = torch.Generator().manual_seed(3)
    table, n_pages = pages_for([length] * batch, page, g, wide=wide)
    K = torch.zeros(1, n_pages, n_kv, page, D, dtype=torch.bfloat16)
    V = torch.zeros_like(K)
    K[..., 0] = -200.0                                             # weight exp(-200): 0 in fp32, and V is 0
    q = torch.zeros(batch, 2 * n_kv, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    want = torch.zeros(batch, 2 * n_kv, dtype=torch.float64)
    tol = torch.zeros_like(want)
    for b in range(batch):
        for j in range(n_kv):
            i = int(order[(b + j) % 8])
            hi, lo, left = (float(t[i]) for t in _two_terms(p))
            at = torch.randperm(length, generator=g)[:3]
            where = table[b][at // page].long(), j, at % page
            K[0][where[0], where[1], where[2], 0] = torch.tensor([0.0, 0.0, float(x[i])]).bfloat16()
            V[0][where[0], where[1], where[2], 7] = torch.tensor([-hi, -lo, 1.0]).bfloat16()
            total = 2 + float(p[i])
            want[b, 2 * j:2 * j + 2] = left / total
            tol[b, 2 * j:2 * j + 2] = (float(p[i]) * 2.0 ** -21 + 2.0 ** -22) / total
            assert abs(left) / total > 3 * float(tol[b, 2 * j])    # two terms of p would be off by this
    out, _ = _run(kv, [length] * batch, 2 * n_kv, n_kv, page, q, K, V, table, 1.0)
    got = out.double()[..., 7]
    assert bool(((got - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()), float(((got - want).abs() / tol).max())
    assert bool((out[..., :7] == 0).all()) and bool((out[..., 8:] == 0).all())


def test_sums_over_many_tiles_are_rounded_and_not_cut_off():
    """Tiles that add three quarters of the running sum's last bit (256, until -256 ends it 30 tiles later).

    Tolerance: a running sum of 256 to 512 in fp32 is off by half its last bit, 2^-16, a tile; weights by 2^-22."""
    import rank_compressed_kv_b200 as kv
    page, n_kv, tiles = 256, 4, 1024
    length = 16 * tiles
    table, n_pages = pages_for([length], page, torch.Generator().manual_seed(6), wide=0)
    K = torch.zeros(1, n_pages, n_kv, page, D, dtype=torch.bfloat16)                   # all weights 1
    v = torch.full((tiles, 16), 1.5 * 2.0 ** -20)
    v[0::32], v[31::32] = 0.0, 0.0
    v[0::32, 3], v[31::32, 9] = 256.0, -256.0
    V = torch.zeros_like(K)
    t = torch.arange(length)
    V[0, table[0][t // page].long(), :, t % page, 5] = v.flatten().bfloat16()[:, None]
    q = torch.ones(1, 2 * n_kv, D, dtype=torch.bfloat16)
    out, lse = _run(kv, [length], 2 * n_kv, n_kv, page, q, K, V, table, 0.5)
    want = float(v.double().sum()) / length
    tol = (tiles * 2.0 ** -16 + 64 * 256 * 2.0 ** -22) / length
    assert tol + 2.0 ** -8 * want < want                           # what sums that lose these adds are off by
    got = out.double()[..., 5]
    assert bool(((got - want).abs() <= tol + 2.0 ** -8 * want).all()), (got, want, tol)
    assert float((lse.double() - math.log(length)).abs().max()) <= 2.0 ** -20 * math.log(length)
