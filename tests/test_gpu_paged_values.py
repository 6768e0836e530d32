"""The value product of the paged attention, against fp64: values that nearly cancel, long sums, and infinite values."""
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


@pytest.mark.parametrize("batch,wide", FORMS)
def test_infinite_values_follow_the_formula(batch, wide):
    """An infinite value of a weight above 0 makes its entry infinite, infinities of both signs, a NaN value and an infinite
    one of weight 0 (a logit of -inf) make theirs NaN; all other entries are as they are without them."""
    import rank_compressed_kv_b200 as kv
    page, n_kv = 16, 4
    length = 60 if wide == 0 else 700
    g = torch.Generator().manual_seed(4)
    table, n_pages = pages_for([length] * batch, page, g, wide=wide)
    K, V = normal(g, 1, n_pages, n_kv, page, D), normal(g, 1, n_pages, n_kv, page, D)
    q = normal(g, batch, 2 * n_kv, D)
    lens = [length] * batch
    clean, clean_lse = _run(kv, lens, 2 * n_kv, n_kv, page, q, K, V, table, 0.3)
    want = clean.clone()

    def put(X, b, j, t, e, value):
        X[0, int(table[b, t // page]), j, t % page, e] = value

    for b in range(0, batch, 3):
        for t in range(length):                                    # the entries 0 and 1: every token, the last among them
            put(V, b, 0, t, 0, math.inf)
            put(V, b, 0, t, 1, -math.inf)
        want[b, :2, 0], want[b, :2, 1] = math.inf, -math.inf
        for e, t in ((2, 0), (3, length // 2), (4, length - 1), (100, 17)):
            put(V, b, 1, t, e, -math.inf)
            want[b, 2:4, e] = -math.inf
        put(V, b, 2, 5, 50, math.inf)
        put(V, b, 2, length - 2, 50, -math.inf)
        put(V, b, 2, 9, 51, math.nan)
        want[b, 4:6, 50:52] = math.nan
    out, lse = _run(kv, lens, 2 * n_kv, n_kv, page, q, K, V, table, 0.3)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[~torch.isnan(want)], want[~torch.isnan(want)])
    assert torch.equal(lse, clean_lse)
    # a weight of 0: 0 times infinity
    q[..., 0] = 1.0
    put(K, 0, 3, 20, 0, -math.inf)
    put(V, 0, 3, 20, 60, math.inf)
    out, _ = _run(kv, lens, 2 * n_kv, n_kv, page, q, K, V, table, 0.3)
    assert bool(torch.isnan(out[0, 6:8, 60]).all()) and not bool(torch.isnan(out[0, 6:8, :60]).any())


@pytest.mark.parametrize("batch,wide", FORMS)
def test_weights_of_zero_take_nothing_of_the_largest_values(batch, wide):
    """Tokens of a logit of -inf, and of one 200 below the largest (exp2 gives 0 in fp32), with values of 2e35: the largest of
    which the sum of 700, the weights of a part that holds no others being 1, stays below fp32's largest, 3.4e38."""
    import rank_compressed_kv_b200 as kv
    page, n_kv = 16, 4
    length = 60 if wide == 0 else 700
    g = torch.Generator().manual_seed(5)
    table, n_pages = pages_for([length] * batch, page, g, wide=wide)
    K = torch.zeros(1, n_pages, n_kv, page, D, dtype=torch.bfloat16)
    V = torch.full_like(K, 2e35)
    K[..., 0] = torch.tensor([-math.inf, -200.0]).repeat(page // 2)
    for b in range(batch):                                          # one token of weight 1
        at = int(torch.randint(0, length, (1,), generator=g))
        K[0, int(table[b, at // page]), :, at % page, 0] = 0
        V[0, int(table[b, at // page]), :, at % page] = 0.25
    q = torch.zeros(batch, 2 * n_kv, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out, lse = _run(kv, [length] * batch, 2 * n_kv, n_kv, page, q, K, V, table, 1.0)
    assert bool((out == 0.25).all()) and bool((lse == 0).all())


def test_infinite_text_values_in_the_decode_step():
    """The decode over a paged tail gives an infinite text value's entry what it gives over the dense tail."""
    import rank_compressed_kv_b200 as kv
    import synth
    from gpu_util import bf, u32
    from synth import cases
    n_q, n_kv, T, L = 16, 8, 200, 90
    w = synth.Workload("paged", 7, 2, 1, n_q, n_kv, T, L, 1, "lowrank32")
    c = cases.decode_case(w, n_layers=1, T=T, Lcap=L)
    g = {k: bf(c[k]) for k in ("q", "CK_lo", "CK_hi", "BK", "CV_lo", "CV_hi", "BV", "K_text", "V_text")}
    Vt = g["V_text"].view(2, n_kv // 4, L, 4, D)
    Vt[0, 0, 3, 1, 7], Vt[0, 1, 89, 2, 127], Vt[1, 1, :, 3, 64] = math.inf, -math.inf, math.inf
    page = 32
    table, n_pages = pages_for([L, L], page, torch.Generator().manual_seed(2))
    K, V = (torch.zeros(1, n_pages, n_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    t = torch.arange(L)
    for b in range(2):
        at = table[b][t // page].long(), t % page
        for X, x in ((K, g["K_text"].view(2, n_kv // 4, L, 4, D)), (V, Vt)):
            X[0, at[0].to(DEV), :, at[1].to(DEV)] = x[b].transpose(0, 1).reshape(L, n_kv, D)
    outs = []
    for paged in (True, False):
        dims = kv.Dims(batch=2, n_q_heads=n_q, n_kv_heads=n_kv, T_vis=T, L_text_cap=L)
        pd = kv.PagedDims(2, n_q, n_kv, page, n_pages, table.shape[1])
        out, mass = torch.empty(2, n_q, D, dtype=torch.bfloat16, device=DEV), torch.empty(dims.units(1), T, device=DEV)
        args = [g[k] for k in ("q", "CK_lo", "CK_hi", "BK", "CV_lo", "CV_hi", "BV")]
        if paged:
            ws = torch.empty(kv.decode_paged_workspace(dims, pd, 1), dtype=torch.uint8, device=DEV)
            kv.decode_attn_paged(dims, pd, 1, *args, K, V, table.to(DEV), torch.tensor([L, L], dtype=torch.int32, device=DEV),
                                 u32(c["mask"]), 1.0, out, mass, ws)
        else:
            ws = torch.empty(kv.decode_workspace(dims, 1), dtype=torch.uint8, device=DEV)
            kv.decode_attn(dims, 1, *args, g["K_text"], g["V_text"], L, u32(c["mask"]), 1.0, out, mass, ws)
        assert kv.last_device_status() == 0
        outs.append(out.float().cpu())
    for value in (math.inf, -math.inf):
        assert torch.equal(outs[0] == value, outs[1] == value)
    assert not bool(torch.isnan(outs[0]).any()) and int(torch.isinf(outs[0]).sum()) == 6     # three entries, two heads each
