"""The paged cache through the binding: append, decode attention, the decode step with its text tail in
pages, and all of them together, against plain fp64 forms (paged_util.py) and the oracle."""
import math

import numpy as np
import pytest
import torch

import synth
from gpu_util import DEV, assert_decode_close, bf, oracle_decode, u32
from paged_util import (D, attend, blank_unused, close_attend, close_turned, normal, pages_for, turned, turned_bound)
from synth import cases

pytestmark = pytest.mark.gpu


def _attend(kv, dims, layers, q, K, V, table, lens, scale, want_lse=True):
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV) if want_lse else None
    ws = torch.full((kv.paged_decode_workspace(dims, layers),), 0xFF, dtype=torch.uint8, device=DEV)
    kv.paged_decode_attn(dims, layers, q, K, V, table, lens, scale, out, lse, ws)
    return out, lse


def _case(seed, layers, lens, n_q, n_kv, page, qscale=2.0, fill=float("nan"), behind=-1, wide=2):
    import rank_compressed_kv_b200 as kv
    g = torch.Generator().manual_seed(seed)
    table, n_pages = pages_for(lens, page, g, behind=behind, wide=wide)
    K, V = normal(g, layers, n_pages, n_kv, page, D), normal(g, layers, n_pages, n_kv, page, D)
    if fill is not None:
        blank_unused(K, table, lens, page, fill)
        blank_unused(V, table, lens, page, fill)
    q = normal(g, layers * len(lens), n_q, D, scale=qscale)
    dims = kv.PagedDims(len(lens), n_q, n_kv, page, n_pages, table.shape[1])
    return kv, dims, q, K, V, table


def _dev(*ts):
    return [t.to(DEV) for t in ts]


# spare columns of the table: where it could hold long caches, the attention takes its runs over all units; else a
# cluster of blocks per unit, or (some thousand units of up to 1024 tokens) a warp per unit
WIDE = [2, 2100]


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("layers,lens,n_q,n_kv,page", [
    (1, [1], 8, 8, 16),
    (1, [16], 8, 1, 16),
    (1, [17], 16, 8, 32),
    (1, [0, 1, 15, 16, 17, 0, 31, 33], 12, 4, 16),
    (2, [5, 0, 300, 64], 28, 4, 64),
    (1, [0, 0], 4, 4, 32),
    (1, [577], 32, 32, 256),
    (3, [129, 1, 700], 5, 1, 128),
    (1, [4999], 32, 8, 64),
    (1, [40001, 3, 1025], 16, 2, 256),
    (1, [(37 * i) % 211 for i in range(130)], 24, 4, 16),
    (1, [0] * 40 + [(11 * i) % 37 for i in range(1100)] + [900, 0, 16], 4, 2, 16),
    (1, [0, 7, 20000, 0], 8, 2, 64),
    (2, [33] * 64, 8, 8, 32),
    (1, [(29 * i) % 600 for i in range(260)], 28, 4, 128),
    (4, [0, 1, 17, 300] * 10, 32, 32, 16),
    (1, [3000, 5, 0, 16390], 8, 4, 256),
])
def test_attend_matches_fp64(layers, lens, n_q, n_kv, page, wide):
    """Slots that hold no token are NaN, table entries behind the last page out of range."""
    kv, dims, q, K, V, table = _case(len(lens) * 100 + n_q, layers, lens, n_q, n_kv, page, behind=2 ** 31 - 1, wide=wide)
    scale = D ** -0.5
    ln = torch.tensor(lens, dtype=torch.int32)
    d = _dev(q, K, V, table, ln)
    out, lse = _attend(kv, dims, layers, *d, scale)
    assert kv.last_device_status() == 0
    close_attend(out.cpu(), lse.cpu(), attend(q, K, V, table, lens, page, scale))
    again, lse2 = _attend(kv, dims, layers, *d, scale)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    only, _ = _attend(kv, dims, layers, *d, scale, want_lse=False)
    assert torch.equal(out, only)


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("per", range(1, 9))
def test_every_number_of_query_heads_per_cached_head(per, wide):
    lens = [70, 2000, 19]
    kv, dims, q, K, V, table = _case(per, 1, lens, 2 * per, 2, 32, wide=wide)
    out, lse = _attend(kv, dims, 1, *_dev(q, K, V, table, torch.tensor(lens, dtype=torch.int32)), 0.1)
    close_attend(out.cpu(), lse.cpu(), attend(q, K, V, table, lens, 32, 0.1))


@pytest.mark.parametrize("what", ["one token stands out", "all logits equal", "late maximum", "large logits"])
def test_distributions(what):
    lens = [3000, 47]
    kv, dims, q, K, V, table = _case(9, 1, lens, 8, 2, 64)
    if what == "one token stands out":
        q[:] = 0
        q[:, :, 0] = 30.0
        page, at = int(table[0, 20]), 13
        K[0, :, :, :, 0] = 0
        K[0, page, :, at, 0] = 8.0
    elif what == "all logits equal":
        q[:] = 0
    elif what == "late maximum":
        q[:, :, 0] = 5.0
        t = torch.arange(3000)
        K[0, table[0][t // 64].long(), :, t % 64, 0] = (t[:, None] / 100.0).bfloat16()
    else:
        q *= 40
    d = _dev(q, K, V, table, torch.tensor(lens, dtype=torch.int32))
    out, lse = _attend(kv, dims, 1, *d, D ** -0.5)
    close_attend(out.cpu(), lse.cpu(), attend(q, K, V, table, lens, 64, D ** -0.5))


@pytest.mark.parametrize("wide", WIDE)
def test_infinite_and_nan_values_follow_the_formula(wide):
    """Logits of -inf weigh nothing (all of a row: NaN, as 0 / 0); a NaN or +inf logit makes its heads NaN."""
    lens = [100, 100, 100, 100]
    kv, dims, q, K, V, table = _case(4, 1, lens, 4, 4, 16, fill=None, wide=wide)
    q[:, :, 0] = 1.0
    t = torch.arange(100)

    def put(b, head, ts, value):
        K[0, table[b][ts // 16].long(), head, ts % 16, 0] = value

    put(0, 0, t[:40], float("-inf"))          # the first tiles hold nothing else
    put(1, 1, t, float("-inf"))
    put(2, 2, t[50:51], float("nan"))
    put(3, 3, t[99:], float("inf"))
    out, lse = _attend(kv, dims, 1, *_dev(q, K, V, table, torch.tensor(lens, dtype=torch.int32)), 1.0)
    o, l = out.cpu(), lse.cpu()
    ref = attend(q, K, V, table, lens, 16, 1.0)
    bad = torch.zeros(4, 4, dtype=torch.bool)
    bad[1, 1] = bad[2, 2] = bad[3, 3] = True
    assert bool(torch.isnan(o[bad]).all()) and not bool(torch.isnan(o[~bad]).any())
    assert l[1, 1] == -math.inf and math.isnan(l[2, 2]) and not bool(torch.isnan(l[~bad]).any())
    good = ~bad
    good[0, 0] = False                        # its bound is infinite; by hand below
    clean = [r[good] for r in ref]
    close_attend(o[good], l[good], clean)
    x = (q[0, 0].double() @ K[0, table[0][t // 16].long(), 0, t % 16].double().T)
    p = torch.softmax(x, -1)
    want = p @ V[0, table[0][t // 16].long(), 0, t % 16].double()
    assert float((o[0, 0].double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 1e-3


def test_pools_beyond_32_bits():
    """Element offsets past 2^32: a pool of 4.4 G elements of which a few pages are written."""
    import rank_compressed_kv_b200 as kv
    n_kv, page, n_pages = 8, 256, 17000
    lens = [600, 0, 1030]
    K = torch.empty(1, n_pages, n_kv, page, D, dtype=torch.bfloat16, device=DEV)
    V = torch.empty_like(K)
    assert K.numel() > 2 ** 32
    used = [16999, 3, 16998, 9000, 12345, 16500, 16384, 8191]
    g = torch.Generator().manual_seed(8)
    table = torch.full((3, 6), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor(used[:3])
    table[2, :5] = torch.tensor(used[3:])
    small = torch.full((3, 6), -1, dtype=torch.int32)
    small[0, :3], small[2, :5] = torch.arange(3), torch.arange(3, 8)
    Ks, Vs = normal(g, 1, 8, n_kv, page, D), normal(g, 1, 8, n_kv, page, D)
    for i, u in enumerate(used):
        K[0, u], V[0, u] = Ks[0, i].to(DEV), Vs[0, i].to(DEV)
    q = normal(g, 3, 16, D, scale=2.0)
    dims = kv.PagedDims(3, 16, n_kv, page, n_pages, 6)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = _attend(kv, dims, 1, q.to(DEV), K, V, table.to(DEV), ln, 0.09)
    close_attend(out.cpu(), lse.cpu(), attend(q, Ks, Vs, small, lens, page, 0.09))
    # and the append reaches the same slots
    k, v = normal(g, 3, n_kv, D), normal(g, 3, n_kv, D)
    kv.paged_append(dims, 1, None, None, None, None, k.to(DEV), v.to(DEV), None, ln, table.to(DEV), None, K, V)
    assert torch.equal(K[0, used[2], :, 599 - 512].cpu(), k[0]) and torch.equal(V[0, used[7], :, 1029 - 1024].cpu(), v[2])
    assert kv.last_device_status() == 0


@pytest.mark.parametrize("wide", WIDE)
def test_a_replayed_graph_follows_the_lengths_and_two_graphs_have_workspaces_of_their_own(wide):
    lens = [900, 20, 333]
    kv, dims, q, K, V, table = _case(21, 1, lens, 16, 4, 32, fill=None, wide=wide)
    qd, Kd, Vd, td, ln = _dev(q, K, V, table, torch.tensor(lens, dtype=torch.int32))
    sides = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for s in sides:
        o, l = torch.zeros_like(qd), torch.zeros(3, 16, device=DEV)
        ws = torch.empty(kv.paged_decode_workspace(dims, 1), dtype=torch.uint8, device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            kv.paged_decode_attn(dims, 1, qd, Kd, Vd, td, ln, 0.1, o, l, ws)
        graphs.append(gr)
        outs.append((o, l, ws))
    for now in ([900, 20, 333], [1, 0, 300], [17, 20, 0]):
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        torch.cuda.synchronize()
        for s, gr in zip(sides, graphs):
            with torch.cuda.stream(s):
                for _ in range(3):
                    gr.replay()
        torch.cuda.synchronize()
        ref = attend(q, K, V, table, now, 32, 0.1)
        for o, l, _ in outs:
            close_attend(o.cpu(), l.cpu(), ref)


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("what", ["length", "negative length", "page", "negative page"])
def test_lengths_and_pages_out_of_range_are_reported(what, wide):
    lens = [200, 40]
    kv, dims, q, K, V, table = _case(2, 1, lens, 8, 4, 16, fill=None, wide=wide)
    ln = torch.tensor(lens, dtype=torch.int32)
    if what == "length":
        table[1] = 0
        ln[1] = dims.max_pages * 16 + 1
    elif what == "negative length":
        ln[1] = -5
    else:
        table[1, 1] = dims.n_pages if what == "page" else -7
    assert kv.last_device_status() == 0
    d = _dev(q, K, V, table, ln)
    out, lse = _attend(kv, dims, 1, *d, 0.1)
    assert kv.last_device_status() == 8
    ref = attend(q, K, V, table, [200, 0], 16, 0.1)          # the other sequence is as it should be
    close_attend(out[:1].cpu(), lse[:1].cpu(), [r[:1] for r in ref])
    # the append leaves the pools as they are for such a row
    Kb, Vb = d[1].clone(), d[2].clone()
    k = torch.ones(2, 4, D, dtype=torch.bfloat16, device=DEV)
    if "page" in what:
        d[4][1] = 17                                          # its token falls into the bad page
    kv.paged_append(dims, 1, None, None, None, None, k, k, None, d[4], d[3], None, d[1], d[2])
    assert kv.last_device_status() == 8
    page, at = int(table[0, 199 // 16]), 199 % 16
    Kb[0, page, :, at] = 1
    Vb[0, page, :, at] = 1
    assert torch.equal(Kb, d[1]) and torch.equal(Vb, d[2])


# ------------------------------------------------------------------------------------------- append


def _append_case(kv, seed, layers, had, new, pad, n_q, n_kv, page, rotary=128, axes=3, adjacent=False):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(had, new)]
    table, n_pages = pages_for(lens, page, g)
    rows = sum(new) + pad
    K, V = normal(g, layers, n_pages, n_kv, page, D), normal(g, layers, n_pages, n_kv, page, D)
    qkv = normal(g, layers, rows, n_q + 2 * n_kv, D)
    pos = torch.randint(0, 30000, (axes, rows), generator=g, dtype=torch.int32)
    spec = kv.Rope(rotary, axes, axis_of_pair=[p % axes for p in range(rotary // 2)], adjacent=adjacent)
    dims = kv.PagedDims(len(had), n_q, n_kv, page, n_pages, table.shape[1])
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return dims, lens, table, K, V, qkv, pos, spec, off


def _place(X, x, table, lens, new, page):
    """Where the rows x [L][rows][n_kv][128] belong in the pools X (fp64)."""
    row = 0
    for b, n in enumerate(new):
        at = torch.arange(lens[b] - n, lens[b])
        X[:, table[b][at // page].long(), :, at % page] = x[:, row:row + n].transpose(0, 1)
        row += n


@pytest.mark.parametrize("layers,had,new,pad,n_q,n_kv,page,rotary,axes,adjacent", [
    (1, [0], [1], 0, 8, 8, 16, 128, 1, False),
    (1, [0, 15, 16, 250], [577, 0, 1, 40], 5, 28, 4, 16, 128, 3, False),
    (2, [3, 100], [64, 33], 0, 16, 8, 64, 64, 2, True),
    (1, [0] * 70, [(5 * i) % 7 for i in range(70)], 11, 5, 5, 32, 128, 3, False),
    (3, [9], [2000], 2, 6, 2, 256, 96, 4, True),
])
def test_append_of_prompts(layers, had, new, pad, n_q, n_kv, page, rotary, axes, adjacent):
    import rank_compressed_kv_b200 as kv
    dims, lens, table, K, V, qkv, pos, spec, off = _append_case(kv, n_q + page, layers, had, new, pad, n_q, n_kv, page,
                                                                 rotary, axes, adjacent)
    freq = spec.frequencies(1e6, "cpu")
    d = qkv.to(DEV)
    q, k, v = d[:, :, :n_q], d[:, :, n_q:n_q + n_kv], d[:, :, n_q + n_kv:]
    qo = torch.full((layers, sum(new) + pad, n_q, D), 7.0, dtype=torch.bfloat16, device=DEV)
    Kd, Vd, td, ln, pd, fd, od = _dev(K, V, table, torch.tensor(lens, dtype=torch.int32), pos, freq, off)
    kv.paged_append(dims, layers, spec, fd, pd, q, k, v, od, ln, td, qo, Kd, Vd)
    assert kv.last_device_status() == 0
    n = sum(new)
    qc, kc, vc = qkv[:, :, :n_q], qkv[:, :, n_q:n_q + n_kv], qkv[:, :, n_q + n_kv:]
    ref_q = turned(qc, pos, freq, spec.axis_of_pair, adjacent)
    close_turned(qo.cpu()[:, :n], ref_q[:, :n], turned_bound(qc, spec.axis_of_pair, adjacent)[:, :n])
    assert bool((qo.cpu()[:, n:] == 7.0).all())                                    # padding rows
    want_k, bound, want_v = K.double(), torch.zeros_like(K.double()), V.clone()
    _place(want_k, turned(kc, pos, freq, spec.axis_of_pair, adjacent), table, lens, new, page)
    _place(bound, turned_bound(kc, spec.axis_of_pair, adjacent), table, lens, new, page)
    _place(want_v, vc, table, lens, new, page)
    close_turned(Kd.cpu(), want_k, bound)
    untouched = bound.sum(-1) == 0                                                 # every other slot bit for bit
    assert torch.equal(Kd.cpu()[untouched], K[untouched]) and torch.equal(Vd.cpu(), want_v)
    # without a rotation and without queries: copies
    kv.paged_append(dims, layers, None, None, None, None, k, v, od, ln, td, None, Kd, Vd)
    want = K.clone()
    _place(want, kc, table, lens, new, page)
    assert torch.equal(Kd.cpu(), want)


def test_append_of_single_tokens_with_idle_sequences():
    import rank_compressed_kv_b200 as kv
    lens = [1, 0, 17, 64, 0, 300]
    dims, _, table, K, V, qkv, pos, spec, _ = _append_case(kv, 1, 1, lens, [1] * 6, -0, 16, 8, 64)
    freq = spec.frequencies(1e4, "cpu")
    d = qkv[0].to(DEV)
    Kd, Vd, td, ln, pd, fd = _dev(K, V, table, torch.tensor(lens, dtype=torch.int32), pos, freq)
    before = d.clone()
    kv.paged_append(dims, 1, spec, fd, pd, d[:, :16], d[:, 16:24], d[:, 24:], None, ln, td, d[:, :16], Kd, Vd)   # q in place
    assert kv.last_device_status() == 0
    ref = turned(qkv[0, :, :16], pos, freq, spec.axis_of_pair)
    bound = turned_bound(qkv[0, :, :16], spec.axis_of_pair)
    live = torch.tensor(lens) > 0
    close_turned(d[:, :16].cpu()[live], ref[live], bound[live])
    assert torch.equal(d[~live.to(DEV)], before[~live.to(DEV)]) and torch.equal(d[:, 16:], before[:, 16:])
    want_v, want_k = V.clone(), turned(qkv[0, :, 16:24], pos, freq, spec.axis_of_pair)
    kb = turned_bound(qkv[0, :, 16:24], spec.axis_of_pair)
    rest = torch.ones(K.shape[1], 64, dtype=torch.bool)
    for b, n in enumerate(lens):
        if n:
            page, at = int(table[b, (n - 1) // 64]), (n - 1) % 64
            want_v[0, page, :, at] = qkv[0, b, 24:]
            close_turned(Kd[0, page, :, at].cpu(), want_k[b], kb[b])
            rest[page, at] = False
    assert torch.equal(Vd.cpu(), want_v)
    assert torch.equal(Kd.cpu().permute(1, 3, 0, 2, 4)[rest], K.permute(1, 3, 0, 2, 4)[rest])


# --------------------------------------------------------------------------- together, as they are used


def test_prompts_and_steps_together():
    """Ragged prompts appended, then steps of append and attention on a captured graph, with lengths, positions and
    inputs advanced between replays; every step's attention is the fp64 attention over what was appended."""
    import rank_compressed_kv_b200 as kv
    n_q, n_kv, page, B, steps = 28, 4, 32, 4, 5
    g = torch.Generator().manual_seed(77)
    new = [45, 1, 200, 31]
    table, n_pages = pages_for([n + steps for n in new], page, g)
    dims = kv.PagedDims(B, n_q, n_kv, page, n_pages, table.shape[1])
    spec = kv.Rope(n_axes=3, sections=(16, 24, 24))
    freq = spec.frequencies(1e6, "cpu")
    K = torch.full((1, n_pages, n_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    V = torch.full_like(K, float("nan"))
    td, fd = table.to(DEV), freq.to(DEV)
    x = normal(g, sum(new), n_q + 2 * n_kv, D)
    pos = torch.randint(0, 400, (3, sum(new)), generator=g, dtype=torch.int32)
    lens = torch.tensor(new, dtype=torch.int32, device=DEV)
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    d = x.to(DEV)
    kv.paged_append(dims, 1, spec, fd, pos.to(DEV), None, d[:, n_q:n_q + n_kv], d[:, n_q + n_kv:], off, lens, td, None, K, V)

    xs = torch.zeros(B, n_q + 2 * n_kv, D, dtype=torch.bfloat16, device=DEV)
    ps = torch.zeros(3, B, dtype=torch.int32, device=DEV)
    qr, out = torch.zeros(B, n_q, D, dtype=torch.bfloat16, device=DEV), torch.zeros(B, n_q, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(B, n_q, device=DEV)
    ws = torch.empty(kv.paged_decode_workspace(dims, 1), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.paged_append(dims, 1, spec, fd, ps, xs[:, :n_q], xs[:, n_q:n_q + n_kv], xs[:, n_q + n_kv:], None, lens, td, qr, K, V)
        kv.paged_decode_attn(dims, 1, qr, K, V, td, lens, D ** -0.5, out, lse, ws)

    keys = list(torch.split(x[:, n_q:n_q + n_kv], new))
    vals = list(torch.split(x[:, n_q + n_kv:], new))
    poss = list(torch.split(pos, new, dim=1))
    for step in range(steps):
        xn = normal(g, B, n_q + 2 * n_kv, D)
        pn = torch.randint(400, 500, (3, B), generator=g, dtype=torch.int32)
        xs.copy_(xn)
        ps.copy_(pn)
        lens += 1
        graph.replay()
        got_q, got_o, got_l = qr.cpu(), out.cpu(), lse.cpu()
        close_turned(got_q, turned(xn[:, :n_q], pn, freq, spec.axis_of_pair), turned_bound(xn[:, :n_q], spec.axis_of_pair))
        Kc, Vc = K.cpu(), V.cpu()
        now = lens.tolist()
        for b in range(B):
            keys[b] = torch.cat([keys[b], xn[b:b + 1, n_q:n_q + n_kv]])
            vals[b] = torch.cat([vals[b], xn[b:b + 1, n_q + n_kv:]])
            poss[b] = torch.cat([poss[b], pn[:, b:b + 1]], 1)
            at = torch.arange(now[b])
            pg = table[b][at // page].long()
            close_turned(Kc[0, pg, :, at % page], turned(keys[b], poss[b], freq, spec.axis_of_pair),
                         turned_bound(keys[b], spec.axis_of_pair))
            assert torch.equal(Vc[0, pg, :, at % page], vals[b])
        close_attend(got_o, got_l, attend(got_q, Kc, Vc, table, now, page, D ** -0.5))
    assert kv.last_device_status() == 0


@pytest.mark.parametrize("wide", WIDE)
def test_launches_behind_one_another_see_what_came_before(wide):
    """Steps without a wait between them (kernels start before their predecessors end): inputs, lengths and table written
    by the kernel just before, append, attention, and an overwrite of the inputs right behind; bit for bit as with waits."""
    import rank_compressed_kv_b200 as kv
    n_q, n_kv, page, B = 32, 8, 32, 6
    g = torch.Generator().manual_seed(5)
    start = [300, 1, 77, 640, 0, 31]
    steps = 12
    table, n_pages = pages_for([n + steps for n in start], page, g, wide=wide)
    dims = kv.PagedDims(B, n_q, n_kv, page, n_pages, table.shape[1])
    spec = kv.Rope(n_axes=2)
    freq = spec.frequencies(1e4)
    K0, V0 = normal(g, 1, n_pages, n_kv, page, D).to(DEV), normal(g, 1, n_pages, n_kv, page, D).to(DEV)
    xs = normal(g, steps, B, n_q + 2 * n_kv, D).to(DEV)
    noise = torch.randn(4096, 4096, device=DEV)
    ws = torch.empty(kv.paged_decode_workspace(dims, 1), dtype=torch.uint8, device=DEV)

    def play(wait):
        K, V = K0.clone(), V0.clone()
        x, q = torch.zeros_like(xs[0]), torch.zeros(B, n_q, D, dtype=torch.bfloat16, device=DEV)
        lens, td = torch.tensor(start, dtype=torch.int32, device=DEV), torch.full_like(table, -1, device=DEV)
        real = table.to(DEV)
        pos = torch.zeros(2, B, dtype=torch.int32, device=DEV)
        outs = []
        for i in range(steps):
            noise @ noise                                  # something to still be running
            x.copy_(xs[i])
            td.copy_(real)
            pos.copy_(lens[None].expand(2, B))
            lens += 1
            if wait:
                torch.cuda.synchronize()
            kv.paged_append(dims, 1, spec, freq, pos, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], None, lens, td, q, K, V)
            if wait:
                torch.cuda.synchronize()
            out, lse = torch.empty_like(q), torch.empty(B, n_q, device=DEV)
            kv.paged_decode_attn(dims, 1, q, K, V, td, lens, 0.1, out, lse, ws)
            x.fill_(float("nan"))
            q.fill_(float("nan"))
            td.fill_(-1)
            outs += [out, lse]
            if wait:
                torch.cuda.synchronize()
        return outs + [K, V]

    with_waits, without = play(True), play(False)
    assert kv.last_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(with_waits, without))
    assert not any(bool(torch.isnan(t).any()) for t in without)


def _paged_tail(c, w, n_layers, lens, page, seed, wide):
    """The dense text tails K_text, V_text [units][L][4][128] of a decode case as pools and a table."""
    g = torch.Generator().manual_seed(seed)
    table, n_pages = pages_for(lens, page, g, wide=wide)
    pools = []
    for name in ("K_text", "V_text"):
        dense = torch.from_numpy(c[name].view(np.int16)).view(torch.bfloat16)
        dense = dense.view(n_layers, w.batch, w.groups, -1, 4, D)
        X = torch.full((n_layers, n_pages, w.n_kv, page, D), float("nan"), dtype=torch.bfloat16)
        for b, n in enumerate(lens):
            at = torch.arange(n)
            rows = dense[:, b, :, :n].permute(0, 2, 1, 3, 4).reshape(n_layers, n, w.n_kv, D)
            X[:, table[b][at // page].long(), :, at % page] = rows.transpose(0, 1)
        pools.append(X.to(DEV))
    return pools[0], pools[1], table.to(DEV), n_pages


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("batch,layers,n_q,n_kv,T,lens,rank_lo", [
    (2, 2, 8, 8, 300, [45, 45], 16), (3, 1, 32, 8, 700, [0, 1, 130], 16), (2, 1, 28, 4, 1500, [17, 1000], 16),
    (2, 1, 32, 4, 600, [64, 0], 0), (1, 1, 8, 8, 64, [0], 16),
    (2, 1, 16, 8, 200, [5000, 77], 16), (36, 1, 32, 32, 40, [0, 5, 40] * 12, 16)])
def test_decode_with_a_paged_text_tail_matches_the_oracle(batch, layers, n_q, n_kv, T, lens, rank_lo, wide):
    import rank_compressed_kv_b200 as kv
    w = synth.Workload("paged", 50 + T, batch, layers, n_q, n_kv, T, max(max(lens), 1), 1, "lowrank32")
    Lcap = w.text0
    c = cases.decode_case(w, n_layers=layers, T=T, Lcap=Lcap)
    K, V, table, n_pages = _paged_tail(c, w, layers, lens, 32, T, wide)
    dims = kv.Dims(batch=batch, n_q_heads=n_q, n_kv_heads=n_kv, T_vis=T, L_text_cap=0, rank_lo=rank_lo)
    pd = kv.PagedDims(batch, n_q, n_kv, 32, n_pages, table.shape[1])
    g = {k: bf(c[k]) for k in ("q", "CK_lo", "CK_hi", "BK", "CV_lo", "CV_hi", "BV")}
    out = torch.full((layers * batch, n_q, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    mass = torch.full((dims.units(layers), T), float("nan"), dtype=torch.float32, device=DEV)
    ws = torch.full((kv.decode_paged_workspace(dims, pd, layers),), 0xFF, dtype=torch.uint8, device=DEV)
    kv.decode_attn_paged(dims, pd, layers, g["q"], g["CK_lo"], g["CK_hi"], g["BK"], g["CV_lo"], g["CV_hi"], g["BV"], K, V,
                         table, torch.tensor(lens, dtype=torch.int32, device=DEV), u32(c["mask"]), 1.0, out, mass, ws)
    assert kv.last_device_status() == 0
    o, ms = out.float().cpu().numpy(), mass.cpu().numpy()
    refs = {n: oracle_decode(w, c, n, rank_lo=rank_lo) for n in set(lens)}
    for b, n in enumerate(lens):                      # the oracle has one text length for the batch: row by row
        ref_o, ref_m = refs[n]
        rows = [l * batch + b for l in range(layers)]
        units = [r * w.groups + G for r in rows for G in range(w.groups)]
        got_u = cases.per_unit_outputs(w, o)
        for u in units:
            assert np.abs(got_u[u] - ref_o[u]).max() <= 2e-2 * np.abs(ref_o[u]).max()
        np.testing.assert_allclose(ms[units], ref_m[units], rtol=1e-4, atol=1e-10)
    if len(set(lens)) == 1 and lens[0] > 0:           # the dense tail gives the same within the same tolerance
        od, md = torch.empty_like(out), torch.empty_like(mass)
        dd = kv.Dims(batch=batch, n_q_heads=n_q, n_kv_heads=n_kv, T_vis=T, L_text_cap=Lcap, rank_lo=rank_lo)
        w2 = torch.empty(kv.decode_workspace(dd, layers), dtype=torch.uint8, device=DEV)
        kv.decode_attn(dd, layers, g["q"], g["CK_lo"], g["CK_hi"], g["BK"], g["CV_lo"], g["CV_hi"], g["BV"], bf(c["K_text"]),
                       bf(c["V_text"]), lens[0], u32(c["mask"]), 1.0, od, md, w2)
        assert_decode_close(w, o, ms, cases.per_unit_outputs(w, od.float().cpu().numpy()), md.cpu().numpy())


def test_a_video_prompt_from_positions_to_the_step():
    """Keys rotated by (time, height, width) straight into the compression's input, compressed, and a decode step over
    them with text tokens that were appended to pages: the step is the attention over the cache's own factors."""
    import oracle
    import rank_compressed_kv_b200 as kv
    n_q, n_kv, T, page = 16, 4, 588, 32
    g = torch.Generator().manual_seed(123)
    spec = kv.Rope(n_axes=3, sections=(16, 24, 24))
    freq = spec.frequencies(1e6)
    i = torch.arange(T)
    pos = torch.stack([i // 196, (i // 14) % 14, i % 14]).int()
    base = torch.randn(24, n_kv * D, generator=g)                            # keys of rank 24 before the rotation, and noise
    k = (torch.randn(T, 24, generator=g) @ base / 5 + 0.05 * torch.randn(T, n_kv * D, generator=g)).bfloat16().view(T, n_kv, D)
    v = (torch.randn(T, 24, generator=g) @ base / 5).bfloat16().view(T, n_kv, D)
    dims = kv.Dims(batch=1, n_q_heads=n_q, n_kv_heads=n_kv, T_vis=T, L_text_cap=0)
    X = torch.empty(1, 1, T, 4, D, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq, pos.to(DEV), None, None, k.to(DEV), X)
    sides = []
    wc = torch.empty(kv.compress_workspace(dims, 1), dtype=torch.uint8, device=DEV)
    for x in (X, v.to(DEV)):
        lo, hi = (torch.empty(1, T, r, dtype=torch.bfloat16, device=DEV) for r in (16, 48))
        B = torch.empty(1, 64, 512, dtype=torch.bfloat16, device=DEV)
        kv.compress(dims, 1, x.reshape(1, T, 512), lo, hi, B, None, wc)
        sides.append((lo, hi, B))
    # a spectrum this flat past the rank (rotated keys, values without noise) may stop the eigen-solver at its
    # iteration cap; its last iterate is written then, and what follows holds for any factors
    assert kv.last_device_status() in (0, 6)
    new = [70]
    table, n_pages = pages_for(new, page, g)
    pd = kv.PagedDims(1, n_q, n_kv, page, n_pages, table.shape[1])
    K = torch.full((1, n_pages, n_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    V = torch.full_like(K, float("nan"))
    x = normal(g, 70, n_q + 2 * n_kv, D).to(DEV)
    at = (T + torch.arange(70)).int().expand(3, 70).contiguous().to(DEV)
    off, ln = torch.tensor([0, 70], dtype=torch.int32, device=DEV), torch.tensor(new, dtype=torch.int32, device=DEV)
    qr = torch.empty(70, n_q, D, dtype=torch.bfloat16, device=DEV)
    kv.paged_append(pd, 1, spec, freq, at, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], off, ln, table.to(DEV), qr, K, V)
    q = (qr[69:70] * 0.1).contiguous()
    mask = torch.full((1, (T + 31) // 32), -1, dtype=torch.int32, device=DEV)
    out, mass = torch.empty(1, n_q, D, dtype=torch.bfloat16, device=DEV), torch.empty(1, T, device=DEV)
    ws = torch.empty(kv.decode_paged_workspace(dims, pd, 1), dtype=torch.uint8, device=DEV)
    (kl, kh, kb), (vl, vh, vb) = sides
    kv.decode_attn_paged(dims, pd, 1, q, kl, kh, kb, vl, vh, vb, K, V, table.to(DEV), ln, mask, 1.0, out, mass, ws)
    assert kv.last_device_status() == 0
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    idx = torch.arange(70)
    pg = table[0][idx // page].long()
    Kt, Vt = (f(P[0].cpu()[pg, :, idx % page])[None] for P in (K, V))
    ref_o, ref_m = oracle.decode(f(torch.cat([kl, kh], -1)), f(kb), f(torch.cat([vl, vh], -1)), f(vb), Kt, Vt,
                                 np.full((1, (T + 31) // 32), 0xFFFFFFFF, dtype=np.uint32), f(q).reshape(1, n_q, D), scale=1.0)
    assert np.abs(out.double().cpu().numpy().reshape(ref_o.shape) - ref_o).max() <= 2e-2 * np.abs(ref_o).max()
    np.testing.assert_allclose(mass.cpu().numpy(), ref_m, rtol=1e-4, atol=1e-10)
