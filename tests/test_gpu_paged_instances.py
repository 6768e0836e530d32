"""The position and paged-cache kernels at the sizes that choose among their compiled forms: the join of two and of four
warps a row, rotations and appends of many rows with partial quads and shares, and a whole prompt against what it was
made from."""
import math

import numpy as np
import pytest
import torch

import synth
import test_gpu_paged as paged
import test_gpu_rope as rope
from gpu_util import DEV, bf
from paged_util import D, close_turned, normal, pages_for, turned, turned_bound

pytestmark = pytest.mark.gpu

WIDE = 4200          # columns of the table to spare: runs over all units, and their join


# units of one query head (rows: not a multiple of the rows a block joins) and of seven; most of them in several runs
JOINS = [
    (1, [(53 * i) % 901 for i in range(67)], 1, 1, 16),                    # 67 units: four warps a row, two rows a block
    (1, [0, 3000] + [(61 * i) % 400 for i in range(15)], 28, 4, 32),       # 68 units of seven heads
    (3, [0, 1, 700, 16, 1200, 40, 900], 5, 5, 16),                         # 105 units, three layers
    (1, [(53 * i) % 901 for i in range(131)], 1, 1, 16),                   # 131 units: two warps a row, four rows a block
    (1, [0, 2000] + [(61 * i) % 400 for i in range(31)], 28, 4, 64),       # 132 units of seven heads
    (2, [(97 * i) % 777 for i in range(39)], 15, 3, 16),                   # 234 units, two layers
    (1, [(53 * i) % 700 for i in range(259)], 3, 1, 16),                   # 259 units of three heads
]


@pytest.mark.parametrize("layers,lens,n_q,n_kv,page", JOINS)
def test_joins_of_two_and_four_warps(layers, lens, n_q, n_kv, page):
    paged.test_attend_matches_fp64(layers, lens, n_q, n_kv, page, WIDE)


@pytest.mark.parametrize("batch,layers,n_q,n_kv,T,lens", [
    (17, 1, 28, 4, 64, [0, 400, 33] * 5 + [900, 1]),                       # four warps a row
    (33, 1, 20, 4, 64, [0, 300, 33] * 10 + [1000, 1, 16]),                 # two
    (9, 2, 32, 8, 40, [0, 300, 33] * 3),                                   # 144 units, two layers: two
])
def test_joins_into_the_decode_step(batch, layers, n_q, n_kv, T, lens):
    paged.test_decode_with_a_paged_text_tail_matches_the_oracle(batch, layers, n_q, n_kv, T, lens, 16, WIDE)


@pytest.mark.parametrize("batch,rows,n_q,n_k,rotary,axes,inter,adjacent,inverse", [
    (1, 4600, 32, 8, 64, 2, True, True, True),         # two shares of five quads, three at a time
    (2, 2999, 37, 9, 128, 3, False, False, False),     # between one and one and a half waves: two shares, partial quads
    (1, 5501, 37, 9, 128, 3, False, True, False),
    (1, 7500, 9, 6, 96, 2, True, True, False),         # a warp per row, four quads at a time and one more
    (1, 7300, 31, 1, 128, 1, False, True, True),       # eight quads and one
    (3, 2501, 11, 0, 128, 3, False, True, False),      # three quads, of queries alone
    (1, 1500, 45, 3, 128, 4, True, False, False),      # shares of three quads
    (1, 1501, 42, 3, 128, 4, True, True, False),       # of two
])
def test_rotations_of_many_rows(batch, rows, n_q, n_k, rotary, axes, inter, adjacent, inverse):
    if n_k > 0:
        rope.test_rope_matches_fp64(batch, rows, n_q, n_k, rotary, axes, inter, adjacent, inverse)
        return
    kv, spec = rope._spec(rotary, axes, inter, adjacent)
    g = torch.Generator().manual_seed(rows)
    x = normal(g, batch, rows, n_q, D)
    pos = torch.randint(0, 9000, (axes, batch, rows), generator=g, dtype=torch.int32)
    freq = spec.frequencies(1e4, "cpu")
    out = torch.full_like(x, 9.0, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), x.to(DEV), out, inverse=inverse)
    rope._check(kv, spec, freq, pos, x, out.cpu(), inverse)


@pytest.mark.parametrize("layers,had,new,pad,n_q,n_kv,page,rotary,axes,adjacent", [
    (1, [0, 100, 15], [3000, 4001, 2500], 37, 28, 4, 64, 128, 3, False),   # a warp per row, three quads at a time
    (1, [7, 0, 300, 16], [2500, 1, 0, 5000], 5, 21, 3, 32, 64, 2, True),   # adjacent, partial quads
    (2, [0, 40], [2000, 1700], 3, 28, 4, 16, 128, 1, False),
    (1, [0, 9], [2600, 3400], 1, 30, 6, 256, 96, 3, True),                 # two shares of a row's quads
    (1, [0, 9], [1300, 1201], 0, 32, 8, 16, 128, 3, False),                # shares of several quads, two at a time
])
def test_appends_of_many_rows(layers, had, new, pad, n_q, n_kv, page, rotary, axes, adjacent):
    paged.test_append_of_prompts(layers, had, new, pad, n_q, n_kv, page, rotary, axes, adjacent)


def test_a_prompt_against_the_keys_and_values_it_was_made_from():
    """Keys whose rotated form has the spectrum the compression is made for, rotated into its input and compressed, and a
    decode step over them and text in pages, against attention over the rotated keys and the values themselves.

    The factors are off by R = X - C B, held to the error of the best rank-64 approximation.  With d_t = scale q . R_t the
    weights change by the factor e^(d_t) / sum p e^d, so |ln mass'_t / mass_t| <= 2 max |d|, and the output by
    sum p |e^(d_t - c) - 1| |V_t| and what R of the values adds; the step itself is held to 1e-4 of the mass and 2 % of
    the largest output."""
    import rank_compressed_kv_b200 as kv
    n_q, n_kv, T, page, L = 16, 4, 1000, 32, 70
    w = synth.WORKLOADS["C0"]
    g = torch.Generator().manual_seed(9)
    spec = kv.Rope(n_axes=3, sections=(16, 24, 24))
    freq = spec.frequencies(1e6, "cpu")
    i = torch.arange(T)
    pos = torch.stack([i // 196, (i // 14) % 14, i % 14]).int()
    as_bf16 = lambda bits: torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).view(T, n_kv, D)  # noqa: E731
    x, v = (as_bf16(synth.visual_kv(w, 0, 0, 0, kind, T)) for kind in (synth.K_VIS, synth.V_VIS))
    k = turned(x, pos, freq, spec.axis_of_pair, inverse=True).bfloat16()
    dims = kv.Dims(batch=1, n_q_heads=n_q, n_kv_heads=n_kv, T_vis=T, L_text_cap=0)
    X = torch.empty(1, 1, T, 4, D, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), None, None, k.to(DEV), X)
    close_turned(X.cpu().view(T, n_kv, D), turned(k, pos, freq, spec.axis_of_pair), turned_bound(k, spec.axis_of_pair))
    sides, off = [], []
    wc = torch.empty(kv.compress_workspace(dims, 1), dtype=torch.uint8, device=DEV)
    for side in (X, v.to(DEV)):
        lo, hi = (torch.empty(1, T, r, dtype=torch.bfloat16, device=DEV) for r in (16, 48))
        B = torch.empty(1, 64, 512, dtype=torch.bfloat16, device=DEV)
        kv.compress(dims, 1, side.reshape(1, T, 512), lo, hi, B, None, wc)
        assert kv.last_device_status() == 0
        sides += [lo, hi, B]
        full = side.reshape(T, 512).double().cpu()
        rest = full - torch.cat([lo, hi], -1)[0].double().cpu() @ B[0].double().cpu()
        best = float(torch.linalg.svdvals(full)[64:].square().sum().sqrt())
        assert best <= float(rest.norm()) * (1 + 1e-9) and float(rest.norm()) <= 1.02 * best
        off.append(rest.view(T, n_kv, D))
    table, n_pages = pages_for([L], page, g)
    pd = kv.PagedDims(1, n_q, n_kv, page, n_pages, table.shape[1])
    K = torch.full((1, n_pages, n_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    V = torch.full_like(K, float("nan"))
    text = normal(g, L, n_q + 2 * n_kv, D)
    at = (T + torch.arange(L)).int().expand(3, L).contiguous()
    d = text.to(DEV)
    rows, ln = torch.tensor([0, L], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV)
    qr = torch.empty(L, n_q, D, dtype=torch.bfloat16, device=DEV)
    kv.paged_append(pd, 1, spec, freq.to(DEV), at.to(DEV), d[:, :n_q], d[:, n_q:n_q + n_kv], d[:, n_q + n_kv:], rows, ln,
                    table.to(DEV), qr, K, V)
    q = (qr[L - 1:] * 0.1).contiguous()
    mask = torch.full((1, (T + 31) // 32), -1, dtype=torch.int32, device=DEV)
    out, mass = torch.empty(1, n_q, D, dtype=torch.bfloat16, device=DEV), torch.empty(1, T, device=DEV)
    ws = torch.empty(kv.decode_paged_workspace(dims, pd, 1), dtype=torch.uint8, device=DEV)
    kv.decode_attn_paged(dims, pd, 1, q, *sides, K, V, table.to(DEV), ln, mask, 1.0, out, mass, ws)
    assert kv.last_device_status() == 0
    # the keys and values themselves: those of the image, and the text's, rotated in fp64
    kt = turned(text[:, n_q:n_q + n_kv], at, freq, spec.axis_of_pair).bfloat16().double()
    keys = torch.cat([X.cpu().view(T, n_kv, D).double(), kt])
    vals = torch.cat([v.double(), text[:, n_q + n_kv:].double()])
    qq = q.cpu().double().view(n_kv, n_q // n_kv, D)
    p = torch.softmax(torch.einsum("jhd,tjd->jht", qq, keys), -1)
    dt = torch.zeros_like(p)
    dt[..., :T] = -torch.einsum("jhd,tjd->jht", qq, off[0])
    most = float(dt.abs().max())
    want = p[..., :T].sum((0, 1))
    apart = (mass[0].double().cpu() / want).log().abs().max()
    assert float(apart) <= 2 * most + 1e-4
    assert float(want.log().std()) > most                      # the masses of other keys would be further apart than that
    c = torch.einsum("jht,jht->jh", p, dt.exp()).log()[..., None]
    p2 = p * (dt - c).exp()
    ref = torch.einsum("jht,tjd->jhd", p, vals)
    more = torch.einsum("jht,tjd->jhd", (p2 - p).abs(), vals.abs())
    more += torch.einsum("jht,tjd->jhd", p2[..., :T], off[1].abs())
    err = (out.cpu().double().view(ref.shape) - ref).abs()
    assert bool((err <= more + 2e-2 * float(ref.abs().max())).all())
    assert math.isfinite(float(err.max())) and float(more.max()) < float(ref.abs().max())
