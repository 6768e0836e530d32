"""Plain fp64 forms of the position and paged-cache operators, and draws for their tests (CPU, torch)."""
import math

import torch

D = 128
BF16_HALF = 2.0 ** -8          # eps / 2: a rounding to bf16 is off by at most this, relative to the value


def turned(x, pos, freq, axis, adjacent=False, inverse=False):
    """x [..., heads, 128] fp64 at positions pos [axes][...] (int): every pair turned by its angle."""
    n = len(axis)
    a = pos[torch.tensor(axis)].movedim(0, -1).double() * freq
    c, s = torch.cos(a).unsqueeze(-2), torch.sin(a).unsqueeze(-2)
    s = -s if inverse else s
    y = x.double().clone()
    i = torch.arange(n)
    p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    u, v = x[..., p].double(), x[..., q].double()
    y[..., p], y[..., q] = u * c - v * s, v * c + u * s
    return y


def turned_bound(x, axis, adjacent=False):
    """What the rotation's fp32 steps may be off by: angles, sines and products to 2^-20 of |x| + |y| of the pair."""
    n = len(axis)
    b = torch.zeros_like(x.double())
    i = torch.arange(n)
    p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    both = x[..., p].double().abs() + x[..., q].double().abs()
    b[..., p], b[..., q] = both, both
    return 2.0 ** -20 * b


def close_turned(got, ref, bound):
    err = (got.double() - ref).abs()
    tol = BF16_HALF * ref.abs() + (1 + BF16_HALF) * bound
    assert bool((err <= tol).all()), f"off by {float((err - tol).max()):.3e} more than allowed"


def attend(q, K, V, table, lens, page, scale):
    """q [L*B][n_q][128], K, V [L][pages][n_kv][page][128], in fp64.  Returns out, lse, and how far a kernel
    may be off: (abs of out beyond its rounding, abs of lse)."""
    L, n_kv = K.shape[0], K.shape[2]
    B, n_q = len(lens), q.shape[1]
    per = n_q // n_kv
    out = torch.zeros(L * B, n_q, D, dtype=torch.float64)
    lse = torch.full((L * B, n_q), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for l in range(L):
        for b, n in enumerate(lens):
            if n == 0:
                continue
            at = torch.arange(n)
            pg, r = table[b][at // page].long(), at % page
            k = K[l].double()[pg, :, r].transpose(0, 1)          # [n_kv][n][128]
            v = V[l].double()[pg, :, r].transpose(0, 1)
            qq = q[l * B + b].double().view(n_kv, per, D)
            s = torch.einsum("jhd,jtd->jht", qq, k) * scale
            p = torch.softmax(s, -1)
            out[l * B + b] = torch.einsum("jht,jtd->jhd", p, v).reshape(n_q, D)
            lse[l * B + b] = torch.logsumexp(s, -1).reshape(n_q)
            # 128 products of bf16 pairs summed in fp32: at most 2^-16 of the sum of magnitudes; the scaled
            # logit, the reference and their difference in the log2 domain: 2^-22 of the largest logit
            mag = torch.einsum("jhd,jtd->jht", qq.abs(), k.abs()) * scale
            ds = (2.0 ** -16 * mag + 2.0 ** -22 * (s.abs() + 1)).amax(-1)
            # p as bf16 hi + lo: 2^-16; sums and the joining of parts: 2^-18
            rel = 2 * ds + 2.0 ** -16 + 2.0 ** -18
            tol_o[l * B + b] = (torch.einsum("jht,jtd->jhd", p, v.abs()) * rel[..., None]).reshape(n_q, D)
            tol_l[l * B + b] = (ds + 2.0 ** -20 * (1 + lse[l * B + b].view(n_kv, per).abs())).reshape(n_q)
    return out, lse, tol_o, tol_l


def close_attend(got_o, got_l, ref):
    out, lse, tol_o, tol_l = ref
    err = (got_o.double() - out).abs()
    tol = BF16_HALF * out.abs() + (1 + BF16_HALF) * tol_o
    assert bool((err <= tol).all()), f"out off by {float((err - tol).max()):.3e} more than allowed"
    if got_l is not None:
        none = torch.isinf(lse)
        assert bool((got_l.double()[none] == lse[none]).all())
        err = (got_l.double() - lse)[~none].abs()
        assert bool((err <= tol_l[~none]).all()), f"lse off by {float((err - tol_l[~none]).max()):.3e} more than allowed"


def pages_for(lens, page, g, spare=3, wide=2, behind=-1):
    """Block table [B][..] over randomly ordered pages (entries behind a sequence's last: `behind`), number of pages."""
    count = [-(-n // page) for n in lens]
    n_pages = sum(count) + spare
    order = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lens), max(1, max(count)) + wide), behind, dtype=torch.int32)
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n].int()
        at += n
    return table, n_pages


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def blank_unused(X, table, lens, page, value):
    """Every slot that no sequence's tokens use set to value (pools [L][pages][n_kv][page][128], in place)."""
    used = torch.zeros(X.shape[1], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        at = torch.arange(n)
        used[table[b][at // page].long(), at % page] = True
    X.permute(1, 3, 0, 2, 4)[~used] = value
    return X
