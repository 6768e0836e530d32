"""kvpack_rope through the binding, against the rotation in fp64.

Tolerance: one rounding to bf16 (2^-8 of the value) and the fp32 steps, 2^-20 of the pair's magnitudes."""
import pytest
import torch

from paged_util import close_turned, normal, turned, turned_bound

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _spec(rotary, axes, inter, adjacent):
    import rank_compressed_kv_b200 as kv
    n = rotary // 2
    m = [p % axes if inter else p * axes // n for p in range(n)]
    return kv, kv.Rope(rotary_dim=rotary, n_axes=axes, axis_of_pair=m, adjacent=adjacent)


def _check(kv, spec, freq, pos, x, got, inverse=False):
    ref = turned(x, pos, freq, spec.axis_of_pair, spec.adjacent, inverse)
    close_turned(got, ref, turned_bound(x, spec.axis_of_pair, spec.adjacent))
    assert torch.equal(got[..., spec.rotary_dim:], x[..., spec.rotary_dim:])


@pytest.mark.parametrize("batch,rows,n_q,n_k,rotary,axes,inter,adjacent,inverse", [
    (1, 1, 1, 1, 128, 1, False, False, False),
    (1, 1, 32, 8, 128, 3, False, False, False),
    (2, 3, 5, 3, 128, 3, True, False, False),
    (1, 577, 28, 4, 128, 3, False, False, False),
    (3, 17, 8, 8, 64, 2, True, True, False),
    (1, 100, 7, 1, 16, 1, False, True, True),
    (2, 65, 4, 2, 96, 4, True, False, True),
    (1, 33, 32, 32, 128, 4, False, True, False),
    (1, 6001, 9, 6, 48, 3, False, False, False),
])
def test_rope_matches_fp64(batch, rows, n_q, n_k, rotary, axes, inter, adjacent, inverse):
    kv, spec = _spec(rotary, axes, inter, adjacent)
    g = torch.Generator().manual_seed(rows * 31 + n_q)
    qkv = normal(g, batch, rows, n_q + 2 * n_k, 128)
    pos = torch.randint(0, 9000, (axes, batch, rows), generator=g, dtype=torch.int32)
    freq = spec.frequencies(1e4, "cpu")
    d = qkv.to(DEV)
    q, k = d[:, :, :n_q], d[:, :, n_q:n_q + n_k]
    qo, ko = torch.full_like(q, 9.0, memory_format=torch.contiguous_format), torch.full_like(k, 9.0, memory_format=torch.contiguous_format)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), q, qo, k, ko, inverse=inverse)
    _check(kv, spec, freq, pos, qkv[:, :, :n_q], qo.cpu(), inverse)
    _check(kv, spec, freq, pos, qkv[:, :, n_q:n_q + n_k], ko.cpu(), inverse)
    # in place, and only the rotated heads change
    kv.rope(spec, freq.to(DEV), pos.to(DEV), q, q, inverse=inverse)
    assert torch.equal(q, qo)
    assert torch.equal(d[:, :, n_q:].cpu(), qkv[:, :, n_q:])


def test_far_and_negative_positions():
    kv, spec = _spec(128, 2, True, False)
    g = torch.Generator().manual_seed(5)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1_000_003, 16_777_217],
                        [2 ** 31 - 1, 2, -7, 0, 5, 123_456_789, -2 ** 30]], dtype=torch.int32)
    x = normal(g, 7, 4, 128)
    freq = spec.frequencies(1e6, "cpu")
    out = torch.empty(7, 4, 128, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), x.to(DEV), out)
    _check(kv, spec, freq, pos, x, out.cpu())


@pytest.mark.parametrize("heads,rows", [(8, 196), (4, 1), (32, 35)])
def test_keys_in_the_compression_layout(heads, rows):
    kv, spec = _spec(128, 3, False, False)
    g = torch.Generator().manual_seed(heads)
    x = normal(g, 2, rows, heads, 128)
    pos = torch.randint(0, 500, (3, 2, rows), generator=g, dtype=torch.int32)
    freq = spec.frequencies(1e6, "cpu")
    X = torch.empty(2, heads // 4, rows, 4, 128, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), None, None, x.to(DEV), X)
    got = X.cpu().transpose(1, 2).reshape(2, rows, heads, 128)
    _check(kv, spec, freq, pos, x, got)
    # and back from that layout
    back = torch.empty_like(x, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), X, back, inverse=True)
    _check(kv, spec, freq, pos, got, back.cpu(), inverse=True)


@pytest.mark.parametrize("rotary,adjacent", [(128, False), (64, True)])
def test_the_inverse_is_the_gradient(rotary, adjacent):
    """With y = rope(x): d<y, u>/dx is rope^-1(u) -- by the formula, and by differences of the kernel's own y
    (the rotation is linear: a step of 2^6 keeps the roundings small against it)."""
    kv, spec = _spec(rotary, 3, True, adjacent)
    g = torch.Generator().manual_seed(11)
    x, u = normal(g, 50, 4, 128), normal(g, 50, 4, 128)
    pos = torch.randint(0, 4000, (3, 50), generator=g, dtype=torch.int32)
    freq = spec.frequencies(1e4, "cpu")
    grad = torch.empty(50, 4, 128, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), u.to(DEV), grad, inverse=True)
    _check(kv, spec, freq, pos, u, grad.cpu(), inverse=True)
    def y(t):
        o = torch.empty(50, 4, 128, dtype=torch.bfloat16, device=DEV)
        kv.rope(spec, freq.to(DEV), pos.to(DEV), t.to(DEV), o)
        return o.cpu().double()
    for at in (0, 5, rotary // 2, rotary - 1, 127):
        step = torch.zeros_like(x)
        step[..., at] = 64.0
        diff = ((y(step) - y(-step)) * u.double()).sum(-1) / 128.0
        have = grad.cpu().double()[..., at]
        # y's two entries of the pair and grad are each rounded to bf16 once
        tol = 2.0 ** -8 * (2 * u.double().abs().amax(-1) + have.abs()) + 2.0 ** -18
        assert bool(((diff - have).abs() <= tol).all())


def test_nothing_outside_the_rows_is_written_and_empty_calls_do_nothing():
    kv, spec = _spec(128, 1, False, False)
    freq = spec.frequencies(1e4, DEV)
    big = torch.full((10, 6, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(4, 3, 128, dtype=torch.bfloat16, device=DEV)
    kv.rope(spec, freq, torch.arange(4, dtype=torch.int32, device=DEV)[None], x, big[3:7, :3])
    keep = torch.ones(10, 6, dtype=torch.bool)
    keep[3:7, :3] = False
    assert bool((big.cpu()[keep] == 3.0).all()) and not bool((big.cpu()[~keep] == 3.0).any())
    kv.rope(spec, freq, torch.empty(1, 0, dtype=torch.int32, device=DEV), x[:0], x[:0])


def test_strides_of_single_rows_do_not_matter():
    kv, spec = _spec(128, 1, False, False)
    freq = spec.frequencies(1e4, "cpu")
    x = normal(torch.Generator().manual_seed(1), 1, 1, 3, 128)
    odd = torch.as_strided(x.to(DEV), (1, 1, 3, 128), (7, 3, 128, 1))
    out = torch.empty(1, 1, 3, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([[[12]]], dtype=torch.int32)
    kv.rope(spec, freq.to(DEV), pos.to(DEV), odd, out)
    _check(kv, spec, freq, pos, x, out.cpu())


def test_captured_and_on_another_stream():
    kv, spec = _spec(128, 3, False, False)
    g = torch.Generator().manual_seed(3)
    freq = spec.frequencies(1e4, "cpu")
    x = normal(g, 40, 8, 128)
    pos = torch.randint(0, 999, (3, 40), generator=g, dtype=torch.int32)
    xd, pd, fd, out = x.to(DEV), pos.to(DEV), freq.to(DEV), torch.zeros(40, 8, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.rope(spec, fd, pd, xd, out)
    torch.cuda.current_stream().wait_stream(side)
    _check(kv, spec, freq, pos, x, out.cpu())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.rope(spec, fd, pd, xd, out)
    pos2 = torch.randint(0, 999, (3, 40), generator=g, dtype=torch.int32)
    pd.copy_(pos2)
    graph.replay()
    _check(kv, spec, freq, pos2, x, out.cpu())
