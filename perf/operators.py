"""What is measured of the position and paged-cache operators, and their plain forms.

Three operators, each a case's "op":

  rope     rotary positions with one or several axes (time, height, width), queries and keys of a
           prompt; the keys may go straight into the layout that the cache compression takes
  append   queries, keys and values of new tokens: keys rotated and written with the values into
           their sequences' pages, queries rotated
  attend   attention of one new token per sequence over its pages

Pools are [layers][pages][n_kv][page][128] bf16, a block table row per sequence names its pages.
"""
import math

import torch

own = False

D = 128
THETA = 1e6
DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # rotation of four sequences' single new tokens: nothing but latency
        dict(name="rope step b4", op="rope", batch=4, tokens=1, n_q=32, n_kv=8, rotary=128, axes=1, interleaved=False,
             adjacent=False, inverse=False, units=False, base=70000),
        # one image's 576 patches, 32 heads of each kind, keys laid out for the compression
        dict(name="rope image 576", op="rope", batch=1, tokens=576, n_q=32, n_kv=32, rotary=128, axes=3,
             interleaved=False, adjacent=False, inverse=False, units=True, base=35),
        # the gradient of a partial rotation, adjacent pairs, an odd number of tokens
        dict(name="rope gradient 2x2305", op="rope", batch=2, tokens=2305, n_q=32, n_kv=8, rotary=64, axes=2,
             interleaved=True, adjacent=True, inverse=True, units=False, base=0),
        # sixteen videos of 32 frames of 196 patches, keys laid out for the compression
        dict(name="rope video 16x6272", op="rope", batch=16, tokens=6272, n_q=28, n_kv=4, rotary=128, axes=3,
             interleaved=False, adjacent=False, inverse=False, units=True, base=100),
        # one decode step of sixteen sequences
        dict(name="append step b16", op="append", batch=16, new=1, ragged=False, pad=0, cached=6900, n_q=28, n_kv=4,
             rotary=128, axes=3, page=64),
        # one decode step of a large batch
        dict(name="append step b256", op="append", batch=256, new=1, ragged=False, pad=0, cached=700, n_q=32, n_kv=32,
             rotary=128, axes=1, page=16),
        # ragged prompts of up to 6272 tokens in one call, with padding rows behind the last
        dict(name="append prompts 16x6272", op="append", batch=16, new=6272, ragged=True, pad=37, cached=130, n_q=28,
             n_kv=4, rotary=128, axes=3, page=64),
        # one sequence with a short cache: latency
        dict(name="attend b1 608", op="attend", layers=1, batch=1, longest=608, ragged=False, empty=0, n_q=32, n_kv=32,
             page=16),
        # a batch of image prompts, one query head per cached head
        dict(name="attend b64 704", op="attend", layers=1, batch=64, longest=704, ragged=False, empty=0, n_q=32,
             n_kv=32, page=16),
        # a ragged batch, two idle rows among it
        dict(name="attend b32 ragged 2561", op="attend", layers=1, batch=32, longest=2561, ragged=True, empty=2, n_q=32,
             n_kv=8, page=32),
        # video prompts of several layers in one call, seven query heads per cached head
        dict(name="attend b16 6785 x4", op="attend", layers=4, batch=16, longest=6785, ragged=True, empty=0, n_q=28,
             n_kv=4, page=64),
        # four long contexts
        dict(name="attend b4 66560", op="attend", layers=1, batch=4, longest=66560, ragged=False, empty=0, n_q=32,
             n_kv=8, page=128),
    ]


_HEADS = [(32, 32), (32, 8), (28, 4), (16, 8), (8, 4), (20, 4)]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend"])
    n_q, n_kv = rng.choice(_HEADS)
    if op == "rope":
        tokens = _spread(rng, 1, min(66000, 3_200_000 // (n_q + n_kv)))
        batch = _spread(rng, 1, max(1, min(64, 3_200_000 // (tokens * (n_q + n_kv)))))
        rotary = rng.choice([32, 64, 96, 128, 128, 128])
        return dict(op=op, batch=batch, tokens=tokens, n_q=n_q, n_kv=n_kv, rotary=rotary, axes=rng.choice([1, 2, 3, 3, 4]),
                    interleaved=rng.random() < 0.4, adjacent=rng.random() < 0.4, inverse=rng.random() < 0.3,
                    units=rng.random() < 0.5, base=_spread(rng, 1, 1_000_000))
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        if rng.random() < 0.5:
            batch, new = _spread(rng, 1, 512), 1
        else:
            new = _spread(rng, 2, 8000)
            batch = _spread(rng, 1, max(1, min(64, 3_200_000 // (new * (n_q + 2 * n_kv)))))
        cached = _spread(rng, 1, max(1, min(8000, 6_000_000 // (batch * n_kv))))
        return dict(op=op, batch=batch, new=new, ragged=new > 1, pad=rng.choice([0, 1, 37]) if new > 1 else 0,
                    cached=cached, n_q=n_q, n_kv=n_kv, rotary=rng.choice([64, 128, 128]), axes=rng.choice([1, 3]), page=page)
    longest = _spread(rng, 1, min(132000, 2_000_000 // n_kv))
    batch = _spread(rng, 1, max(1, min(256, 2_000_000 // (longest * n_kv))))
    layers = rng.choice([1, 1, 2, 3]) if batch * longest * n_kv * 3 <= 2_000_000 else 1
    empty = rng.choice([0, 0, 1, 2]) if batch > 2 else 0
    return dict(op=op, layers=layers, batch=batch, longest=longest, ragged=rng.random() < 0.7, empty=empty, n_q=n_q,
                n_kv=n_kv, page=page)


def _lengths(case):
    """The sequences' lengths, ascending (prepare() shuffles them)."""
    if case["op"] == "append":
        b, n = case["batch"], case["new"]
        return [max(1, n * (i + 1) // b) if case["ragged"] else n for i in range(b)]
    b, n, e = case["batch"], case["longest"], case["empty"]
    return [0 if i < e else max(1, n * (i + 1) // b) if case["ragged"] else n for i in range(b)]


def work(case):
    heads = case["n_q"] + case["n_kv"]
    if case["op"] == "rope":
        rows = case["batch"] * case["tokens"]
        return {"bytes": rows * (heads * D * 4 + 4 * case["axes"]), "flops": rows * heads * case["rotary"] * 3}
    if case["op"] == "append":
        rows = sum(_lengths(case))
        return {"bytes": rows * ((heads + case["n_kv"]) * D * 4 + 4 * case["axes"] + 4),
                "flops": rows * heads * case["rotary"] * 3}
    tokens, units = sum(_lengths(case)), case["layers"] * case["batch"]
    return {"bytes": tokens * case["layers"] * case["n_kv"] * D * 4 + units * case["n_q"] * (D * 4 + 4),
            "flops": tokens * case["layers"] * case["n_q"] * D * 4}


# ---------------------------------------------------------------------------------------- prepare


def _positions(case, rows, g):
    """int32 [axes][rows...]: a running position, or a grid of frames, rows and columns."""
    i = torch.arange(rows, device=DEV)
    start = case.get("base", case.get("cached", 0)) + int(torch.randint(0, 64, (1,), generator=g, device=DEV))
    if case["axes"] == 1:
        return (start + i)[None].int()
    w = 14
    grid = torch.stack([i // (w * w), (i // w) % w, i % w, i // 7])[: case["axes"]]
    return (start + grid).int()


def _axis_of_pair(case):
    n, a = case["rotary"] // 2, case["axes"]
    if case.get("interleaved"):
        return [p % a for p in range(n)]
    first = n // 4 if a > 1 else n                      # a quarter for the time axis, the rest shared evenly
    return [0 if p < first else 1 + (p - first) * (a - 1) // (n - first) for p in range(n)]


def _pages(case, need, g):
    """Block table and number of pages for `need` tokens in each sequence: pages in a random order, -1 where none is."""
    P = case["page"]
    count = [(n + P - 1) // P for n in need]
    total, wide = sum(count), max(1, max(count)) + 1
    order = torch.randperm(total + 3, generator=g, device=DEV).int()
    table = torch.full((case["batch"], wide), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total + 3


def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    n_q, n_kv = case["n_q"], case["n_kv"]
    s = {"case": case}
    if case["op"] != "attend":
        n = case["rotary"] // 2
        s["freq"] = THETA ** (-torch.arange(n, dtype=torch.float64, device=DEV) / n)
        s["axis"] = _axis_of_pair(case)
        s["axis_t"] = torch.tensor(s["axis"], device=DEV)
    if case["op"] == "rope":
        B, T = case["batch"], case["tokens"]
        qkv = _normal(g, B, T, n_q + 2 * n_kv, D)       # the projection's output: q, k and v of a token side by side
        s["q"], s["k"] = qkv[:, :, :n_q], qkv[:, :, n_q:n_q + n_kv]
        pos = _positions(case, T, g)
        shift = torch.randint(0, 50, (B,), generator=g, device=DEV).int()
        s["pos"] = (pos[:, None, :] + shift[None, :, None]).contiguous()
        s["q_out"] = torch.zeros(B, T, n_q, D, dtype=torch.bfloat16, device=DEV)
        shape = (B, n_kv // 4, T, 4, D) if case["units"] else (B, T, n_kv, D)
        s["k_out"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        return s
    order = torch.randperm(case["batch"], generator=g, device=DEV).tolist()
    lens = _lengths(case)
    lens = [lens[i] for i in order]
    if case["op"] == "append":
        had = [max(0, case["cached"] - (i % 13)) for i in order]
        s["lens"] = torch.tensor([a + b for a, b in zip(had, lens)], dtype=torch.int32, device=DEV)
        s["new"] = lens
        table, n_pages = _pages(case, [a + b for a, b in zip(had, lens)], g)
        rows = sum(lens)
        s["rows"] = rows
        s["offsets"] = None
        if case["ragged"]:
            s["offsets"] = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
        qkv = _normal(g, rows + case["pad"], n_q + 2 * n_kv, D)
        s["q"], s["k"], s["v"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        s["pos"] = _positions(case, rows + case["pad"], g).contiguous()
        s["q_out"] = torch.zeros(rows + case["pad"], n_q, D, dtype=torch.bfloat16, device=DEV)
        layers = 1
    else:
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        table, n_pages = _pages(case, lens, g)
        layers = case["layers"]
        # logits of a standard deviation near two: some tokens stand out, as they do in a trained model
        s["q"] = _normal(g, layers * case["batch"], n_q, D, scale=2.0)
        s["scale"] = D ** -0.5
        s["out"] = torch.zeros(layers * case["batch"], n_q, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(layers * case["batch"], n_q, dtype=torch.float32, device=DEV)
    s["table"] = table
    s["K"] = _normal(g, layers, n_pages, n_kv, case["page"], D)
    s["V"] = _normal(g, layers, n_pages, n_kv, case["page"], D)
    return s


# --------------------------------------------------------------------------------------- plain form


def _rotated(x, s, adjacent=False, inverse=False):
    """x [..., rows, heads, 128] rotated by s["pos"] [axes][..., rows]: 32 bits, the angles in 64."""
    n = len(s["axis"])
    angle = s["pos"][s["axis_t"]].movedim(0, -1).double() * s["freq"]
    c, w = angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)
    w = -w if inverse else w
    x = x.float()
    rot, rest = x[..., :2 * n], x[..., 2 * n:]
    if adjacent:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack([a * c - b * w, b * c + a * w], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :n], rot[..., n:]
        y = torch.cat([a * c - b * w, b * c + a * w], dim=-1)
    return torch.cat([y, rest], dim=-1).bfloat16()


def _plain_rope(s):
    c = s["case"]
    s["q_out"].copy_(_rotated(s["q"], s, c["adjacent"], c["inverse"]))
    k = _rotated(s["k"], s, c["adjacent"], c["inverse"])
    if c["units"]:
        B, T = c["batch"], c["tokens"]
        k = k.view(B, T, -1, 4, D).transpose(1, 2)
    s["k_out"].copy_(k)
    return s["q_out"], s["k_out"]


def _plain_append(s):
    c, n = s["case"], s["rows"]
    rows = torch.arange(n, device=DEV)
    if s["offsets"] is None:
        seq, index = rows, s["lens"].long() - 1
    else:
        off = s["offsets"].long()
        seq = torch.searchsorted(off, rows, right=True) - 1
        index = s["lens"].long()[seq] - off[seq + 1] + rows
    page = s["table"][seq, index // c["page"]].long()
    s["K"][0][page, :, index % c["page"]] = _rotated(s["k"], s)[:n]
    s["V"][0][page, :, index % c["page"]] = s["v"][:n]
    s["q_out"][:n] = _rotated(s["q"], s)[:n]
    return s["q_out"], s["K"], s["V"]


def _plain_attend(s):
    c = s["case"]
    L, B, n_q, n_kv = c["layers"], c["batch"], c["n_q"], c["n_kv"]
    at = s["table"].clamp(min=0).long()
    live = torch.arange(at.shape[1] * c["page"], device=DEV) < s["lens"][:, None]          # [B][T]
    q = s["q"].float().view(L, B, n_kv, n_q // n_kv, D)
    K = s["K"][:, at].float().transpose(2, 3).reshape(L, B, n_kv, -1, D)
    x = (q @ K.transpose(-1, -2) * s["scale"]).masked_fill(~live[None, :, None, None], -torch.inf)
    del K
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    V = s["V"][:, at].float().transpose(2, 3).reshape(L, B, n_kv, -1, D)
    out = e @ V / total.clamp(min=1e-30)
    lse = top + total.log()
    return out.view(L * B, n_q, D).bfloat16(), lse.view(L * B, n_q)


# -------------------------------------------------------------------------------------------- run


def _plan(s):
    """What a program of the framework keeps next to its buffers: the shapes, the rotation and a workspace."""
    import rank_compressed_kv_b200 as kv
    c = s["case"]
    s["kv"] = kv
    if c["op"] != "attend":
        s["rope"] = kv.Rope(rotary_dim=c["rotary"], n_axes=c["axes"], axis_of_pair=tuple(s["axis"]),
                            adjacent=bool(c.get("adjacent", False)))
    if c["op"] != "rope":
        s["dims"] = kv.PagedDims(batch=c["batch"], n_q_heads=c["n_q"], n_kv_heads=c["n_kv"], page_size=c["page"],
                                 n_pages=s["K"].shape[1], max_pages=s["table"].shape[1])
    if c["op"] == "attend":
        s["ws"] = torch.empty(kv.paged_decode_workspace(s["dims"], c["layers"]), dtype=torch.uint8, device=DEV)


def _own_run(s):
    if "kv" not in s:
        _plan(s)
    kv, c = s["kv"], s["case"]
    if c["op"] == "rope":
        kv.rope(s["rope"], s["freq"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"], inverse=c["inverse"])
        return s["q_out"], s["k_out"]
    if c["op"] == "append":
        kv.paged_append(s["dims"], 1, s["rope"], s["freq"], s["pos"], s["q"], s["k"], s["v"], s["offsets"], s["lens"],
                        s["table"], s["q_out"], s["K"], s["V"])
        return s["q_out"], s["K"], s["V"]
    kv.paged_decode_attn(s["dims"], c["layers"], s["q"], s["K"], s["V"], s["table"], s["lens"], s["scale"], s["out"],
                         s["lse"], s["ws"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ exact


def _turned(x, pos, freq, axis, adjacent, inverse):
    """x [rows][heads][128] times e^(i angle), pair by pair, as complex numbers in 64 bits."""
    n = len(axis)
    angle = torch.stack([pos[a].double() * freq[p] for p, a in enumerate(axis)], dim=-1)
    turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None]
    y = x.double().clone()
    i = torch.arange(n, device=DEV)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    z = torch.complex(y[..., a], y[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["case"]
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    k = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        how = s["pos"][:, b], s["freq"], s["axis"], c["adjacent"], c["inverse"]
        q[b] = _turned(s["q"][b], *how)
        y = _turned(s["k"][b], *how)
        if c["units"]:
            for h in range(c["n_kv"]):
                k[b, h // 4, :, h % 4] = y[:, h]
        else:
            k[b] = y
    return q, k


def _exact_append(s):
    c = s["case"]
    K, V, out = s["K"].double(), s["V"].double(), s["q_out"].double()
    row = 0
    for b, (n, end) in enumerate(zip(s["new"], s["lens"].tolist())):
        mine = slice(row, row + n)
        how = s["pos"][:, mine], s["freq"], s["axis"], False, False
        index = torch.arange(end - n, end, device=DEV)
        page, at = s["table"][b][index // c["page"]].long(), index % c["page"]
        K[0, page, :, at] = _turned(s["k"][mine], *how)
        V[0, page, :, at] = s["v"][mine].double()
        out[mine] = _turned(s["q"][mine], *how)
        row += n
    return out, K, V


def _exact_attend(s):
    c = s["case"]
    n_kv, per = c["n_kv"], c["n_q"] // c["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -torch.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // c["page"])].long()
        for layer in range(c["layers"]):
            row = layer * c["batch"] + b
            k = s["K"][layer, pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
            v = s["V"][layer, pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
            q = s["q"][row].double().view(n_kv, per, D)
            x = torch.einsum("jhd,jtd->jht", q, k) * s["scale"]
            out[row] = torch.einsum("jht,jtd->jhd", torch.softmax(x, -1), v).reshape(-1, D)
            lse[row] = torch.logsumexp(x, -1).reshape(-1)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
