"""What is measured of the operators around the latent and indexer-key caches: RMSNorm with the residual's
addition and an 8-bit output, rotary positions, the append to the caches, and MLA attention with a sliding
window and sinks.

``own`` chooses between their plain form (elementary torch operations in 32 bits, angles in 64, rounded once at
the end) and the calls of this repository's package.  ``exact`` gives the definition in 64 bits."""

import math

import torch

own = False

LATENT, VALUE, ROT = 576, 512, 64  # a latent row: 512 normalised dims, 64 rotated ones
PAGE = 64                          # tokens of a page of the caches
GROUP = 128                        # columns that share a scale of the 8-bit output, where it is not one a row
E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the norm before a block's projections, for a decode batch: residual stream kept, input of an 8-bit product
        dict(name="norm_decode_64x8192", op="norm", rows=64, cols=8192, dtype="bf16", residual=True, y=False, quant="group"),
        # the same for a long prompt, with one scale a token
        dict(name="norm_prompt_32768x4096", op="norm", rows=32768, cols=4096, dtype="bf16", residual=True, y=True, quant="row"),
        # a norm without a residual in half precision on an odd width, rows too narrow for wide loads
        dict(name="norm_odd_5003x1001", op="norm", rows=5003, cols=1001, dtype="f16", residual=False, y=True, quant="none"),
        # the gradient of a training step's norm, with the residual stream's own gradient joined
        dict(name="norm_backward_16384x5120", op="norm_backward", rows=16384, cols=5120, dtype="bf16", residual=True),
        # the query's rope dims of a decode batch at far positions, long-context frequencies
        dict(name="rope_decode_q_64x128x576", op="rope", rows=64, heads=128, dim=LATENT, offset=VALUE, rot=ROT, layout="interleaved",
             dtype="bf16", span=131072, factor=40.0, transpose=False),
        # a prompt's indexer queries: half layout, the first 64 of 128 dims
        dict(name="rope_prompt_index_q", op="rope", rows=16384, heads=64, dim=128, offset=0, rot=ROT, layout="half", dtype="bf16",
             span=131072, factor=40.0, transpose=False),
        # the gradient of the indexer queries (32 bits, as the indexer's backward writes it) back through the rotation
        dict(name="rope_backward_f32", op="rope", rows=6001, heads=64, dim=128, offset=0, rot=ROT, layout="half", dtype="f32", span=65536,
             factor=1.0, transpose=True),
        # one new token for each of 64 sequences
        dict(name="append_decode_64", op="append", rows=64, seqs=64, span=131072, d_i=128, layout="interleaved", key_layout="half"),
        # a chunk of a long prompt batch, ragged
        dict(name="append_prompt_65536", op="append", rows=65536, seqs=5, span=40000, d_i=128, layout="interleaved", key_layout="half"),
        # a prompt of two ragged sequences under a window of 1024 with 4 sinks
        dict(name="window_prefill_4093_w1024", op="window_prefill", tokens=4093, seqs=2, heads=128, window=1024, sinks=4),
        # a decode batch over long contexts, window of 4096
        dict(name="window_decode_64_w4096", op="window_decode", seqs=64, heads=128, ctx=32768, window=4096, sinks=16),
        # few long sequences with every key visible: the split along the keys
        dict(name="dense_decode_3_128k", op="window_decode", seqs=3, heads=128, ctx=131072, window=131072, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "rope", "rope", "append", "window_prefill", "window_decode"])
    if op in ("norm", "norm_backward"):
        cols = _log_int(rng, 1, 16384)
        if rng.random() < 0.6:
            cols = max(8, cols // 64 * 64)
        rows = _log_int(rng, 1, max(1, min(65536, 16384 * 4096 // cols)))
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), residual=rng.random() < 0.6)
        if op == "norm":
            c["quant"] = rng.choice(["none", "row", "group"])
            c["y"] = c["quant"] == "none" or rng.random() < 0.5
        return c
    if op == "rope":
        heads, dim = rng.choice([(1, 64), (1, 576), (64, 128), (128, 576), (8, 128), (5, 100), (3, 72)])
        rot = rng.choice([r for r in (2, 6, 32, 64) if r <= dim])
        return dict(op=op, rows=_log_int(rng, 1, max(1, 12000 * 64 * 128 // (heads * dim))), heads=heads, dim=dim,
                    offset=rng.choice([0, dim - rot]), rot=rot, layout=rng.choice(["interleaved", "half"]),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), span=rng.choice([4096, 131072, 1000000]),
                    factor=rng.choice([1.0, 8.0, 40.0]), transpose=rng.random() < 0.4)
    if op == "append":
        rows = _log_int(rng, 1, 65536)
        return dict(op=op, rows=rows, seqs=rng.randint(1, min(rows, 70)), span=rng.choice([70000, 100000, 131072]),
                    d_i=rng.choice([64, 128]), layout=rng.choice(["interleaved", "half"]), key_layout=rng.choice(["interleaved", "half"]))
    sinks = rng.choice([0, 1, 4, 16, 100])
    if op == "window_prefill":
        window = _log_int(rng, 1, 1024)
        return dict(op=op, tokens=_log_int(rng, 1, 4093), seqs=rng.randint(1, 6), heads=rng.choice([16, 128, 128]), window=window, sinks=sinks)
    if rng.random() < 0.7:
        return dict(op=op, seqs=_log_int(rng, 1, 64), heads=128, ctx=_log_int(rng, 1, 32768), window=_log_int(rng, 1, 4096), sinks=sinks)
    return dict(op=op, seqs=rng.randint(1, 3), heads=128, ctx=_log_int(rng, 1000, 131072), window=131072, sinks=0)


# ---- inputs --------------------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) + 101)
    return g


def _normal(shape, g, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = torch.randn((n,) + tuple(shape[1:]), generator=g, device="cuda").mul_(std)
    return out


def _freqs(rot, factor, theta=10000.0, original=4096.0, fast=32.0, slow=1.0):
    """Rotation in radians per position of each pair: plain, or blended for contexts `factor` times as long."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = theta ** (-2.0 * i / rot)
    if factor == 1.0:
        return f.cuda(), 1.0
    at = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(0, math.floor(at(fast))), min(rot - 1, math.ceil(at(slow)))
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return (f / factor * ramp + f * (1 - ramp)).cuda(), 0.1 * math.log(factor) + 1.0


def _split(total, parts, g):
    """`total` in `parts` ragged lengths that the seed gives (an empty one among them now and then)."""
    cut = torch.sort(torch.randint(0, total + 1, (parts - 1,), generator=g)).values.tolist()
    edges = [0] + cut + [total]
    return [b - a for a, b in zip(edges, edges[1:])]


def _pages(ctx, g, pool=None):
    """Scattered pages for contexts of these lengths: the block table, and how many pages the pool has."""
    need = [max(1, -(-c // PAGE)) for c in ctx]
    pool = pool or sum(need) + 3
    perm = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), pool


def prepare(case, seed):
    c, g, host = dict(case), _gen(seed), _gen(seed, "cpu")
    s = {"case": c}
    op = c["op"]
    if op in ("norm", "norm_backward"):
        dt, shape = DTYPES[c["dtype"]], (c["rows"], c["cols"])
        s["x"] = _normal(shape, g, dt)
        s["w"] = (1 + 0.1 * torch.randn(c["cols"], generator=g, device="cuda")).to(dt)
        s["res"] = _normal(shape, g, dt, 2.0) if c["residual"] else None
        if op == "norm":
            quant = c["quant"]
            s["y"] = torch.empty(shape, dtype=dt, device="cuda") if c["y"] else None
            s["res_out"] = torch.empty(shape, dtype=dt, device="cuda") if c["residual"] else None
            s["codes"] = torch.empty(shape, dtype=torch.uint8, device="cuda") if quant != "none" else None
            s["scale"] = {"none": None, "row": torch.empty(c["rows"], device="cuda") if quant == "row" else None,
                          "group": torch.empty((c["rows"], -(-c["cols"] // GROUP)), device="cuda") if quant == "group" else None}[quant]
        else:  # x is the sum that the forward pass normalised, res the gradient of the residual stream
            s["dy"] = _normal(shape, g, dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dh"] = torch.empty(shape, dtype=dt, device="cuda")
            s["dw"] = torch.empty(c["cols"], device="cuda")
    elif op == "rope":
        s["x"] = _normal((c["rows"], c["heads"], c["dim"]), g, DTYPES[c["dtype"]])
        s["pos"] = torch.randint(0, c["span"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
        s["freqs"], s["m"] = _freqs(c["rot"], c["factor"])
        s["out"] = torch.empty_like(s["x"])
    elif op == "append":
        n, b = c["rows"], c["seqs"]
        lens = [1] * b if n == b else [m + 1 for m in _split(n - b, b, host)]
        start = [int(torch.randint(0, max(1, c["span"] - m), (1,), generator=host)) for m in lens]
        s["seq"] = torch.cat([torch.full((m,), i, dtype=torch.int32) for i, m in enumerate(lens)]).cuda()
        s["pos"] = torch.cat([torch.arange(a, a + m, dtype=torch.int32) for a, m in zip(start, lens)]).cuda()
        s["table"], pool = _pages([m + PAGE for m in lens], host, n // PAGE + 2 * b + 3)
        # only the pages that the new tokens reach are in the pool: the table's rows hold them at their place
        full = torch.full((b, max(a // PAGE for a in start) + s["table"].shape[1]), -1, dtype=torch.int32, device="cuda")
        for i, a in enumerate(start):
            full[i, a // PAGE:a // PAGE + s["table"].shape[1]] = s["table"][i]
        s["table"] = full
        s["ctx"] = torch.tensor([a + m for a, m in zip(start, lens)], dtype=torch.int32, device="cuda")
        s["kv"] = _normal((n, LATENT), g, torch.bfloat16)
        s["w"] = (1 + 0.1 * torch.randn(VALUE, generator=g, device="cuda")).to(torch.bfloat16)
        s["key"] = _normal((n, c["d_i"]), g, torch.bfloat16)
        s["freqs"], s["m"] = _freqs(ROT, 40.0)
        s["latent"] = torch.zeros((pool, PAGE, LATENT), dtype=torch.bfloat16, device="cuda")
        s["codes"] = torch.zeros((pool, PAGE, c["d_i"]), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.ones((pool, PAGE), device="cuda")
    elif op == "window_prefill":
        n = c["tokens"]
        lens = _split(n, c["seqs"], host)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        s["max_len"] = max(lens)
        s["q"] = _normal((n, c["heads"], LATENT), g, torch.bfloat16, 2.0)
        s["latent"] = _normal((n, LATENT), g, torch.bfloat16)
        s["out"] = torch.empty((n, c["heads"], VALUE), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((n, c["heads"]), device="cuda")
    else:
        b = c["seqs"]
        ctx = torch.randint(max(1, c["ctx"] // 4), c["ctx"] + 1, (b,), generator=host).tolist()
        s["max_len"] = max(ctx)
        s["table"], pool = _pages(ctx, host)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["latent"] = _normal((pool, PAGE, LATENT), g, torch.bfloat16)
        s["q"] = _normal((b, c["heads"], LATENT), g, torch.bfloat16, 2.0)
        s["out"] = torch.empty((b, c["heads"], VALUE), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((b, c["heads"]), device="cuda")
    s["sm"] = 1.0 / math.sqrt(LATENT)
    return s


# ---- plain forms -----------------------------------------------------------------------------------

def _quantise(y, group):
    """e4m3 codes of y and their scales, one for `group` columns of a row (0: one a row)."""
    rows, cols = y.shape
    n = 1 if group == 0 else -(-cols // group)
    width = cols if group == 0 else group
    p = torch.nn.functional.pad(y, (0, n * width - cols)).reshape(rows, n, width)
    amax = p.abs().amax(2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    codes = (p / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(rows, n * width)[:, :cols], scale



def _plain_norm(s, c):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
        s["res_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    if s["y"] is not None:
        s["y"].copy_(y)
    if s["codes"] is not None:
        codes, scale = _quantise(y, GROUP if c["quant"] == "group" else 0)
        s["codes"].copy_(codes)
        s["scale"].copy_(scale.reshape(s["scale"].shape))


def _plain_norm_backward(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    gr = dy * s["w"].float()
    dh = r * (gr - h * (r * r * (gr * h).mean(1, keepdim=True)))
    if s["res"] is not None:
        dh = dh + s["res"].float()
    s["dh"].copy_(dh)
    s["dw"].copy_((dy * h * r).sum(0))


def _rotate(x, pos, freqs, m, layout, transpose=False):
    """x [rows, heads, rot] in 32 bits, turned by pos * freqs."""
    angle = (pos.double()[:, None] * freqs[None, :])[:, None, :]
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()
    if transpose:
        sin = -sin
    half = x.shape[2] // 2
    a, b = (x[:, :, 0::2], x[:, :, 1::2]) if layout == "interleaved" else (x[:, :, :half], x[:, :, half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), 3).flatten(2) if layout == "interleaved" else torch.cat((u, v), 2)


def _plain_rope(s, c):
    a, b = c["offset"], c["offset"] + c["rot"]
    s["out"].copy_(s["x"])
    s["out"][:, :, a:b] = _rotate(s["x"][:, :, a:b].float(), s["pos"], s["freqs"], s["m"], c["layout"], c["transpose"]).to(s["out"].dtype)


def _plain_append(s, c):
    pos, seq = s["pos"].long(), s["seq"].long()
    page, at = s["table"][seq, pos // PAGE].long(), pos % PAGE
    kv, key = s["kv"].float(), s["key"].float()
    n = kv[:, :VALUE]
    n = n * torch.rsqrt(n.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    r = _rotate(kv[:, None, VALUE:], s["pos"], s["freqs"], s["m"], c["layout"])[:, 0]
    s["latent"][page, at] = torch.cat((n, r), 1).bfloat16()
    k = torch.cat((_rotate(key[:, None, :ROT], s["pos"], s["freqs"], s["m"], c["key_layout"])[:, 0], key[:, ROT:]), 1)
    codes, scale = _quantise(k, 0)
    s["codes"][page, at] = codes
    s["scale"][page, at] = scale[:, 0]


def _soft(s, logits, visible, values):
    """softmax over the last axis where visible, then values: (out, lse)."""
    logits = logits.masked_fill(~visible, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    s["out"].copy_(values(p / total))
    s["lse"].copy_((top + torch.log(total))[..., 0])


def _plain_window_prefill(s, c):
    n, w, sinks = c["tokens"], min(c["window"], s["max_len"]), min(c["sinks"], s["max_len"])
    cu = s["cu"].long()
    tok = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu, tok, right=True) - 1
    first = cu[seq]
    lat = torch.nn.functional.pad(s["latent"].float(), (0, 0, w - 1, 0))   # w - 1 rows before the first token
    near = lat.as_strided((n, w, LATENT), (LATENT, LATENT, 1))              # row t: packed tokens t - w + 1 .. t
    at = tok[:, None] - (w - 1) + torch.arange(w, device="cuda")
    seen = at >= first[:, None]
    q = s["q"].float() * s["sm"]
    logits = torch.bmm(q, near.transpose(1, 2))
    visible = seen[:, None, :]
    if sinks == 0:
        return _soft(s, logits, visible, lambda p: torch.bmm(p, near[:, :, :VALUE]))
    rows = first[:, None] + torch.arange(sinks, device="cuda")
    begin = s["latent"].float()[rows.clamp(max=n - 1)]
    ahead = rows <= tok[:, None] - w
    logits = torch.cat((torch.bmm(q, begin.transpose(1, 2)), logits), 2)
    visible = torch.cat((ahead[:, None, :], visible), 2)
    return _soft(s, logits, visible,
                 lambda p: torch.bmm(p[:, :, :sinks], begin[:, :, :VALUE]) + torch.bmm(p[:, :, sinks:].contiguous(), near[:, :, :VALUE]))


def _plain_window_decode(s, c):
    w, sinks = min(c["window"], s["max_len"]), min(c["sinks"], s["max_len"])
    ctx = s["ctx"].long()[:, None]
    near = ctx - w + torch.arange(w, device="cuda")
    begin = torch.arange(sinks, device="cuda").expand(ctx.shape[0], sinks)
    pos = torch.cat((begin, near), 1)
    visible = torch.cat((begin < ctx - w, near >= 0), 1)
    pos = torch.where(visible, pos, torch.zeros_like(pos))
    rows = s["table"].long().gather(1, pos // PAGE) * PAGE + pos % PAGE
    k = s["latent"].reshape(-1, LATENT)[rows].float()
    logits = torch.bmm(s["q"].float() * s["sm"], k.transpose(1, 2))
    return _soft(s, logits, visible[:, None, :], lambda p: torch.bmm(p, k[:, :, :VALUE]))


# ---- the package's calls ----------------------------------------------------------------------------

def _handles(s, c):
    """What a program makes once for its caches: their descriptors and the workspace."""
    import sparse_attention_09_b200 as dsa
    s["dsa"] = dsa
    if c["op"] == "norm_backward":
        s["ws"] = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
    elif c["op"] == "append":
        room = s["table"].shape[1] * PAGE
        s["latents"] = dsa.paged_desc(s["latent"], s["table"], s["ctx"], room)
        s["keys"] = dsa.paged_desc(s["codes"], s["table"], s["ctx"], room, scale=s["scale"])
    elif c["op"] == "window_prefill":
        s["latents"] = dsa.contiguous_desc(s["latent"], s["cu"], s["max_len"])
    elif c["op"] == "window_decode":
        s["latents"] = dsa.paged_desc(s["latent"], s["table"], s["ctx"], s["max_len"])
        size = dsa.dsa_window_mla_workspace_size(c["seqs"], c["heads"], c["window"], c["sinks"], s["max_len"])
        s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return dsa


def _own(s, c):
    dsa, op = s.get("dsa") or _handles(s, c), c["op"]
    if op == "norm":
        dsa.dsa_rmsnorm(s["x"], s["w"], EPS, y=s["y"], residual=s["res"], residual_out=s["res_out"], codes=s["codes"], scale=s["scale"])
    elif op == "norm_backward":
        dsa.dsa_rmsnorm_backward(s["dy"], s["x"], s["w"], s["rstd"], s["dh"], s["dw"], s["ws"], dresidual=s["res"])
    elif op == "rope":
        dsa.dsa_rope(s["x"], s["pos"], s["freqs"], s["out"], c["offset"], c["rot"],
                     dsa.DSA_ROPE_INTERLEAVED if c["layout"] == "interleaved" else dsa.DSA_ROPE_HALF, s["m"], c["transpose"])
    elif op == "append":
        kinds = {"interleaved": dsa.DSA_ROPE_INTERLEAVED, "half": dsa.DSA_ROPE_HALF}
        dsa.dsa_cache_append(s["kv"], s["w"], EPS, s["key"], s["seq"], s["pos"], s["freqs"], s["latents"], s["keys"],
                             kinds[c["layout"]], kinds[c["key_layout"]], 0, s["m"])
    elif op == "window_prefill":
        dsa.dsa_window_mla_prefill(s["q"], s["latents"], c["seqs"], c["heads"], c["window"], c["sinks"], s["sm"], s["out"], s["lse"])
    else:
        dsa.dsa_window_mla_decode(s["q"], s["latents"], c["seqs"], c["heads"], c["window"], c["sinks"], s["sm"], s["out"], s["lse"], s["ws"])


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        _own(s, c)
    elif op == "norm":
        _plain_norm(s, c)
    elif op == "norm_backward":
        _plain_norm_backward(s)
    elif op == "rope":
        _plain_rope(s, c)
    elif op == "append":
        _plain_append(s, c)
    elif op == "window_prefill":
        _plain_window_prefill(s, c)
    else:
        _plain_window_decode(s, c)
    if op == "norm":
        out = {"y": s["y"], "residual": s["res_out"], "scale": s["scale"]}
        return dict(out, codes=s["codes"].view(torch.float8_e4m3fn)) if s["codes"] is not None else out
    if op == "norm_backward":
        return {"dh": s["dh"], "dw": s["dw"]}
    if op == "rope":
        return s["out"]
    if op == "append":
        return {"latent": s["latent"], "codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    c, op = case, case["op"]
    if op in ("norm", "norm_backward"):
        n, size = c["rows"] * c["cols"], 4 if c["dtype"] == "f32" else 2
        if op == "norm_backward":
            return {"bytes": n * size * (4 if c["residual"] else 3) + c["rows"] * 4 + c["cols"] * (size + 4), "flops": 10 * n}
        scales = {"none": 0, "row": 1, "group": -(-c["cols"] // GROUP)}[c["quant"]] * c["rows"]
        moved = n * size * (1 + 2 * c["residual"] + c["y"]) + c["cols"] * size + (n if c["quant"] != "none" else 0) + 4 * scales
        return {"bytes": moved, "flops": 6 * n}
    if op == "rope":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * c["rows"] * c["heads"] * c["dim"] * size + 4 * c["rows"] + 4 * c["rot"], "flops": 3 * c["rows"] * c["heads"] * c["rot"]}
    if op == "append":
        return {"bytes": c["rows"] * (2 * LATENT * 2 + 3 * c["d_i"] + 4 + 12) + 2 * VALUE, "flops": c["rows"] * (6 * LATENT + 6 * c["d_i"])}
    if op == "window_prefill":
        n = c["tokens"]
        per = n / c["seqs"]  # sequences of the mean length
        seen = min(per, c["window"] + c["sinks"])
        pairs = c["seqs"] * (seen * (seen + 1) / 2 + (per - seen) * seen)
        return {"bytes": n * (c["heads"] * (LATENT + VALUE) * 2 + LATENT * 2 + 4 * c["heads"]), "flops": 2 * c["heads"] * (LATENT + VALUE) * pairs}
    mean = 0.625 * c["ctx"]
    seen = c["seqs"] * min(mean, c["window"] + c["sinks"])
    return {"bytes": seen * LATENT * 2 + c["seqs"] * c["heads"] * ((LATENT + VALUE) * 2 + 4), "flops": 2 * c["heads"] * (LATENT + VALUE) * seen}


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def _turn64(x, pos, freqs, m, layout, sign=1.0):
    """Rotation as a product of complex numbers."""
    half = x.shape[-1] // 2
    z = torch.polar(torch.full_like(freqs, m).expand(pos.shape[0], -1).contiguous(), sign * pos.double().outer(freqs))
    pairs = x.unflatten(-1, (half, 2)) if layout == "interleaved" else x.unflatten(-1, (2, half)).transpose(-1, -2)
    t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z.reshape((x.shape[0],) + (1,) * (x.dim() - 2) + (half,)))
    return (t if layout == "interleaved" else t.transpose(-1, -2)).flatten(-2)


def _attend64(q, k, sm, visible):
    logits = torch.einsum("rhd,kd->rhk", q, k) * sm
    logits[~visible[:, None, :].expand_as(logits)] = -math.inf
    lse = torch.logsumexp(logits, 2)
    return torch.einsum("rhk,kv->rhv", torch.exp(logits - lse[:, :, None]), k[:, :VALUE]), lse


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS) * s["w"].double()
        scale = None
        if case["quant"] == "row":
            scale = torch.linalg.vector_norm(y, math.inf, dim=1) / E4M3_MAX
        elif case["quant"] == "group":
            scale = torch.stack([torch.linalg.vector_norm(p, math.inf, dim=1) for p in y.split(GROUP, 1)], 1) / E4M3_MAX
        out = {"y": y if case["y"] else None, "residual": h if case["residual"] else None, "scale": scale}
        return dict(out, codes=None) if scale is not None else out
    if op == "norm_backward":
        h, dy, w, r = s["x"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
        unit = h * r
        back = r * (dy * w) - r * unit * torch.einsum("rc,rc,c->r", unit, dy, w)[:, None] / h.shape[1]
        return {"dh": back + s["res"].double() if s["res"] is not None else back, "dw": torch.einsum("rc,rc->c", unit, dy)}
    if op == "rope":
        a, b = case["offset"], case["offset"] + case["rot"]
        x = s["x"].double()
        turned = _turn64(x[:, :, a:b], s["pos"], s["freqs"], s["m"], case["layout"], -1.0 if case["transpose"] else 1.0)
        return torch.cat((x[:, :, :a], turned, x[:, :, b:]), 2)
    if op == "append":
        slot = s["table"].long()[s["seq"].long(), s["pos"].long() // PAGE] * PAGE + s["pos"].long() % PAGE
        kv, key = s["kv"].double(), s["key"].double()
        latent, scale = s["latent"].double().flatten(0, 1), s["scale"].double().flatten()
        n = kv[:, :VALUE]
        n = n / torch.sqrt((n * n).sum(1, keepdim=True) / VALUE + EPS) * s["w"].double()
        latent[slot] = torch.cat((n, _turn64(kv[:, VALUE:], s["pos"], s["freqs"], s["m"], case["layout"])), 1)
        turned = _turn64(key[:, :ROT], s["pos"], s["freqs"], s["m"], case["key_layout"])
        scale[slot] = torch.maximum(turned.abs().amax(1), key[:, ROT:].abs().amax(1) if case["d_i"] > ROT else turned.abs().amax(1)) / E4M3_MAX
        return {"latent": latent.reshape(s["latent"].shape), "codes": None, "scale": scale.reshape(s["scale"].shape)}
    out, lse = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    q, window, sinks = s["q"].double(), case["window"], case["sinks"]
    if op == "window_prefill":
        cu = s["cu"].tolist()
        for a, b in zip(cu, cu[1:]):
            for t in range(a, b, 128):
                rows = torch.arange(t, min(b, t + 128), device="cuda")
                keys = torch.arange(a, int(rows[-1]) + 1, device="cuda")
                keys = keys[(keys > t - window) | (keys < a + sinks)]
                visible = (keys <= rows[:, None]) & ((keys > rows[:, None] - window) | (keys < a + sinks))
                out[rows], lse[rows] = _attend64(q[rows], s["latent"][keys].double(), s["sm"], visible)
    else:
        flat = s["latent"].reshape(-1, LATENT)
        for b, n in enumerate(s["ctx"].tolist()):
            pos = torch.arange(n, device="cuda")
            pos = pos[(pos >= n - window) | (pos < sinks)]
            k = flat[s["table"][b].long()[pos // PAGE] * PAGE + pos % PAGE].double()
            o, e = _attend64(q[b:b + 1], k, s["sm"], torch.ones((1, len(pos)), dtype=torch.bool, device="cuda"))
            out[b], lse[b] = o[0], e[0]
    return {"out": out, "lse": lse}
