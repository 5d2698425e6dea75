"""dsa_window_mla_prefill / _decode against the float64 oracle.

Tolerances, from the arithmetic: an unnormalised probability is rounded to bf16 for the product with the
values (half a step, 2^-8 relative), the result once more: 2^-8 (sum_i p_i |v_i| + |out|) on each element, and
2^-10 of the first for the fp32 steps (logits: 576 exact products summed in fp32, at most 576 * 2^-24 of
sm_scale |q| |c|, here under 2^-11 absolute; the exponential 2^-22).  The row sum takes the unrounded
probabilities, so lse is within 2^-10 absolute."""
import math

import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(576)


def rnd(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def f64(t):
    return t.double().cpu().numpy()


def check_row(out, lse, q, latent, length, window, sinks, what):
    want, wlse = oracle.window_mla_token(q, latent, length, window, sinks, SM)
    sel = oracle.window_positions(length, window, sinks)
    if len(sel) == 0:
        assert (out == 0).all() and np.isneginf(lse).all(), what
        return
    p = np.exp(SM * (q @ latent[sel].T) - wlse[:, None])
    mag = p @ np.abs(latent[sel, :512])
    err, bound = np.abs(out - want), 2.0 ** -8 * (mag + np.abs(want)) + 2.0 ** -10 * mag
    assert np.all(err <= bound), f"{what}: {np.argwhere(~(err <= bound))[0]} {err.max()}"
    assert np.all(np.abs(lse - wlse) <= 2.0 ** -10), f"{what}: lse {np.abs(lse - wlse).max()}"


def prefill(lens, H, window, sinks, seed=0, rows=None, pad=0):
    T = sum(lens) + pad
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    q, latent = rnd((T, H, 576), seed, 2.0), rnd((T, 576), seed + 1)
    out = torch.full((T, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 3.0, device="cuda")
    dsa.dsa_window_mla_prefill(q, dsa.contiguous_desc(latent, cu, max(max(lens), 1)), len(lens), H, window, sinks, SM, out, lse)
    assert dsa.dsa_device_error() == 0
    qh, lh, oh, sh = f64(q), f64(latent), f64(out), f64(lse)
    edges = cu.tolist()
    for a, b in zip(edges, edges[1:]):
        for t in range(a, b):
            if rows is None or t - a in rows or t == b - 1:
                check_row(oh[t], sh[t], qh[t], lh[a:b], t - a + 1, window, sinks, (lens, H, window, sinks, t))
    assert (oh[edges[-1]:] == 3).all() and (sh[edges[-1]:] == 3).all(), "rows behind the last sequence were written"


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (63, 0), (64, 1), (65, 64), (100, 130), (2 ** 31 - 1, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)])
def test_prefill(window, sinks):
    prefill([1, 0, 63, 130, 64, 0], 128, window, sinks, rows=range(0, 130, 9))


@pytest.mark.parametrize("H", [1, 16, 63, 64, 65, 128])
def test_prefill_heads_and_rows_behind_the_last_sequence(H):
    prefill([70, 9], H, 20, 3, seed=H, rows=range(0, 70, 11), pad=37)


def test_prefill_long_window_over_many_tokens():
    prefill([700, 333], 128, 300, 4, rows=[0, 1, 299, 300, 303, 304, 305, 500])


def test_prefill_of_empty_sequences_writes_nothing():
    prefill([0, 0], 128, 8, 1, pad=5)


def paged_cache(ctx, seed=1, spare=2, fill=None):
    """(latent pool, block table, logical rows per sequence): scattered pages, unused slots NaN."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-c // 64) for c in ctx]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(ctx), max(max(need), 1)), -1, dtype=torch.int32)
    latent = torch.full((pool, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    logical, at = [], 0
    for b, c in enumerate(ctx):
        rows = rnd((c, 576), seed + 10 + b) if c else torch.zeros((0, 576), device="cuda").bfloat16()
        logical.append(rows)
        for j in range(need[b]):
            table[b, j] = perm[at]
            n = min(64, c - 64 * j)
            latent[perm[at], :n] = rows[64 * j:64 * j + n]
            at += 1
    return latent, table.cuda(), logical


def decode_call(q, latent, table, ctx, window, sinks, max_ctx=None, H=128, stream=None):
    B = q.shape[0]
    if not isinstance(ctx, torch.Tensor):
        ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    max_ctx = max_ctx or max(int(ctx.max()), 1)
    out = torch.full((B, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), 3.0, device="cuda")
    size = dsa.dsa_window_mla_workspace_size(B, H, window, sinks, max_ctx)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    dsa.dsa_window_mla_decode(q, dsa.paged_desc(latent, table, ctx, max_ctx), B, H, window, sinks, SM, out, lse, ws)
    return out, lse


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (65, 1), (100, 16), (1000, 130), (2 ** 31 - 1, 7)])
@pytest.mark.parametrize("ctx", [[1], [0, 1, 63, 64, 65, 0], [500, 3000, 129], [5, 700] * 40])
def test_decode(ctx, window, sinks):
    H = 128 if len(ctx) < 50 else 16
    latent, table, logical = paged_cache(ctx)
    q = rnd((len(ctx), H, 576), 5, 2.0)
    out, lse = decode_call(q, latent, table, ctx, window, sinks, H=H)
    assert dsa.dsa_device_error() == 0
    for b, c in enumerate(ctx):
        if b < 12 or b % 7 == 0:
            check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), c, window, sinks, (ctx, window, sinks, b))


@pytest.mark.parametrize("H", [1, 33, 64, 100])
def test_decode_heads(H):
    ctx = [300, 40, 1500]
    latent, table, logical = paged_cache(ctx)
    q = rnd((3, H, 576), 5, 2.0)
    for window in (700, 1400):  # whole sequences, shared out
        out, lse = decode_call(q, latent, table, ctx, window, 2, H=H)
        for b, c in enumerate(ctx):
            check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), c, window, 2, (H, window, b))


@pytest.mark.parametrize("ctx", [[5000, 0, 1, 64, 900, 0], [1] * 40 + [9000] + [70] * 40, [1500] * 75, [20000], [2000, 1] * 75])
def test_decode_shared_out(ctx):
    """Ragged batches whose chunks are shared out: sequences in one cluster, over several, over all; empty ones between."""
    H = 16
    assert dsa.dsa_window_mla_workspace_size(len(ctx), H, 2 ** 30, 0, 9000 if max(ctx) < 9000 else max(ctx)) > 0
    latent, table, logical = paged_cache(ctx)
    if table.shape[1] * 64 < 9000:  # room to declare longer contexts than there are
        table = torch.nn.functional.pad(table, (0, 141 - table.shape[1]), value=-1).contiguous()
    q = rnd((len(ctx), H, 576), 5, 2.0)
    for window, sinks in ((2 ** 30, 0), (1400, 70)):
        out, lse = decode_call(q, latent, table, ctx, window, sinks, H=H, max_ctx=max(9000, max(ctx)))
        assert dsa.dsa_device_error() == 0
        again = decode_call(q, latent, table, ctx, window, sinks, H=H, max_ctx=max(9000, max(ctx)))
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)  # the same parts in the same order
        for b, c in enumerate(ctx):
            if b < 8 or b % 9 == 0 or c > 4000 or b > len(ctx) - 3:
                check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), c, window, sinks, (window, b))


def test_decode_equals_the_last_prefill_row_and_the_sparse_path():
    L = 900
    latent, table, logical = paged_cache([L])
    q = rnd((L, 128, 576), 9, 2.0)
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    for window, sinks in ((200, 8), (L, 0)):
        out = torch.empty((L, 128, 512), dtype=torch.bfloat16, device="cuda")
        dsa.dsa_window_mla_prefill(q, dsa.contiguous_desc(logical[0], cu, L), 1, 128, window, sinks, SM, out)
        got, _ = decode_call(q[-1:].contiguous(), latent, table, [L], window, sinks)
        # each is within 2^-8 (mag + |out|) of the same value; mag <= max |v|
        assert (got[0].float() - out[-1].float()).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -10) * logical[0].abs().max()
        sel = torch.full((1, 1024), -1, dtype=torch.int32, device="cuda")
        pos = torch.tensor(oracle.window_positions(L, window, sinks), dtype=torch.int32, device="cuda")
        sel[0, :len(pos)] = pos
        ctx = torch.tensor([L], dtype=torch.int32, device="cuda")
        clean = torch.nan_to_num(latent)
        ws = torch.empty(dsa.dsa_workspace_size(dsa.DSA_MODE_DECODE, 1, 0, L, 128, 1024), dtype=torch.uint8, device="cuda")
        sparse = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda")
        dsa.dsa_sparse_mla_decode(q[-1:].contiguous(), dsa.paged_desc(clean, table, ctx, L), sel, 1, 128, 1024, SM, sparse, None, ws)
        assert (got.float() - sparse.float()).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -10) * logical[0].abs().max()


def test_nan_and_infinity_outside_the_window_are_not_seen_and_inside_are():
    L, H, window, sinks = 400, 128, 50, 3
    q, latent = rnd((L, H, 576), 1, 2.0), rnd((L, 576), 2)
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")

    def go(lat):
        out, lse = torch.empty((L, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((L, H), device="cuda")
        dsa.dsa_window_mla_prefill(q, dsa.contiguous_desc(lat, cu, L), 1, H, window, sinks, SM, out, lse)
        return out, lse

    clean, clean_lse = go(latent)
    bad = latent.clone()
    bad[100], bad[101, 600 - 25:] = float("nan"), float("inf")
    out, lse = go(bad)
    unseen = [t for t in range(L) if t < 100 or t - window >= 101]
    assert torch.equal(out[unseen], clean[unseen]) and torch.equal(lse[unseen], clean_lse[unseen])
    assert out[100:150].isnan().all() and lse[100:150].isnan().all()
    # decode: seen by one split of several, the NaN reaches the merged result
    pool, table, _ = paged_cache([3000])
    q1 = q[:1].contiguous()
    ref, _ = decode_call(q1, pool, table, [3000], 2000, 4)
    hit = pool.clone()
    hit[table[0, 5], 0] = float("nan")      # position 320: outside
    out, lse = decode_call(q1, hit, table, [3000], 2000, 4)
    assert torch.equal(out, ref)
    hit[table[0, 40], 3] = float("nan")     # position 2563: inside
    out, lse = decode_call(q1, hit, table, [3000], 2000, 4)
    assert out.isnan().all() and lse.isnan().all()


def test_large_logits_rescale():
    # logits grow along the sequence, so the running maximum moves in every chunk
    L, H = 600, 128
    latent = rnd((L, 576), 3)
    latent[:, 512] = (torch.arange(L, device="cuda") * 0.25).bfloat16()
    q = rnd((L, H, 576), 4)
    q[:, :, 512] = 24.0
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    out, lse = torch.empty((L, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((L, H), device="cuda")
    dsa.dsa_window_mla_prefill(q, dsa.contiguous_desc(latent, cu, L), 1, H, 400, 2, SM, out, lse)
    for t in (0, 63, 64, 399, 400, 599):
        want, wlse = oracle.window_mla_token(f64(q[t]), f64(latent), t + 1, 400, 2, SM)
        # logits reach 150: their fp32 sums of 576 terms are within 576 * 2^-24 * (24 * 150 + 600) / 24 = 2^-7.4
        assert np.abs(f64(lse[t]) - wlse).max() <= 2.0 ** -7 and np.abs(f64(out[t]) - want).max() <= 2.0 ** -5 * 5


def test_pages_outside_the_pool_and_contexts_beyond_the_declared():
    ctx = [500, 1000, 2500]
    latent, table, logical = paged_cache(ctx)
    q = rnd((3, 128, 576), 5, 2.0)
    ref, ref_lse = decode_call(q, latent, table, ctx, 600, 4)
    bad = table.clone()
    bad[1, 10] = latent.shape[0]        # positions 640..703, inside sequence 1's window
    bad[2, 0] = -7                      # the sinks' page of sequence 2
    bad[0, -1], bad[2, 5] = -9, 10 ** 6  # never read: outside the context, outside the window
    out, lse = decode_call(q, latent, bad, ctx, 600, 4)
    assert dsa.dsa_device_error() == dsa.DSA_ERR_DEVICE_CHECK
    assert torch.equal(out[0], ref[0]) and torch.equal(lse[0], ref_lse[0])
    for b, gone in ((1, set(range(640, 704))), (2, set(range(4)))):
        keep = [s for s in oracle.window_positions(ctx[b], 600, 4) if s not in gone]
        want, wlse = oracle.sparse_mla_token(f64(q[b]), f64(logical[b]), keep, SM)
        assert np.abs(f64(lse[b]) - wlse).max() <= 2.0 ** -10
        assert np.abs(f64(out[b]) - want).max() <= (2.0 ** -7 + 2.0 ** -10) * f64(logical[b]).__abs__().max()
    # a context longer than max_seqlen is clamped, a negative one is empty; both are reported
    for c, eff in (([500, 1000, 2500], [500, 1000, 2000]), ([-3, 1000, 2000], [0, 1000, 2000])):
        out, lse = decode_call(q, latent, table, c, 600, 4, max_ctx=2000)
        assert dsa.dsa_device_error() == dsa.DSA_ERR_DEVICE_CHECK
        for b in range(3):
            check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), eff[b], 600, 4, (c, b))


def test_pages_past_2_31_elements_of_a_pool():
    pages = 60000
    latent = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    rows = rnd((130, 576), 1)
    table = torch.tensor([[3, pages - 1, 58300]], dtype=torch.int32, device="cuda")
    latent[3], latent[pages - 1], latent[58300, :2] = rows[:64], rows[64:128], rows[128:]
    q = rnd((1, 128, 576), 2, 2.0)
    out, lse = decode_call(q, latent, table, [130], 100, 2)
    assert dsa.dsa_device_error() == 0
    check_row(f64(out[0]), f64(lse[0]), f64(q[0]), f64(rows), 130, 100, 2, "far pages")


def test_two_streams_with_their_own_workspaces_and_a_captured_graph():
    ctx = [3000, 2000]
    latent, table, logical = paged_cache(ctx)
    qs = [rnd((2, 128, 576), s, 2.0) for s in (1, 2)]
    want = [decode_call(q, latent, table, ctx, 1500, 4) for q in qs]
    n = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    desc = dsa.paged_desc(latent, table, n, 3000)
    size = dsa.dsa_window_mla_workspace_size(2, 128, 1500, 4, 3000)
    assert size > 0  # split
    out = [torch.empty((2, 128, 512), dtype=torch.bfloat16, device="cuda") for _ in qs]
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, w, s in zip(qs, out, ws, streams):
            dsa.dsa_window_mla_decode(q, desc, 2, 128, 1500, 4, SM, o, None, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r[0]) for o, r in zip(out, want))
    # a captured step reads the contexts of the moment it is replayed
    g = torch.cuda.CUDAGraph()
    lse = torch.empty((2, 128), device="cuda")
    with torch.cuda.graph(g):
        dsa.dsa_window_mla_decode(qs[0], desc, 2, 128, 1500, 4, SM, out[0], lse, ws[0])
    for now in ([3000, 2000], [1, 0], [130, 1999]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        for b, c in enumerate(now):
            check_row(f64(out[0][b]), f64(lse[b]), f64(qs[0][b]), f64(logical[b]), c, 1500, 4, (now, b))
    assert dsa.dsa_device_error() == 0


def test_vanishing_scale_gives_the_mean():
    latent, table, logical = paged_cache([100])
    q = rnd((1, 128, 576), 5)
    out, lse = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 128), device="cuda")
    n = torch.tensor([100], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, dsa.dsa_window_mla_workspace_size(1, 128, 10, 2, 100)), dtype=torch.uint8, device="cuda")
    dsa.dsa_window_mla_decode(q, dsa.paged_desc(latent, table, n, 100), 1, 128, 10, 2, 2.0 ** -60, out, lse, ws)
    rows = f64(logical[0])[list(range(2)) + list(range(90, 100))]
    assert np.abs(f64(out[0]) - rows[:, :512].mean(0)).max() <= 2.0 ** -7 * np.abs(rows).max()
    assert np.abs(f64(lse) - math.log(12)).max() <= 2.0 ** -20


def test_wrapper_refusals():
    latent, table, _ = paged_cache([100])
    n = torch.tensor([100], dtype=torch.int32, device="cuda")
    desc = dsa.paged_desc(latent, table, n, 100)
    q, out = rnd((1, 128, 576), 5), torch.zeros((1, 128, 512), dtype=torch.bfloat16, device="cuda")
    for a in ((q.float(), desc, 1, 128, out), (q[:, :64], desc, 1, 128, out), (q, desc, 2, 128, out), (q, desc, 1, 64, out),
              (q, desc, 1, 128, out[:, :, :256]), (q.cpu(), desc, 1, 128, out), (q.repeat(2, 1, 1), desc, 1, 128, out.repeat(2, 1, 1))):
        with pytest.raises(ValueError):
            dsa.dsa_window_mla_decode(*a[:4], 10, 0, SM, a[4])
    with pytest.raises(dsa.DSAError):
        dsa.dsa_window_mla_decode(q, desc, 1, 128, 100, 0, 0.0, out)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_window_mla_prefill(q, desc, 1, 128, 10, 0, SM, out)  # paged
    for window, sinks, scale, kind in ((2 ** 31, 0, SM, ValueError), (10, -2 ** 40, SM, ValueError), (4.5, 0, SM, TypeError),
                                       (10, 0, "a", TypeError)):
        with pytest.raises(kind):
            dsa.dsa_window_mla_decode(q, desc, 1, 128, window, sinks, scale, out)
    flat = dsa.contiguous_desc(latent.flatten(0, 1), torch.tensor([0, 64], dtype=torch.int32, device="cuda"), 64)
    with pytest.raises(ValueError):
        dsa.dsa_window_mla_prefill(q, flat, 1, 128, 10, 0, SM, out)  # as many queries as tokens
    assert (out == 0).all()


@pytest.mark.parametrize("sinks", [0, 3, 64])
def test_decode_of_every_last_chunk(sinks):
    """Key counts on either side of the halves and the wholes of a chunk, whole sequences and shared out."""
    counts = [n + d for n in (64, 128, 192, 256) for d in (-1, 0, 1)] + [31, 32, 33]
    ctx = counts + [c + 1000 for c in counts]
    latent, table, logical = paged_cache(ctx)
    table = torch.nn.functional.pad(table, (0, 141 - table.shape[1]), value=-1).contiguous()
    q = rnd((len(ctx), 16, 576), 5, 2.0)
    for window, shared in [(1 << 20, True)] + [(c, False) for c in (32, 63, 64, 65, 127, 128, 129, 191, 193, 256)]:
        assert (dsa.dsa_window_mla_workspace_size(len(ctx), 16, window, sinks, 9000) > 0) == shared
        out, lse = decode_call(q, latent, table, ctx, window, sinks, H=16, max_ctx=9000)
        assert dsa.dsa_device_error() == 0
        for b, c in enumerate(ctx):
            check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), c, window, sinks, (window, b))


def test_two_captured_graphs_in_turn_over_one_workspace():
    """Replayed one after the other, with the contexts changed between them; each replay plans and merges anew."""
    H, window = 16, 1 << 20
    latent, table, logical = paged_cache([3000, 900, 2000])
    qs = [rnd((3, H, 576), s, 2.0) for s in (5, 6)]
    ctx = torch.tensor([3000, 900, 2000], dtype=torch.int32, device="cuda")
    desc = dsa.paged_desc(latent, table, ctx, 3000)
    ws = torch.full((dsa.dsa_window_mla_workspace_size(3, H, window, 0, 3000),), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    outs, lses, graphs = [torch.empty(3, H, 512, dtype=torch.bfloat16, device="cuda") for _ in qs], [torch.empty(3, H, device="cuda") for _ in qs], []
    for q, out, lse in zip(qs, outs, lses):
        dsa.dsa_window_mla_decode(q, desc, 3, H, window, 0, SM, out, lse, ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            dsa.dsa_window_mla_decode(q, desc, 3, H, window, 0, SM, out, lse, ws)
    for lens in ([3000, 900, 2000], [64, 1, 1999], [0, 900, 129]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for q, out, lse in zip(qs, outs, lses):
            for b, c in enumerate(lens):
                check_row(f64(out[b]), f64(lse[b]), f64(q[b]), f64(logical[b]), c, window, 0, (lens, b))
    assert dsa.dsa_device_error() == 0
