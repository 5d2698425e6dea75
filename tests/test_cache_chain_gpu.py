"""The operators around the caches used together, as a serving loop uses them: a hidden state is normed, projected, its
queries rotated, its latent and indexer key appended to the paged caches; then one attention runs over the selection of
the indexer and one over a window with sinks.  Each step's output is checked against the oracle run on what the caches hold,
and the caches against the oracle of what was appended."""
import math

import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(576)
HID, H, H_I, D_I, K, WINDOW, SINKS = 1024, 128, 64, 128, 64, 100, 4


def rnd(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std).bfloat16()


def test_prompt_then_decode_steps():
    lens = [150, 1, 70]
    B, T = len(lens), sum(lens)
    pages = 4
    table = torch.randperm(B * pages + 3, generator=torch.Generator().manual_seed(1))[:B * pages].reshape(B, pages).int().cuda()
    latent = torch.full((B * pages + 3, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((B * pages + 3, 64, D_I), 0x7F, dtype=torch.uint8, device="cuda")
    scale = torch.full((B * pages + 3, 64), float("nan"), device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lat_desc = dsa.paged_desc(latent, table, ctx, pages * 64)
    key_desc = dsa.paged_desc(codes, table, ctx, pages * 64, scale=scale)
    w_in, w_kv = 1 + 0.1 * rnd((HID,), 2), 1 + 0.1 * rnd((512,), 3)
    p_kv, p_key, p_q, p_qi = (rnd((HID, n), 4 + i, HID ** -0.5) for i, n in enumerate((576, D_I, H * 576, H_I * D_I)))
    freqs, m = dsa.dsa_rope_frequencies(64, 10000.0, dsa.DSA_ROPE_YARN, 8.0, 64.0)
    freqs = freqs.cuda()
    w = rnd((B, H_I), 9).float()
    logical = [[] for _ in range(B)]  # what the oracle says each sequence's caches hold

    def layer_in(x, res):
        y, total = torch.empty_like(x), torch.empty_like(x)
        dsa.dsa_rmsnorm(x, w_in, 1e-6, y=y, residual=res, residual_out=total)
        v, h, _ = oracle.rmsnorm(x.double().cpu().numpy(), w_in.double().cpu().numpy(), 1e-6, res.double().cpu().numpy())
        assert np.all(np.abs(y.double().cpu().numpy() - v) <= np.abs(v) * (2.0 ** -8 + 2.0 ** -15))
        return y

    def append(y, seq, pos):
        kv, key = y @ p_kv, y @ p_key
        dsa.dsa_cache_append(kv, w_kv, 1e-6, key, seq, pos, freqs, lat_desc, key_desc, dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF, 0, m)
        rows, _ = oracle.cache_rows(kv.double().cpu().numpy(), w_kv.double().cpu().numpy(), 1e-6, key.double().cpu().numpy(),
                                    pos.cpu().numpy(), freqs.cpu().numpy(), False, True, 0, m)
        for r, (b, t) in enumerate(zip(seq.tolist(), pos.tolist())):
            assert t == len(logical[b])
            logical[b].append(rows[r])

    seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(lens)]).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    append(layer_in(rnd((T, HID), 20), rnd((T, HID), 21)), seq, pos)
    ws_s = torch.empty(dsa.dsa_workspace_size(dsa.DSA_MODE_DECODE, B, 0, pages * 64, H, K), dtype=torch.uint8, device="cuda")
    ws_w = torch.empty(max(1, dsa.dsa_window_mla_workspace_size(B, H, WINDOW, SINKS, pages * 64)), dtype=torch.uint8, device="cuda")
    every = torch.arange(B, dtype=torch.int32, device="cuda")
    for step in range(4):
        y = layer_in(rnd((B, HID), 30 + step), rnd((B, HID), 40 + step))
        append(y, every, ctx.clone())
        ctx += 1
        at = ctx - 1
        q = (y @ p_q).view(B, H, 576)
        dsa.dsa_rope(q, at, freqs, q, 512, 64, dsa.DSA_ROPE_INTERLEAVED, m)
        qi = (y @ p_qi).view(B, H_I, D_I)
        dsa.dsa_rope(qi, at, freqs, qi, 0, 64, dsa.DSA_ROPE_HALF, m)
        q8, qs = torch.empty((B, H_I, D_I), dtype=torch.uint8, device="cuda"), torch.empty(B, device="cuda")
        dsa.dsa_quantize_fp8(qi, q8, qs)
        out, idx = torch.empty((B, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((B, K), dtype=torch.int32, device="cuda")
        clean = torch.nan_to_num(latent)  # the sparse path copies a real row for its padding entries
        dsa.dsa_forward(dsa.DSA_MODE_DECODE, q8, qs, w, key_desc, q, dsa.paged_desc(clean, table, ctx, pages * 64), B, H_I, D_I, H, K, SM,
                        out, None, idx, ws_s)
        win = torch.empty_like(out)
        dsa.dsa_window_mla_decode(q, lat_desc, B, H, WINDOW, SINKS, SM, win, None, ws_w)
        assert dsa.dsa_device_error() == 0
        for b in range(B):
            n = int(ctx[b])
            rows = np.stack(logical[b])
            held = oracle.paged_gather(latent.double().cpu().numpy(), table[b].cpu().numpy(), n)
            assert np.all(np.abs(held - rows) <= np.abs(rows) * (2.0 ** -8 + 2.0 ** -15) + 2.0 ** -17 * np.abs(rows).max())
            sel = idx[b][idx[b] >= 0].cpu().numpy()
            assert len(sel) == min(K, n)
            # the selection is the top-k of the scores of the appended keys
            s = torch.empty((1, pages * 64), device="cuda")
            dsa.dsa_indexer_scores(q8, qs, w, key_desc, B, H_I, D_I, b, b + 1, s)
            assert np.array_equal(idx[b].cpu().numpy(), oracle.topk_rows(s.cpu().numpy()[:, :n], np.array([n]), K)[0])
            k8 = oracle.paged_gather(codes.cpu().numpy(), table[b].cpu().numpy(), n)
            ks = oracle.paged_gather(scale.double().cpu().numpy(), table[b].cpu().numpy(), n)
            ref = oracle.indexer_scores_query(q8[b].cpu().numpy(), float(qs[b]), w[b].double().cpu().numpy(), k8, ks)
            mag = oracle.indexer_magnitude_query(q8[b].cpu().numpy(), float(qs[b]), w[b].double().cpu().numpy(), k8, ks)
            assert np.all(np.abs(s.cpu().numpy()[0, :n] - ref) <= 1e-3 * mag + 1e-30)
            want, _ = oracle.sparse_mla_token(q[b].double().cpu().numpy(), held, sel, SM)
            assert np.linalg.norm(out[b].double().cpu().numpy() - want) <= 1e-2 * np.linalg.norm(want), (step, b)
            want, _ = oracle.window_mla_token(q[b].double().cpu().numpy(), held, n, WINDOW, SINKS, SM)
            assert np.linalg.norm(win[b].double().cpu().numpy() - want) <= 1e-2 * np.linalg.norm(want), (step, b)


def test_indexer_gradients_back_through_the_rotation_and_the_norm():
    """dq_I of the indexer's backward, through the transposed rotation and the norm of each head, against differences in 64 bits."""
    T, cols = 6, 64
    x = rnd((T * 4, cols), 1).float()
    w = 1 + 0.1 * rnd((cols,), 2).float()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 17
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    y, rstd = torch.empty_like(x), torch.empty(T * 4, device="cuda")
    dsa.dsa_rmsnorm(x, w, 1e-6, y=y, rstd=rstd)
    g = rnd((T, 4, cols), 3).float()  # the gradient of the rotated queries
    back = torch.empty_like(g)
    dsa.dsa_rope(g, pos, freqs, back, 0, 64, dsa.DSA_ROPE_HALF, transpose=True)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(T * 4, cols), dtype=torch.uint8, device="cuda")
    dsa.dsa_rmsnorm_backward(back.view(T * 4, cols), x, w, rstd, dx, dw, ws)
    x64, w64, g64 = (t.double().cpu().numpy() for t in (x, w, g))

    def loss(a, b):
        v = oracle.rmsnorm(a, b, 1e-6)[0].reshape(T, 4, cols)
        return (oracle.rope(v, pos.cpu().numpy(), freqs.cpu().numpy(), 0, 64, True) * g64).sum()

    e = 1e-5  # differences in 64 bits: 1e-10 of the third derivative, 1e-10 of the loss's own rounding
    scale = float(dx.abs().max()) + float(dw.abs().max())
    for r, c in [(0, 0), (5, 40), (23, 63)]:
        d = np.zeros_like(x64)
        d[r, c] = e
        assert abs((loss(x64 + d, w64) - loss(x64 - d, w64)) / (2 * e) - float(dx[r, c])) <= 2.0 ** -16 * scale
    for c in (0, 33, 63):
        d = np.zeros_like(w64)
        d[c] = e
        assert abs((loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * e) - float(dw[c])) <= 2.0 ** -16 * scale
