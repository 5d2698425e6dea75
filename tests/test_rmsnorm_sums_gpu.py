"""The sum of dw over many rows, in every form of the backward, against the float64 oracle with the bound of
the sums that run.

A form gives its rows to n CTAs (n = 148 times 16 KB / row bytes, at least 1 and at most 16, not above the rows; 592 and 8 to 32
rows at once in the forms of a part of a warp or a warp per row).  A column's chain in a CTA is rows / n fused
additions (or one for each of a CTA's rows at once, whose sums are then added: 2 steps within a warp at most and
8 warps), after the product dy h (one rounding); rmsnorm_dw_kernel adds n / 32 partial sums in a thread
and those of 32 threads in 5 steps.  With the rounding of a product by rstd where it is one of its own (general form), each term
passes through at most rows / n + 10 + n / 32 + 5 + 2 roundings of 2^-24; first order, with a quarter added for the rest."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
SIZE = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4}


def rnd(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def dw_bound(rows, cols, dtype):
    n = min(rows, 148 * min(max(16384 // (cols * SIZE[dtype]), 1), 16))
    fewest = min(n, 592) if cols <= 256 else n  # the longest chain and the longest second sum of the forms that may run
    return 1.25 * (rows / fewest + 1 + 10 + n / 32 + 1 + 5 + 2) * 2.0 ** -24


@pytest.mark.parametrize("rows,cols,dtype,dres", [
    (4000, 5120, torch.bfloat16, True),    # the ring with the residual's gradient: 28 rows to a CTA, one CTA to an SM
    (16384, 5120, torch.bfloat16, True),
    (9000, 8192, torch.bfloat16, False), (3001, 4096, torch.float32, True),
    (2500, 12288, torch.bfloat16, True), (2000, 16384, torch.float32, True),  # rows beyond the ring
    (40000, 512, torch.float16, False),    # narrow ring rows: 16 CTAs to an SM
    (60000, 64, torch.bfloat16, True), (30000, 250, torch.float32, False),    # parts of a warp, a warp
    (9000, 1001, torch.bfloat16, True), (4000, 5002, torch.float16, True), (1500, 17001, torch.bfloat16, False)])
def test_dw_over_many_rows(rows, cols, dtype, dres):
    dy, h, w = rnd((rows, cols), dtype, 1), rnd((rows, cols), dtype, 2), rnd((cols,), dtype, 3)
    res = rnd((rows, cols), dtype, 4) if dres else None
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dh, dw = torch.empty_like(dy), torch.full((cols,), float("nan"), device="cuda")
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dsa.dsa_rmsnorm_backward(dy, h, w, rstd, dh, dw, ws.fill_(0xFF), dresidual=res)
    assert dsa.dsa_device_error() == 0
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for i in range(0, rows, 1024):
        term = dy[i:i + 1024].double() * h[i:i + 1024].double() * rstd[i:i + 1024].double()[:, None]
        want += term.sum(0)
        mag += term.abs().sum(0)
    err = (dw.double() - want).abs()
    bound = dw_bound(rows, cols, dtype) * mag + 2.0 ** -24 * want.abs()
    assert (err <= bound).all(), (err / bound).max().item()
    pick = [0, 1, rows // 2, rows - 1]  # and the rows' gradients, where the oracle is quick
    args = [t[pick].double().cpu().numpy() for t in (dy, h)] + [w.double().cpu().numpy(), rstd[pick].double().cpu().numpy()]
    wanth, _ = oracle.rmsnorm_backward(*args, None if res is None else res[pick].double().cpu().numpy())
    g, r = args[0] * args[2], args[3][:, None]
    magh = r * (np.abs(g) + np.abs(args[1]) * r * r * np.abs(g * args[1]).mean(1, keepdims=True))
    magh = magh + (0 if res is None else np.abs(res[pick].double().cpu().numpy()))
    half = torch.finfo(dtype).eps / 2
    rel = 2.0 ** -18 if cols <= 16384 else 2.0 ** -17  # the bound of the norm's sums over a row
    assert np.all(np.abs(dh[pick].double().cpu().numpy() - wanth) <= np.abs(wanth) * half * (1 + 2.0 ** -10) + rel * magh + (2.0 ** -25 if dtype is torch.float16 else 0))
