"""One workspace for calls of several sizes, as a program keeps it for its largest."""
import pytest
import torch

import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu


def rnd(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def test_norm_backward_of_narrower_layers_and_shorter_batches():
    rows = 2400  # more than the most CTAs of any width
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(rows, 5120), dtype=torch.uint8, device="cuda")
    for n, cols in ((rows, 5120), (rows, 4096), (rows, 2048), (rows, 500), (rows, 8), (100, 4096)):
        dy, h, w = rnd((n, cols), 1), rnd((n, cols), 2), rnd((cols,), 3)
        rstd = h.float().square().mean(1).rsqrt()
        got = []
        for space in (ws, torch.empty(1 << 24, dtype=torch.uint8, device="cuda")):
            dh, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
            dsa.dsa_rmsnorm_backward(dy, h, w, rstd, dh, dw, space.fill_(0xFF))
            got.append((dh, dw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[0][1].isfinite().all()


def test_window_decode_of_a_batch_that_shrinks():
    """A workspace for 64 sequences, for which one call needs none, serves 40 and 1; every row is the one that a call with its
    own workspace gives."""
    B, H, pages, window, sinks = 64, 16, 32, 1500, 4
    latent, q = rnd((B * pages, 64, 576), 1), rnd((B, H, 576), 2)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(3)).int().view(B, pages).cuda()
    ctx = torch.randint(1, pages * 64 + 1, (B,), generator=torch.Generator().manual_seed(4)).int().cuda()
    ws = torch.full((dsa.dsa_window_mla_workspace_limit(B, H, window, sinks, pages * 64),), 0xFF, dtype=torch.uint8, device="cuda")
    assert dsa.dsa_window_mla_workspace_size(B, H, window, sinks, pages * 64) == 0
    for n in (64, 40, 1, 12, 64):
        lat = dsa.paged_desc(latent, table[:n], ctx[:n], pages * 64)
        got = []
        size = dsa.dsa_window_mla_workspace_size(n, H, window, sinks, pages * 64)
        for space in (ws, torch.empty(size, dtype=torch.uint8, device="cuda") if size else None):
            out, lse = torch.empty((n, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((n, H), device="cuda")
            dsa.dsa_window_mla_decode(q[:n], lat, n, H, window, sinks, 0.04, out, lse, space)
            got.append((out, lse))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[0][1].isfinite().all(), n
    assert dsa.dsa_device_error() == 0
