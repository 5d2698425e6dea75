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
