"""e4m3 codes of values so small that amax / 448 lies below the smallest fp32 (2^-149): the scale is
then 2^-149, the codes are finite and zeros encode as 0.

Amounts: amax is kept below 448 * 2^-150, where the quotient rounds to zero.  A value is a product or two rounded
to a multiple of 2^-149 (half of it each, 2^-149 together), its code half an e4m3 step (2^-4 of the value, 2^-10 of the
scale below the normal range); the quotient by 2^-149 is exact and at most 224, so nothing saturates."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
LEAST = 2.0 ** -149


def check(codes, scale, v):
    """codes and scale of one group whose values are v (float64)."""
    codes = codes.cpu().numpy()
    assert float(scale) == LEAST
    assert not np.isnan(oracle.decode_e4m3(codes)).any()
    assert (codes[v == 0] & 0x7F == 0).all()
    err = np.abs(oracle.decode_e4m3(codes) * LEAST - v)
    assert np.all(err <= np.maximum(np.abs(v) * 2.0 ** -4, LEAST * 2.0 ** -10) * (1 + 2.0 ** -10) + LEAST)


@pytest.mark.parametrize("cols", [256, 250, 1024, 2048, 1001, 4100, 33000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_group_of_zeros_and_one_subnormal(cols, dtype):
    """The first group large, the second zeros and the smallest bf16: 1.3e-43 once normalised."""
    x = torch.zeros((3, cols), dtype=dtype, device="cuda")
    x[:, :128] = 1000.0 * (cols / 256) ** 0.5  # rstd = 1.41e-3 whatever the width
    x[:, 140] = 2.0 ** -133
    w = torch.ones(cols, dtype=dtype, device="cuda")
    codes = torch.empty((3, cols), dtype=torch.uint8, device="cuda")
    scale = torch.empty((3, -(-cols // 128)), device="cuda")
    dsa.dsa_rmsnorm(x, w, 1e-6, codes=codes, scale=scale)
    v, _, _ = oracle.rmsnorm(x.double().cpu().numpy(), np.ones(cols), 1e-6)
    assert 0 < np.abs(v[:, 128:256]).max() < 448 * 2.0 ** -150
    for r in range(3):
        check(codes[r, 128:256], scale[r, 1], v[r, 128:256])
        assert (scale[r, 2:] == 1).all() and (codes[r, 256:] == 0).all()


@pytest.mark.parametrize("cols", [64, 128, 130, 512, 1001, 2048, 8192, 33000])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_rows_under_tiny_weights(cols, group):
    """fp32 weights of 16 * 2^-149 bring every value of a row below the smallest scale."""
    x = torch.randn((5, cols), generator=torch.Generator(device="cuda").manual_seed(cols), device="cuda").clamp_(-3, 3)
    x[:, ::3] = 0
    w = torch.full((cols,), 2.0 ** -145, device="cuda")
    codes = torch.empty((5, cols), dtype=torch.uint8, device="cuda")
    scale = torch.empty((5, -(-cols // 128)) if group else (5,), device="cuda")
    dsa.dsa_rmsnorm(x, w, 1e-6, codes=codes, scale=scale, y=torch.empty_like(x))
    v, _, _ = oracle.rmsnorm(x.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6)
    assert np.abs(v).max() < 448 * 2.0 ** -150
    for r in range(5):
        for g in range(scale[r].numel()):
            part = slice(128 * g, min(128 * g + 128, cols)) if group else slice(0, cols)
            check(codes[r, part], scale[r].reshape(-1)[g], v[r, part])


@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
def test_appended_keys_under_a_tiny_factor(layout):
    """All 64 dims of the key rotated with mscale 16 * 2^-149 (at position 0: only scaled)."""
    key = torch.randn((2, 64), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").clamp_(-3, 3).bfloat16()
    key[:, 5:9], key[:, 37:41] = 0, 0
    seq, pos = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    data = torch.full((2, 64, 64), 0x7F, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, 64), float("nan"), device="cuda")
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    keys = dsa.paged_desc(data, table, torch.ones(2, dtype=torch.int32, device="cuda"), 64, scale=scale)
    dsa.dsa_cache_append(None, None, 0.0, key, seq, pos, dsa.dsa_rope_frequencies(64, 1e4)[0].cuda(), None, keys,
                         key_layout=layout, mscale=2.0 ** -145)
    assert dsa.dsa_device_error() == 0
    v = key.double().cpu().numpy() * 2.0 ** -145
    for b, page in ((0, 1), (1, 0)):
        check(data[page, 0], scale[page, 0], v[b])


def test_quantiser_stays_above_the_smallest_scale():
    """Its input is bf16, so that its smallest scale is 2^-133 / 448: no quotient rounds to zero."""
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    x[1, 3], x[2, 3], x[3, :64] = 2.0 ** -133, -2.0 ** -132, 2.0 ** -133
    codes, scale = torch.empty((4, 128), dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")
    dsa.dsa_quantize_fp8(x, codes, scale)
    want, ws = oracle.quantize_fp8_rows(x.float().cpu().numpy())
    assert (scale > 0).all() and np.array_equal(scale.cpu().numpy(), ws) and np.array_equal(codes.cpu().numpy(), want)
