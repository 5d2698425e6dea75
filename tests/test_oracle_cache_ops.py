"""Pins of the oracle's operators around the caches: closed forms, a library's float64 routines and
finite differences."""
import numpy as np
import pytest
import torch

import oracle


def test_rmsnorm_and_its_gradient_against_the_library_in_64_bits():
    rs = np.random.default_rng(1)
    x, res, dy, dres = rs.standard_normal((4, 7, 33))
    w = 1 + 0.1 * rs.standard_normal(33)
    h = torch.tensor(x + res, requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    ref = torch.nn.functional.rms_norm(h, (33,), wt, 1e-5)
    y, hh, rstd = oracle.rmsnorm(x, w, 1e-5, res)
    assert np.allclose(y, ref.detach().numpy(), rtol=1e-12, atol=1e-14) and np.array_equal(hh, x + res)
    (ref * torch.tensor(dy)).sum().backward()
    dh, dw = oracle.rmsnorm_backward(dy, hh, w, rstd, dres)
    assert np.allclose(dh - dres, h.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_rmsnorm_gradient_against_differences():
    rs = np.random.default_rng(2)
    h, dy = rs.standard_normal((2, 3, 9))
    w = rs.standard_normal(9)
    f = lambda a, b: (oracle.rmsnorm(a, b, 1e-3)[0] * dy).sum()  # noqa: E731
    dh, dw = oracle.rmsnorm_backward(dy, h, w, oracle.rmsnorm(h, w, 1e-3)[2])
    e = 1e-6
    for r in range(3):
        for c in range(9):
            d = np.zeros_like(h)
            d[r, c] = e
            assert abs((f(h + d, w) - f(h - d, w)) / (2 * e) - dh[r, c]) < 1e-7
    for c in range(9):
        d = np.zeros(9)
        d[c] = e
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * e) - dw[c]) < 1e-7


def test_row_scales_of_rows_and_groups():
    v = np.zeros((2, 300))
    v[0, 0], v[0, 130], v[0, 299] = -448.0, 44.8, 4.48
    assert oracle.row_scales(v).tolist() == [1.0, 1.0]  # amax 448 -> 1; an all-zero row -> 1
    assert np.allclose(oracle.row_scales(v, 128), [[1.0, 0.1, 0.01], [1.0, 1.0, 1.0]])


@pytest.mark.parametrize("half", [False, True])
def test_rope_is_a_product_of_complex_numbers(half):
    rs = np.random.default_rng(3)
    x = rs.standard_normal((5, 2, 20))
    pos = np.array([0, 1, 77, 100000, -5])
    freqs, _ = oracle.rope_frequencies(12, 10000.0)
    got = oracle.rope(x, pos, freqs, 4, 12, half, mscale=1.5)
    part = x[:, :, 4:16]
    z = part[:, :, :6] + 1j * part[:, :, 6:] if half else part[:, :, 0::2] + 1j * part[:, :, 1::2]
    z = 1.5 * z * np.exp(1j * pos[:, None, None] * freqs)
    want = x.copy()
    if half:
        want[:, :, 4:10], want[:, :, 10:16] = z.real, z.imag
    else:
        want[:, :, 4:16:2], want[:, :, 5:16:2] = z.real, z.imag
    assert np.allclose(got, want, rtol=0, atol=1e-9)
    # the transpose undoes the turn (and is the gradient: <R x, y> = <x, R^T y>)
    assert np.allclose(oracle.rope(got, pos, freqs, 4, 12, half, mscale=1 / 1.5, transpose=True), x, atol=1e-12)
    y = rs.standard_normal(x.shape)
    assert np.isclose((got * y).sum(), (x * oracle.rope(y, pos, freqs, 4, 12, half, 1.5, True)).sum()
                      + (got * y - x * y)[:, :, :4].sum() + (got * y - x * y)[:, :, 16:].sum())


def test_rope_products_depend_on_the_distance_alone():
    rs = np.random.default_rng(4)
    q, k = rs.standard_normal((2, 1, 1, 64))
    freqs, _ = oracle.rope_frequencies(64, 10000.0)
    dots = [(oracle.rope(q, [a + 13], freqs, 0, 64, False) * oracle.rope(k, [a], freqs, 0, 64, False)).sum() for a in (0, 5, 900)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_scaled_frequencies():
    plain, m = oracle.rope_frequencies(64, 10000.0)
    assert m == 1.0 and plain[0] == 1.0 and np.isclose(plain[16], 10000.0 ** -0.5)
    assert np.allclose(oracle.rope_frequencies(64, 10000.0, "linear", 8.0)[0], plain / 8)
    ntk = oracle.rope_frequencies(64, 10000.0, "ntk", 8.0)[0]
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], plain[-1] / 8)  # the slowest pair is scaled in full
    yarn, m = oracle.rope_frequencies(64, 10000.0, "yarn", 40.0, 4096.0)
    assert np.isclose(m, 0.1 * np.log(40) + 1)
    turns = 4096 * plain / (2 * np.pi)
    assert np.allclose(yarn[turns > 64], plain[turns > 64]) and np.allclose(yarn[turns < 0.5], plain[turns < 0.5] / 40)
    assert (yarn <= plain * (1 + 1e-12)).all() and (yarn >= plain / 40 * (1 - 1e-12)).all()


def test_cache_rows_are_the_norm_and_the_turn():
    rs = np.random.default_rng(5)
    kv, key = rs.standard_normal((3, 576)), rs.standard_normal((3, 128))
    w, pos = rs.standard_normal(512), [0, 9, 300]
    freqs, _ = oracle.rope_frequencies(64, 10000.0)
    lat, k = oracle.cache_rows(kv, w, 1e-6, key, pos, freqs, False, True, 0)
    assert np.allclose(lat[:, :512], oracle.rmsnorm(kv[:, :512], w, 1e-6)[0])
    assert np.allclose(lat[0, 512:], kv[0, 512:]) and np.allclose(k[0], key[0])       # position 0
    assert np.allclose(np.linalg.norm(lat[:, 512:], axis=1), np.linalg.norm(kv[:, 512:], axis=1))
    assert np.array_equal(k[:, 64:], key[:, 64:]) and not np.allclose(k[1, :64], key[1, :64])


@pytest.mark.parametrize("length,window,sinks", [(1, 1, 0), (9, 3, 2), (9, 9, 0), (9, 100, 4), (9, 1, 100), (0, 4, 2)])
def test_window_attention_against_the_library_under_a_mask(length, window, sinks):
    rs = np.random.default_rng(6)
    lat = rs.standard_normal((max(length, 1), 576))
    q = rs.standard_normal((3, 576))
    out, lse = oracle.window_mla_token(q, lat, length, window, sinks, 0.05)
    if length == 0:
        assert (out == 0).all() and np.isneginf(lse).all()
        return
    pos = torch.arange(length)
    mask = (pos > length - 1 - window) | (pos < sinks)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q)[:, None], torch.tensor(lat).expand(3, -1, -1), torch.tensor(lat[:, :512]).expand(3, -1, -1),
        attn_mask=mask[None, None], scale=0.05)
    assert np.allclose(out, ref[:, 0].numpy(), atol=1e-12)
    logits = 0.05 * q @ lat[mask.numpy()].T
    assert np.allclose(lse, np.log(np.exp(logits).sum(1)))


def test_row_scales_stop_at_the_smallest_fp32():
    v = np.zeros((2, 130))
    v[0, 0], v[0, 129], v[1, 0] = 448.0, 1.3e-43, 1e-40
    assert oracle.row_scales(v).tolist() == [1.0, 1e-40 / 448]
    assert oracle.row_scales(v, 128).tolist() == [[1.0, 2.0 ** -149], [1e-40 / 448, 1.0]]
