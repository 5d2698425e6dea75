"""dsa_rope against the float64 oracle.

Tolerance, from the arithmetic: the fraction of a turn is rounded to fp32 once (at most 2^-26 turns, 2^-23.3
rad) and, for 16-bit tensors, once more in radians (2^-23.3); the sine is good to about 2 units in the last place
(2^-23, fp32 tensors) or 2^-21.2 absolute (16-bit ones), and two products and a sum round three times: together
under 2^-20 of mscale (|a| + |b|) on each rotated element, beside half a unit of the output type."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rnd(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def check(x, pos, freqs, out, off, rot, layout, m=1.0, transpose=False):
    x64, half = x.double().cpu().numpy(), layout == dsa.DSA_ROPE_HALF
    want = oracle.rope(x64, pos.cpu().numpy(), freqs.cpu().numpy(), off, rot, half, m, transpose)
    mag = np.abs(x64)
    part = mag[:, :, off:off + rot]
    both = part[:, :, :rot // 2] + part[:, :, rot // 2:] if half else part[:, :, 0::2] + part[:, :, 1::2]
    tol = np.zeros_like(mag)
    tol[:, :, off:off + rot] = abs(m) * 2.0 ** -20 * (np.concatenate([both, both], 2) if half else np.repeat(both, 2, axis=2))
    err = np.abs(out.double().cpu().numpy() - want)
    rounding = np.abs(want) * torch.finfo(x.dtype).eps / 2 * (1 + 2.0 ** -10) + TINY[x.dtype]
    rounding[:, :, :off] = 0
    rounding[:, :, off + rot:] = 0  # copied dims keep their bits
    bad = np.argwhere(~(err <= tol + rounding))
    assert bad.size == 0, f"{len(bad)} off, first at {bad[0]}: {err[tuple(bad[0])]}"


def run(rows, heads, dim, off, rot, layout, dtype, m=1.0, transpose=False, span=131072, seed=1):
    x = rnd((rows, heads, dim), dtype, seed)
    pos = torch.randint(0, span, (rows,), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.int32)
    freqs = dsa.dsa_rope_frequencies(rot, 10000.0)[0].cuda()
    out = torch.full_like(x, float("nan"))
    dsa.dsa_rope(x, pos, freqs, out, off, rot, layout, m, transpose)
    check(x, pos, freqs, out, off, rot, layout, m, transpose)
    same = x.clone()
    dsa.dsa_rope(same, pos, freqs, same, off, rot, layout, m, transpose)
    assert torch.equal(same, out), "in place"


@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,heads,dim,off,rot", [
    (1, 1, 2, 0, 2), (1, 1, 64, 0, 64), (3, 128, 576, 512, 64), (5, 64, 128, 0, 64), (7, 1, 576, 512, 64), (300, 1, 64, 0, 64),
    (4, 5, 100, 36, 64), (4, 3, 72, 8, 48), (6, 2, 24, 8, 8), (2, 7, 33, 5, 6), (1000, 2, 16, 0, 16), (2, 1, 1100, 40, 1024),
    (3, 300, 1024, 0, 1024), (513, 4, 128, 64, 64), (9, 5, 100, 4, 32), (9, 3, 100, 0, 6), (9, 64, 128, 122, 6), (9, 64, 128, 3, 2),
    (700, 3, 52, 10, 20), (9, 2, 64, 3, 50), (5, 2, 2048, 1000, 24), (3, 1, 5000, 4, 1000)])
def test_rope(layout, dtype, rows, heads, dim, off, rot):
    run(rows, heads, dim, off, rot, layout, dtype, m=1.25, transpose=rows % 2 == 0)


def test_far_and_negative_positions():
    # at |position| ~ 2^24 the fp64 angle (~1.7e7 rad) is off by 2^-53 of it, far below the bound
    for layout in (dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF):
        x = rnd((6, 2, 64), torch.float32, 1)
        pos = torch.tensor([0, -1, 1 << 24, -(1 << 24) + 3, 999999, 12345678], dtype=torch.int32, device="cuda")
        freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
        out = torch.empty_like(x)
        dsa.dsa_rope(x, pos, freqs, out, 0, 64, layout)
        check(x, pos, freqs, out, 0, 64, layout)


def test_transpose_is_the_gradient_and_the_inverse():
    x, y = rnd((50, 8, 128), torch.float32, 1), rnd((50, 8, 128), torch.float32, 2)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    freqs, m = dsa.dsa_rope_frequencies(64, 10000.0, dsa.DSA_ROPE_YARN, 40.0, 4096.0)
    freqs = freqs.cuda()
    a, b, c = (torch.empty_like(x) for _ in range(3))
    dsa.dsa_rope(x, pos, freqs, a, 0, 64, dsa.DSA_ROPE_HALF, m)
    dsa.dsa_rope(y, pos, freqs, b, 0, 64, dsa.DSA_ROPE_HALF, m, transpose=True)
    # <R x, y> = <x, R^T y>: each of the 51200 products is off by at most 2^-19 of its magnitude
    left, right = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
    assert abs(left - right) <= 2.0 ** -18 * m * (x.double().abs() * y.double().abs()).sum() * 2
    dsa.dsa_rope(a, pos, freqs, c, 0, 64, dsa.DSA_ROPE_HALF, 1 / m, transpose=True)
    assert (c - x).abs().max() <= 2.0 ** -18 * 2 * x.abs().max()


@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF])
def test_strided_heads_and_rows(layout):
    base = rnd((20, 6, 200), torch.bfloat16, 3)
    freqs = dsa.dsa_rope_frequencies(32, 10000.0)[0].cuda()
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    for lo in (0, 8, 5):  # aligned, aligned, misaligned
        x = base[:, 1:5, lo:lo + 64]
        want = torch.empty((20, 4, 64), dtype=torch.bfloat16, device="cuda")
        dsa.dsa_rope(x.contiguous(), pos, freqs, want, 16, 32, layout)
        room = torch.full((20, 9, 80), 3.0, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_rope(x, pos, freqs, room[:, 2:6, :64], 16, 32, layout)
        assert torch.equal(room[:, 2:6, :64], want)
        room[:, 2:6, :64] = 3
        assert (room == 3).all()
        inside = base.clone()
        dsa.dsa_rope(inside[:, 1:5, lo:lo + 64], pos, freqs, inside[:, 1:5, lo:lo + 64], 16, 32, layout)
        assert torch.equal(inside[:, 1:5, lo:lo + 64], want)
        inside[:, 1:5, lo:lo + 64] = base[:, 1:5, lo:lo + 64]
        assert torch.equal(inside, base)
    # a sequence-major view: heads outside rows
    x = rnd((4, 20, 64), torch.bfloat16, 4).transpose(0, 1)
    out = torch.empty_like(x)
    dsa.dsa_rope(x, pos, freqs, out, 32, 32, layout)
    check(x, pos, freqs, out, 32, 32, layout)


@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_INTERLEAVED, dsa.DSA_ROPE_HALF])
def test_one_head_given_to_many(layout):
    x = rnd((20, 1, 64), torch.bfloat16, 3).expand(20, 16, 64)
    freqs, pos = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda(), torch.arange(20, dtype=torch.int32, device="cuda")
    out, want = (torch.empty((20, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dsa.dsa_rope(x, pos, freqs, out, 0, 64, layout)
    dsa.dsa_rope(x.contiguous(), pos, freqs, want, 0, 64, layout)
    assert torch.equal(out, want)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope(x, pos, freqs, x, 0, 64, layout)  # in place on repeated heads


def test_nothing_to_do():
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    for shape in ((0, 4, 64), (4, 0, 64)):
        x = torch.empty(shape, device="cuda")
        dsa.dsa_rope(x, torch.zeros(shape[0], dtype=torch.int32, device="cuda"), freqs, torch.empty_like(x), 0, 64)


def test_nan_and_infinity_stay_in_their_pair():
    x = rnd((1, 2, 64), torch.float32, 1)
    x[0, 0, 3], x[0, 1, 40] = float("nan"), float("inf")
    clean = rnd((1, 2, 64), torch.float32, 1)
    freqs, pos = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda(), torch.tensor([7], dtype=torch.int32, device="cuda")
    out, ref = torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rope(x, pos, freqs, out, 0, 64)
    dsa.dsa_rope(clean, pos, freqs, ref, 0, 64)
    same = torch.ones_like(x, dtype=torch.bool)
    same[0, 0, 2:4] = False
    same[0, 1, 40:42] = False
    assert torch.equal(out[same], ref[same]) and out[0, 0, 2:4].isnan().all() and not out[0, 1, 40:42].isfinite().any()


def test_more_than_2_31_elements():
    rows, heads, dim = 30000, 128, 576  # 2.2e9 elements
    x = torch.zeros((rows, heads, dim), dtype=torch.bfloat16, device="cuda")
    probe = [0, 14563, 29126, rows - 1]  # 29127 * 128 * 576 passes 2^31
    x[probe] = rnd((4, heads, dim), torch.bfloat16, 1)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    out = torch.full_like(x, 1.0)
    dsa.dsa_rope(x, pos, freqs, out, 512, 64)
    check(x[probe], pos[probe], freqs, out[probe], 512, 64, dsa.DSA_ROPE_INTERLEAVED)
    assert (out[29127:29999] == 0).all() and (out[1:1000] == 0).all()


def test_another_stream_and_a_captured_graph():
    x, pos = rnd((33, 64, 128), torch.bfloat16, 1), torch.arange(33, dtype=torch.int32, device="cuda")
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    want, got, cap = (torch.empty_like(x) for _ in range(3))
    dsa.dsa_rope(x, pos, freqs, want, 0, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.dsa_rope(x, pos, freqs, got, 0, 64, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_rope(x, pos, freqs, cap, 0, 64)
    pos += 5
    g.replay()  # reads the positions of the moment
    check(x, pos, freqs, cap, 0, 64, dsa.DSA_ROPE_INTERLEAVED)


def test_wrapper_refusals():
    x, pos = torch.zeros((4, 2, 64), device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    freqs = torch.zeros(32, dtype=torch.float64, device="cuda")
    for args in ((x, pos.long(), freqs, x), (x, pos[:3], freqs, x), (x, pos, freqs.float(), x), (x, pos, freqs[:16], x),
                 (x, pos, freqs, x.half()), (x, pos, freqs, x[:, :1]), (x[0], pos, freqs, x[0]), (x, pos.cpu(), freqs, x),
                 (x.transpose(1, 2), pos, freqs, x)):
        with pytest.raises(ValueError):
            dsa.dsa_rope(*args, 0, 64)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope(x, pos, freqs, x, 2, 64)                       # past the head
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope(x, pos, freqs, x[:, :1].expand(4, 2, 64), 0, 64)  # heads of out on one another
