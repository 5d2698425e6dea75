"""dsa_rmsnorm and dsa_rmsnorm_backward against the float64 oracle.

Tolerances, from the arithmetic.  One rounding to the output type is at most eps/2 of the value (plus
half the smallest subnormal step).  Before it everything is fp32: h is one addition (2^-24); the sum of
squares adds positive terms along a chain of at most 32 fused adds (wide rows) or cols / 256 (general
rows) and about 10 tree steps, so with cols <= 16384 its relative error is at most 75 * 2^-24 and that of
its square root half of it; a few more roundings make 2^-18 relative on every output.  Backward: the same
bound on the sum of the magnitudes of an element's terms; dw sums rows / 592 + 592 / 8 + 20 terms in a
chain, under 2^-16 of the sum of their magnitudes for the sizes here.  Codes: half an e4m3 step (2^-4
relative, 2^-10 of the scale below the normal range) beside the fp32 bound."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -18
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rnd(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, mag, what, rel=None):
    """|got - want| <= rounding of the type + rel * mag, element by element."""
    rel = rel or (F32 if got.shape[-1] <= 16384 else 2 * F32)
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(f64(got) - want)
    bound = np.abs(want) * half * (1 + 2.0 ** -10) + TINY[got.dtype] + rel * mag
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, f"{what}: {len(bad)} off, first {bad[0]}: {f64(got)[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def check_codes(codes, scale, v, group):
    want = oracle.row_scales(v, group)
    rel = F32 if v.shape[1] <= 16384 else 2 * F32
    assert np.all(np.abs(f64(scale) - want) <= want * (rel + 2.0 ** -24)), "scales"
    s = f64(scale)
    s = np.repeat(s, group, axis=1)[:, :v.shape[1]] if group else s[:, None]
    got = oracle.decode_e4m3(codes.cpu().numpy()) * s
    bound = np.maximum(np.abs(v) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -10) + np.abs(v) * rel
    assert np.all(np.abs(got - v) <= bound), "codes"


def forward(x, w, residual=None, quant="none", y=True, rstd=True):
    rows, cols = x.shape
    out = dict(y=torch.full_like(x, float("nan")) if y else None,
               residual_out=torch.full((rows, cols), float("nan"), dtype=x.dtype, device="cuda") if residual is not None else None,
               codes=torch.full((rows, cols), 0x7F, dtype=torch.uint8, device="cuda") if quant != "none" else None,
               scale={"none": None, "row": torch.full((rows,), float("nan"), device="cuda"),
                      "group": torch.full((rows, -(-cols // 128)), float("nan"), device="cuda")}[quant],
               rstd=torch.full((rows,), float("nan"), device="cuda") if rstd else None)
    dsa.dsa_rmsnorm(x, w, EPS, residual=residual, **out)
    return out


def check_forward(x, w, residual, quant, out):
    v, h, rstd = oracle.rmsnorm(f64(x), f64(w), EPS, None if residual is None else f64(residual))
    if out["y"] is not None:
        close(out["y"], v, np.abs(v), "y")
    if residual is not None:
        close(out["residual_out"], h, np.abs(h), "residual_out")
    if out["rstd"] is not None:
        close(out["rstd"], rstd, rstd, "rstd", rel=2 * F32)
    if quant != "none":
        check_codes(out["codes"], out["scale"], v, 128 if quant == "group" else 0)


# one lane, less than a warp, a warp's four pieces and one more, each register form, the widest, beyond it, odd
COLS = [1, 8, 120, 128, 250, 256, 264, 512, 1000, 1001, 1024, 1032, 2048, 4096, 5120, 8192, 16384, 4103, 9001, 20000, 33001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("quant", ["none", "row", "group"])
def test_forward(cols, dtype, quant):
    for rows in (1, 37):
        x, w = rnd((rows, cols), dtype, cols + rows), 1 + rnd((cols,), dtype, 3, 0.1)
        res = rnd((rows, cols), dtype, 7, 2.0) if cols % 3 else None
        check_forward(x, w, res, quant, forward(x, w, res, quant, y=quant == "none" or cols % 2 == 0))


@pytest.mark.parametrize("rows,cols", [(149, 4096), (1500, 1024), (700, 5120), (300, 33000), (149, 40000)])
def test_forward_many_rows_and_wide_ones(rows, cols):
    x, w = rnd((rows, cols), torch.bfloat16, 1), 1 + rnd((cols,), torch.bfloat16, 2, 0.1)
    res = rnd((rows, cols), torch.bfloat16, 3)
    check_forward(x, w, res, "group", forward(x, w, res, "group"))


@pytest.mark.parametrize("cols", [130, 251, 258, 500, 501, 513, 516, 777, 1001, 1002, 2052, 3001])
@pytest.mark.parametrize("quant", ["row", "group"])
def test_small_pieces_of_few_and_many_rows(cols, quant):
    for rows in (5, 593):
        x, w, res = rnd((rows, cols), torch.bfloat16, 1), 1 + rnd((cols,), torch.bfloat16, 2, 0.1), rnd((rows, cols), torch.bfloat16, 3)
        check_forward(x, w, res, quant, forward(x, w, res, quant))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,stride", [(0, 520), (8, 1024), (3, 517), (0, 515)])
def test_strided_and_misaligned_rows(dtype, offset, stride):
    base = rnd((40, stride), dtype, 5)
    x = base[:, :512] if offset == 0 else base.flatten()[offset:offset + 39 * stride + 512].as_strided((39, 512), (stride, 1))
    w = 1 + rnd((512,), dtype, 2, 0.1)
    out = torch.full((x.shape[0], stride), 7.0, dtype=dtype, device="cuda")
    rs = torch.empty(x.shape[0], device="cuda")
    dsa.dsa_rmsnorm(x, w, EPS, y=out[:, :512], rstd=rs)
    v, _, _ = oracle.rmsnorm(f64(x), f64(w), EPS)
    close(out[:, :512], v, np.abs(v), "y")
    assert (out[:, 512:] == 7).all()  # what lies between the rows is left alone


@pytest.mark.parametrize("cols", [512, 2048, 1001])
def test_outputs_in_place(cols):
    x, res, w = rnd((9, cols), torch.bfloat16, 1), rnd((9, cols), torch.bfloat16, 2), rnd((cols,), torch.bfloat16, 3)
    want = forward(x, w, res, "row")
    a, b = x.clone(), res.clone()
    codes, scale = torch.empty_like(want["codes"]), torch.empty_like(want["scale"])
    dsa.dsa_rmsnorm(a, w, EPS, y=a, residual=b, residual_out=b, codes=codes, scale=scale)
    assert torch.equal(a, want["y"]) and torch.equal(b, want["residual_out"])
    assert torch.equal(codes, want["codes"]) and torch.equal(scale, want["scale"])


@pytest.mark.parametrize("cols", [64, 300, 2048])
@pytest.mark.parametrize("group", [0, 128])
def test_zero_nan_and_infinite_rows(cols, group):
    x = rnd((6, cols), torch.float32, 1)
    x[0] = 0
    x[1, cols // 2] = float("nan")
    x[2, 0] = float("inf")
    x[3] *= 1e-18
    x[4] *= 1e15
    w = torch.ones(cols, device="cuda")
    out = forward(x, w, None, "group" if group else "row")
    y, codes, scale = out["y"].cpu(), out["codes"].cpu(), out["scale"].cpu().reshape(6, -1)
    assert (y[0] == 0).all() and (codes[0] == 0).all() and (scale[0] == 1).all()
    assert y[1].isnan().all() and (codes[1] & 0x7F == 0x7F).all() and (scale[1] == 1).all()
    assert y[2, 0].isnan() and (y[2, 1:] == 0).all() and codes[2, 0] & 0x7F == 0x7F
    rows = [3, 4, 5]
    v, _, _ = oracle.rmsnorm(f64(x[rows]), f64(w), EPS)
    close(out["y"][rows], v, np.abs(v), "y")
    check_codes(out["codes"][rows], out["scale"][rows], v, group)


@pytest.mark.parametrize("cols", [512, 2048, 1001])
def test_repeated_input_rows(cols):
    x, res, w = rnd((9, cols), torch.bfloat16, 1), rnd((1, cols), torch.bfloat16, 2).expand(9, cols), rnd((cols,), torch.bfloat16, 3)
    want, got = forward(x, w, res.contiguous(), "row"), forward(x, w, res, "row")
    assert all(torch.equal(got[k], want[k]) for k in ("y", "residual_out", "codes", "scale", "rstd"))
    dres = rnd((1, cols), torch.bfloat16, 4).expand(9, cols)
    a, b = backward(x, want["residual_out"], w, want["rstd"], dres), backward(x, want["residual_out"], w, want["rstd"], dres.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_zero_rows_are_no_work():
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    dsa.dsa_rmsnorm(x, w, EPS, y=torch.empty_like(x))
    dw = torch.full((64,), 5.0, device="cuda")
    dsa.dsa_rmsnorm_backward(x, x, w, torch.empty(0, device="cuda"), torch.empty_like(x), dw, torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert (dw == 0).all()


def backward(dy, h, w, rstd, dres=None):
    rows, cols = dy.shape
    dh = torch.full_like(dy, float("nan"))
    dw = torch.full((cols,), float("nan"), device="cuda")
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    dsa.dsa_rmsnorm_backward(dy, h, w, rstd, dh, dw, ws, dresidual=dres)
    return dh, dw


def check_backward(dy, h, w, rstd, dres, dh, dw):
    a = [f64(t) for t in (dy, h, w, rstd)]
    want, wantw = oracle.rmsnorm_backward(*a, None if dres is None else f64(dres))
    g, r = a[0] * a[2], a[3][:, None]
    mag = r * (np.abs(g) + np.abs(a[1]) * r * r * np.abs(g * a[1]).mean(1, keepdims=True))
    close(dh, want, mag + (0 if dres is None else np.abs(f64(dres))), "dh")
    close(dw, wantw, np.abs(a[0] * a[1] * r).sum(0), "dw", rel=2.0 ** -16)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_backward(cols, dtype):
    for rows in (1, 37):
        dy, h, w = rnd((rows, cols), dtype, cols + rows), rnd((rows, cols), dtype, 4), 1 + rnd((cols,), dtype, 3, 0.1)
        dres = rnd((rows, cols), dtype, 6) if cols % 3 else None
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
        check_backward(dy, h, w, rstd, dres, *backward(dy, h, w, rstd, dres))


@pytest.mark.parametrize("rows,cols", [(4000, 128), (1500, 2048), (1300, 1001), (5000, 8), (6000, 131), (5000, 202), (5000, 252)])
def test_backward_over_many_rows_repeats_its_bits(rows, cols):
    dy, h, w = rnd((rows, cols), torch.bfloat16, 1), rnd((rows, cols), torch.bfloat16, 2), rnd((cols,), torch.bfloat16, 3)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dh, dw = backward(dy, h, w, rstd)
    check_backward(dy, h, w, rstd, None, dh, dw)
    again = backward(dy, h, w, rstd)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


def test_backward_in_place_and_strided():
    base = rnd((3, 50, 600), torch.bfloat16, 1)
    dy, h, dres = base[0, :, :512], base[1, :, :512], base[2, :, :512]
    w = 1 + rnd((512,), torch.bfloat16, 3, 0.1)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    want = backward(dy.contiguous(), h.contiguous(), w, rstd, dres.contiguous())
    dw = torch.empty(512, device="cuda")
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(50, 512), dtype=torch.uint8, device="cuda")
    rest = base[:, :, 512:].clone()
    dsa.dsa_rmsnorm_backward(dy, h, w, rstd, dres, dw, ws, dresidual=dres)  # dh over the residual's gradient
    assert torch.equal(dres, want[0]) and torch.equal(dw, want[1]) and torch.equal(base[:, :, 512:], rest)


def test_gradient_against_differences_of_the_kernel():
    # fp32: a central difference of step 2^-8 is off by O(step^2) and by the forward's 2^-18 / step = 2^-10 of |y dy|
    rows, cols = 3, 40
    h, w, dy = rnd((rows, cols), torch.float32, 1), rnd((cols,), torch.float32, 2), rnd((rows, cols), torch.float32, 3)
    rstd = forward(h, w)["rstd"]
    dh, dw = backward(dy, h, w, rstd)
    e = 2.0 ** -8
    loss = lambda a, b: (forward(a, b)["y"].double() * dy.double()).sum().item()  # noqa: E731
    mag = (forward(h, w)["y"] * dy).abs().sum().item()
    for r, c in [(0, 0), (1, 17), (2, 39)]:
        d = torch.zeros_like(h)
        d[r, c] = e
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * e) - dh[r, c].item()) <= 2.0 ** -10 * mag + 8 * e * e * mag
    for c in (0, 20, 39):
        d = torch.zeros_like(w)
        d[c] = e
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * e) - dw[c].item()) <= 2.0 ** -10 * mag


def test_more_than_2_31_elements():
    rows, cols = 530000, 4096  # 2.17e9 elements
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    probe = [0, 1, 262143, 524288, rows - 1]
    x[probe] = rnd((5, cols), torch.bfloat16, 1)
    x[rows - 2] = 0
    w = 1 + rnd((cols,), torch.bfloat16, 2, 0.1)
    codes, scale = torch.empty((rows, cols), dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    dsa.dsa_rmsnorm(x, w, EPS, y=x, codes=codes, scale=scale)
    v, _, _ = oracle.rmsnorm(f64(rnd((5, cols), torch.bfloat16, 1)), f64(w), EPS)
    close(x[probe], v, np.abs(v), "y")
    check_codes(codes[probe], scale[probe], v, 0)
    assert (x[rows - 2] == 0).all()


def test_another_stream_and_a_captured_graph():
    x, w = rnd((64, 2048), torch.bfloat16, 1), rnd((2048,), torch.bfloat16, 2)
    want = forward(x, w, x, "group")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = forward(x, w, x, "group")
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["codes"], want["codes"])
    dy, rstd = rnd((64, 2048), torch.bfloat16, 3), want["rstd"]
    eager = backward(dy, x, w, rstd)
    a, b = dy.clone(), torch.empty_like(eager[1])
    dh = torch.empty_like(dy)
    ws = torch.empty(dsa.dsa_rmsnorm_backward_workspace_size(64, 2048), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_rmsnorm_backward(a, x, w, rstd, dh, b, ws)
    for seed in (4, 3):  # new values in the captured buffers, then the eager call's
        a.copy_(rnd((64, 2048), torch.bfloat16, seed))
        dh.zero_()
        g.replay()
        check_backward(a, x, w, rstd, None, dh, b)
    assert torch.equal(dh, eager[0]) and torch.equal(b, eager[1])


def test_calls_from_several_threads():
    """Different sizes at once, each on its own stream with its own workspace."""
    import threading

    cases, errors = [], []
    for i, cols in enumerate((512, 2048, 5120, 8192)):
        dy, h, w = rnd((300, cols), torch.bfloat16, i), rnd((300, cols), torch.bfloat16, 9 + i), rnd((cols,), torch.bfloat16, 3)
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
        cases.append((dy, h, w, rstd, backward(dy, h, w, rstd)))
    torch.cuda.synchronize()

    def work(dy, h, w, rstd, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    dh, dw = backward(dy, h, w, rstd)
                    assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])
        except BaseException as e:  # noqa: BLE001 (shown by the assertion below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_wrapper_refusals():
    x, w = torch.zeros((4, 64), device="cuda"), torch.zeros(64, device="cuda")
    for kw in (dict(y=x.half()), dict(y=x[:, :32]), dict(y=x, residual=x[:2]), dict(y=x, rstd=torch.zeros(5, device="cuda")),
               dict(codes=x, scale=torch.zeros(4, device="cuda")), dict(y=x.t().contiguous().t()), dict(y=torch.zeros(4, 64)),
               dict(codes=torch.zeros((4, 64), dtype=torch.uint8, device="cuda"), scale=torch.zeros((4, 2), device="cuda"))):
        with pytest.raises(ValueError):
            dsa.dsa_rmsnorm(x, w, EPS, **kw)
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm(x.double(), w.double(), EPS, y=x.double())
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm(x, w.half(), EPS, y=x)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rmsnorm(x, w, EPS, y=x[:1].expand(4, 64))  # rows of an output on one another
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rmsnorm(x, w, EPS)                         # no output
