"""The layer norm on the GPU against 64 bits.

Tolerances, before any run.  Statistics are fp32 sums of N terms in a tree over
at most 32 serial additions: 2^-24 · (N/256 + 40) of the sums of absolute
values; a result rounded to bf16 adds 2^-8 of itself.  dweight and dbias are
fp32 sums over rows, serial over at most rows/8 additions."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def api():
    from non_linear_matrix_persistent_b200 import api as a
    return a


def reference(x, w, b, dy, heads, rms, eps):
    x = x.double().requires_grad_()
    w = None if w is None else w.double().requires_grad_()
    b = None if b is None else b.double().requires_grad_()
    z = x.transpose(1, 2) if heads else x
    mean = torch.zeros_like(z[..., :1]) if rms else z.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((z - mean).square().mean(-1, keepdim=True) + eps)
    n = (z - mean) * rstd
    y = n if w is None else n * w
    y = y if b is None else y + b
    y.backward(dy.double())
    return y.detach(), x.grad, n.detach(), rstd.detach(), mean.detach(), None if w is None else w.grad


def check(shape, heads=False, x=BF, y=BF, dx=None, rms=False, weight=True, bias=True, eps=1e-5, scale=1.0, offset=0.0, seed=0):
    a = api()
    g = torch.Generator().manual_seed(seed)
    N = shape[-1]
    xt = (torch.randn(*shape, generator=g) * scale + offset).to(x).to(DEV)
    ws = (shape[1], N) if heads else (N,)
    w = (1 + 0.2 * torch.randn(*ws, generator=g)).to(DEV) if weight else None
    b = (0.3 * torch.randn(*ws, generator=g)).to(DEV) if bias else None
    yshape = (shape[0], shape[2], shape[1], N) if heads else shape
    dy = torch.randn(*yshape, generator=g).to(y).to(DEV)
    got, mean, rstd = a.layer_norm(xt, w, b, eps=eps, rms=rms, out_dtype=y)
    assert got.dtype == y and tuple(got.shape) == tuple(yshape) and (mean is None) == rms
    grads = a.layer_norm_backward(dy, xt, w, mean, rstd, rms=rms, dx_dtype=dx)
    wy, wdx, n, wr, wm, ww = reference(xt, w, b, dy, heads, rms, eps)
    sums = 2.0 ** -24 * (N / 256 + 40)
    half = lambda t: 2.0 ** -8 if t == BF else 2.0 ** -24  # noqa: E731
    # n's error: the mean's (relative to mean |x|, scaled by rstd) and rstd's relative one
    z = (xt.transpose(1, 2) if heads else xt).double()
    en = sums * (z.abs().mean(-1, keepdim=True) + z.abs()) * wr + 2 * sums * n.abs() + 2.0 ** -22 * n.abs()
    # the deviations' own rounding enters rstd as twice its mean over the row
    en = en + n.abs() * en.mean(-1, keepdim=True)
    wa = 1.0 if w is None else w.double().abs()
    err = (got.double() - wy).abs() - (half(y) * wy.abs() + en * wa + 2.0 ** -22 * wy.abs() + 1e-30)
    assert float(err.max()) <= 0, float(err.max())
    gd = dy.double() * (1.0 if w is None else w.double())
    m = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    scale_dx = wr * (gd.abs() + m(gd.abs()) * (0 if rms else 1) + n.abs() * m((gd * n).abs()))
    edx = wr * (en * m((gd * n).abs()) + n.abs() * m(gd.abs() * en)) + 4 * sums * scale_dx + 2.0 ** -21 * scale_dx \
        + scale_dx * (en.mean(-1, keepdim=True))
    wdx = wdx.transpose(1, 2) if heads else wdx
    gdx = grads["dx"].transpose(1, 2) if heads else grads["dx"]
    dt = dx or x
    assert grads["dx"].dtype == dt
    err = (gdx.double() - wdx).abs() - (half(dt) * wdx.abs() + edx + 1e-30)
    assert float(err.max()) <= 0, float(err.max())
    rows = (0, 1) if heads else tuple(range(len(shape) - 1))
    count = wy.numel() // (N * (shape[1] if heads else 1))
    tol = 2.0 ** -24 * (count / 8 + 64)
    dyd = dy.double()
    dw = (dyd * n).sum(rows)
    assert ww is None or torch.allclose(dw, ww)
    err = (grads["dweight"].double() - dw).abs() - (tol * (dyd * n).abs().sum(rows) + (dyd.abs() * en).sum(rows) + 1e-30)
    assert float(err.max()) <= 0, float(err.max())
    err = (grads["dbias"].double() - dyd.sum(rows)).abs() - (tol * dyd.abs().sum(rows) + 1e-30)
    assert float(err.max()) <= 0, float(err.max())
    return got, grads


@pytest.mark.parametrize("N", [1, 2, 7, 8, 16, 24, 31, 64, 100, 128, 200, 256, 257, 264, 1000, 1024, 1032, 2047, 2048, 2056, 4096, 4097, 8192])
@pytest.mark.parametrize("rms", [False, True])
def test_row_lengths(N, rms):
    check((37, N), rms=rms, seed=N, eps=1e-5 if N > 1 else 1.0)


@pytest.mark.parametrize("N", [8200, 9001, 20000])
def test_rows_longer_than_the_registers_hold(N):
    check((5, N), seed=N)
    check((5, N), seed=N, x=F32, y=BF, rms=True, bias=False)


@pytest.mark.parametrize("V", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H,T", [(1, 1, 1), (2, 3, 5), (3, 16, 130), (1, 5, 1000)])
def test_readouts(V, B, H, T):
    check((B, H, T, V), heads=True, seed=V + T)


@pytest.mark.parametrize("x,y,dx", [(BF, BF, None), (BF, F32, None), (F32, F32, None), (F32, BF, None), (F32, BF, BF), (F32, F32, BF)])
@pytest.mark.parametrize("shape,heads", [((2, 4, 70, 64), True), ((33, 300), False), ((33, 301), False), ((9, 2048), False)])
def test_types(x, y, dx, shape, heads):
    check(shape, heads=heads, x=x, y=y, dx=dx, seed=1)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(weight, bias):
    check((19, 96), weight=weight, bias=bias, seed=2)


def test_readout_without_weight_in_the_backward():
    a = api()
    x = torch.randn(2, 3, 20, 64, device=DEV)
    y, mean, rstd = a.layer_norm(x, torch.ones(3, 64, device=DEV))
    dy = torch.randn(2, 20, 3, 64, device=DEV)
    p = a.layer_norm_backward(dy, x, torch.ones(3, 64, device=DEV), mean, rstd)
    r = a.layer_norm_backward(dy, x, None, mean, rstd, heads=True)
    assert all(torch.equal(p[n], r[n]) for n in p)


@pytest.mark.parametrize("scale,offset", [(1e-3, 0.0), (1.0, 1000.0), (1e4, 0.0)])
def test_scales_and_offsets(scale, offset):
    """A mean a thousand times the spread: the two-pass variance keeps it."""
    check((50, 512), x=F32, y=F32, scale=scale, offset=offset, seed=3)


def test_constant_rows_and_one_value():
    a = api()
    x = torch.full((4, 64), 3.0, dtype=BF, device=DEV)
    y, mean, rstd = a.layer_norm(x, torch.ones(64, device=DEV), torch.full((64,), 0.5, device=DEV))
    assert torch.equal(y, torch.full_like(y, 0.5)) and torch.equal(mean, torch.full((4,), 3.0, device=DEV))
    assert torch.allclose(rstd, torch.full((4,), 1e-5, device=DEV).rsqrt(), rtol=1e-6)


def test_a_row_of_nans_stays_in_its_row():
    a = api()
    for N in (64, 100, 2048, 9000):
        x = torch.randn(70, N, device=DEV).to(BF)
        x[3] = float("nan")
        x[11, 0] = float("inf")
        y, mean, rstd = a.layer_norm(x)
        ok = torch.ones(70, dtype=torch.bool)
        ok[[3, 11]] = False
        assert bool(torch.isfinite(y[ok.to(DEV)]).all()) and bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[11]).any())
        dx = a.layer_norm_backward(torch.randn(70, N, device=DEV).to(BF), x, None, mean, rstd)["dx"]
        assert bool(torch.isfinite(dx[ok.to(DEV)]).all())


def test_empty_and_leading_shapes():
    a = api()
    w = torch.ones(64, device=DEV)
    y, m, r = a.layer_norm(torch.zeros(0, 64, device=DEV), w)
    assert y.shape == (0, 64)
    g = a.layer_norm_backward(y, y, w, m, r)
    assert float(g["dweight"].abs().max()) == 0 and float(g["dbias"].abs().max()) == 0
    x = torch.randn(2, 3, 4, 64, device=DEV)
    y, m, r = a.layer_norm(x, w)
    assert y.shape == x.shape and m.shape == (2, 3, 4)
    y1, _, _ = a.layer_norm(x[1, 2, 3], w)
    assert torch.equal(y1, y[1, 2, 3])


def test_in_place_and_repeatable():
    a = api()
    x = torch.randn(3, 7, 501, 64, device=DEV).to(BF)
    w = torch.randn(7, 64, device=DEV)
    dy = torch.randn(3, 501, 7, 64, device=DEV).to(BF)
    _, m, r = a.layer_norm(x, w)
    one = a.layer_norm_backward(dy, x, w, m, r)
    for _ in range(3):
        two = a.layer_norm_backward(dy, x, w, m, r)
        assert all(torch.equal(one[n], two[n]) for n in one)
    buf = x.clone()
    three = a.layer_norm_backward(dy, buf, w, m, r, out={"dx": buf})
    assert all(torch.equal(one[n], three[n]) for n in one)


def test_gradients_against_differences():
    a = api()
    gen = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    args = {"x": n(2, 3, 6, 32), "weight": 1 + 0.2 * n(3, 32), "bias": n(3, 32)}
    dy = n(2, 6, 3, 32)
    for rms in (False, True):
        y, m, r = a.layer_norm(*args.values(), rms=rms)
        g = a.layer_norm_backward(dy, args["x"], args["weight"], m, r, rms=rms)
        for name, t in args.items():
            d = n(*t.shape)
            h = 2.0 ** -8
            f = lambda v: float((a.layer_norm(*{**args, name: v}.values(), rms=rms)[0].double() * dy.double()).sum())  # noqa: E731
            num = (f(t + h * d) - f(t - h * d)) / (2 * h)
            scale = float(g["d" + name].double().norm() * d.double().norm())
            # truncation h^2 (1.5e-5) of third derivatives of size O(1), rounding 2^-24 · |loss| / h
            assert abs(num - float((g["d" + name].double() * d.double()).sum())) <= 2e-3 * scale, (name, rms)


def test_readout_of_the_scan_and_its_gradient():
    """forward -> layer_norm -> layer_norm_backward -> backward, the fp32 readout normalised to bf16 rows and
    its gradient handed to the scan's backward as bf16."""
    from non_linear_matrix_persistent_b200 import Workload, make_inputs
    a = api()
    x = {i: None if t is None else t.to(DEV) for i, t in make_inputs(Workload("n", 2, 4, 40, 64, 64, backward=True)).items()}
    y, _, ck = a.forward(x["k"], x["v"], x["q"], x["f"], x["W"], want_ckpt=True)
    w = 1 + 0.1 * torch.randn(4, 64, device=DEV)
    z, m, r = a.layer_norm(y, w, rms=True, out_dtype=BF)
    dz = x["dY"].transpose(1, 2).contiguous()
    g = a.layer_norm_backward(dz, y, w, m, r, rms=True, dx_dtype=BF)
    wy, wdx, *_ = reference(y, w, None, dz, True, True, 1e-5)
    assert float((z.double() - wy).norm() / wy.norm()) <= 2.0 ** -8
    assert float((g["dx"].double() - wdx).norm() / wdx.norm()) <= 2.0 ** -8
    back = a.backward(x["k"], x["v"], x["q"], x["f"], x["W"], ck, g["dx"])
    assert all(bool(torch.isfinite(t).all()) for t in back.values())


@pytest.mark.parametrize("shape,heads", [((2, 3, 500, 64), True), ((700, 2048), False)])
def test_captured_and_replayed(shape, heads):
    """A captured forward and backward, replayed on new inputs, gives the eager results, twice in a row too."""
    a = api()
    g = torch.Generator().manual_seed(31)
    N = shape[-1]
    x = torch.randn(*shape, generator=g).to(BF).to(DEV)
    dy = torch.randn(*((shape[0], shape[2], shape[1], N) if heads else shape), generator=g).to(BF).to(DEV)
    w = torch.randn(*((shape[1], N) if heads else (N,)), generator=g).to(DEV)

    def work():
        y, mean, rstd = a.layer_norm(x, w)
        d = a.layer_norm_backward(dy, x, w, mean, rstd)
        return [y, d["dx"], d["dweight"], d["dbias"]]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = work()
        second = work()
    for _ in range(2):
        x.copy_(torch.randn(*shape, generator=g))
        dy.copy_(torch.randn(*dy.shape, generator=g))
        want = work()
        for t in first + second:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got in (first, second):
            assert all(torch.equal(p, q) for p, q in zip(got, want))
