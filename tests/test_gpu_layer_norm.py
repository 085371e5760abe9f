"""Layer norm on the GPU against float64 with elementwise bounds (tests/ops_bounds.py)."""
import pytest
import torch

from . import ops_bounds as ob

pytestmark = pytest.mark.gpu


def p3d():
    import geometry_aware_local_pack3d_b200 as m
    return m


def make(rows, cols, dtype, wdtype, seed=0, offset=0.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    size = 0.1 + 4 * torch.rand(rows, 1, generator=gen, device="cuda")
    x = (rnd(rows, cols) * size + offset).to(dtype)
    return x, (1 + 0.3 * rnd(cols)).to(wdtype), rnd(cols).to(wdtype), rnd(rows, cols).to(dtype)


def run_and_check(x, w, b, dy, eps=1e-5):
    f = p3d().pack3d_layer_norm_fwd(x, w, b, eps=eps, save_for_backward=True)
    wt = torch.float32 if w is None else w.dtype
    want = ob.layer_norm(x, w, b, eps, dy, wt)
    for n in ("y", "mean", "rstd"):
        ob.check(f[n], want[n], n)
    g = p3d().pack3d_layer_norm_bwd(dy, x, w, f)
    for n in ("dx", "dweight", "dbias"):
        ob.check(g[n], want[n], n)
    return f, g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 32, 48, 64, 96, 100, 128, 129, 255, 384, 513, 768, 1001,
                                  1024, 1032, 2048, 4095, 4104, 5000, 8184, 8191, 8200, 9001, 17000])
def test_widths(dtype, cols):
    run_and_check(*make(37, cols, dtype, torch.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 96), (3, 768), (5000, 48), (20001, 96), (4099, 201)])
def test_rows_and_types(dtype, wdtype, rows, cols):
    run_and_check(*make(rows, cols, dtype, wdtype, seed=2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_weight_or_bias_and_on_head_rows(dtype):
    x, w, b, dy = make(2 * 3 * 50, 96, dtype, torch.float32)
    run_and_check(x, None, None, dy)
    run_and_check(x, w, None, dy)
    x4, dy4 = x.view(2, 3, 50, 96), dy.view(2, 3, 50, 96)
    f = p3d().pack3d_layer_norm_fwd(x4, w, b, save_for_backward=True)
    assert f["y"].shape == x4.shape and f["mean"].shape == (2, 3, 50)
    g = p3d().pack3d_layer_norm_bwd(dy4, x4, w, f, bias_grad=False)
    assert g["dbias"] is None and g["dx"].shape == x4.shape
    g2 = p3d().pack3d_layer_norm_bwd(dy4, x4, w, f, weight_grad=False, bias_grad=False)
    assert g2["dweight"] is None and torch.equal(g2["dx"], g["dx"])


def test_large_mean_constant_rows_and_no_rows():
    # the variance about the mean, not the difference of two large sums
    x, w, b, dy = make(64, 768, torch.float32, torch.float32, offset=1000.0)
    run_and_check(x, w, b, dy)
    c = torch.full((4, 96), 3.0, device="cuda")
    f = p3d().pack3d_layer_norm_fwd(c, w[:96].contiguous(), b[:96].contiguous())
    assert torch.equal(f["y"], b[:96].expand(4, 96))
    e = torch.empty(0, 96, device="cuda")
    f = p3d().pack3d_layer_norm_fwd(e, save_for_backward=True)
    g = p3d().pack3d_layer_norm_bwd(e, e, None, f)
    assert torch.equal(g["dweight"], torch.zeros(96, device="cuda")) and f["y"].numel() == 0


def test_rows_with_infinities_and_nan_keep_to_themselves():
    x, w, b, _ = make(40, 96, torch.bfloat16, torch.float32)
    ref = p3d().pack3d_layer_norm_fwd(x, w, b)["y"]
    x[7, 3], x[9, 0] = float("nan"), float("inf")
    y = p3d().pack3d_layer_norm_fwd(x, w, b)["y"]
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[7] = keep[9] = False
    assert torch.equal(y[keep], ref[keep]) and bool(y[~keep].isnan().all())


def test_repeats_streams_and_capture():
    x, w, b, dy = make(3000, 768, torch.bfloat16, torch.float32)
    f, g = run_and_check(x, w, b, dy)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    f2 = p3d().pack3d_layer_norm_fwd(x, w, b, save_for_backward=True, stream=s)
    g2 = p3d().pack3d_layer_norm_bwd(dy, x, w, f2, stream=s)
    torch.cuda.synchronize()
    for n in ("dx", "dweight", "dbias"):
        assert torch.equal(g[n], g2[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3 = p3d().pack3d_layer_norm_fwd(x, w, b, save_for_backward=True)
        g3 = p3d().pack3d_layer_norm_bwd(dy, x, w, f3)
    x2, _, _, dy2 = make(3000, 768, torch.bfloat16, torch.float32, seed=8)
    x.copy_(x2)
    dy.copy_(dy2)
    graph.replay()
    torch.cuda.synchronize()
    want = ob.layer_norm(x, w, b, 1e-5, dy)
    for n in ("dx", "dweight", "dbias"):
        ob.check(g3[n], want[n], n)


def test_gradient_against_differences():
    x, w, b, dy = make(6, 50, torch.float32, torch.float32, seed=4)
    f = p3d().pack3d_layer_norm_fwd(x, w, b, save_for_backward=True)
    g = p3d().pack3d_layer_norm_bwd(dy, x, w, f)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for name, at in (("dx", x), ("dweight", w), ("dbias", b)):
        t = torch.randn(at.shape, generator=gen, device="cuda")
        h, vals = 2.0 ** -8, []
        for s in (h, -h):
            a = {"dx": x, "dweight": w, "dbias": b, name: at + s * t}
            y = p3d().pack3d_layer_norm_fwd(a["dx"], a["dweight"], a["dbias"])["y"]
            vals.append(float((y.double() * dy.double()).sum()))
        got, want = (vals[0] - vals[1]) / (2 * h), float((g[name].double() * t.double()).sum())
        assert abs(got - want) <= 5e-3 * (1 + abs(want)), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(30001, 3), (20001, 9), (9001, 31), (5001, 333), (3001, 511), (1, 257)])
def test_ragged_widths_over_many_rows(dtype, rows, cols):
    run_and_check(*make(rows, cols, dtype, torch.float32))


def test_the_longest_row():
    # 2^31 - 1 columns: the last ones lie less than a block's threads below the largest 32-bit number.
    # Of a row of +1, -1, +1, ... every partial sum is a whole number below 2^24 until 512 of them
    # are added, so the mean is 2^-31 to within rounding, and the variance 1.
    cols = 2 ** 31 - 1
    x = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    x[0, 1::2] = -1
    f = p3d().pack3d_layer_norm_fwd(x, save_for_backward=True)
    assert torch.equal(f["y"], x)  # (1 +- 2^-31) / sqrt(1 + 1e-5), rounded
    assert abs(float(f["mean"])) <= 2.0 ** -24 and abs(float(f["rstd"]) - (1 + 1e-5) ** -0.5) <= 8 * ob.U
    del f["y"]
    g = p3d().pack3d_layer_norm_bwd(x, x, None, f)
    rstd = float(f["rstd"])
    for at in (slice(0, 1000), slice(cols - 1000, cols)):
        assert bool(((g["dweight"][at] - rstd).abs() <= 2.0 ** -22).all())
        assert torch.equal(g["dbias"][at], x[0, at].float())
        # dx = rstd (g - mean g - x^ mean(g x^)) with g = x and x^ = rstd x, so x dx is
        # rstd (1 - rstd mean(rstd)) = 1e-5. A thread adds 2^22 terms rstd = 1 - 5e-6 to a float32 sum,
        # whose steps from 2^8 on are 2^-15 and more: there each term counts as 1. The mean lies between
        # rstd and 1, and x dx between rstd (1 - rstd) = 5e-6 and 1e-5, to within a few roundings of
        # terms of size one.
        xdx = g["dx"][0, at].float() * x[0, at].float()
        low, high = float(xdx.min()), float(xdx.max())
        assert rstd * (1 - rstd) - 2.0 ** -20 <= low and high <= 1e-5 + 2.0 ** -20
    assert float(g["dweight"].min()) > 0.99 and float(g["dweight"].max()) < 1.01


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 7, 31, 333, 1001, 8191, 8201, 17001])
def test_ragged_rows_start_at_any_element(dtype, cols):
    # a slice of rows of an odd width starts where the row before it ends
    x, w, b, dy = make(12, cols, dtype, torch.float32, seed=6)
    want, wantg = run_and_check(x[1:].clone(), w, b, dy[1:].clone())
    for shift in (1, 3):
        buf, out = (torch.full((11 * cols + 16,), 5.0, dtype=dtype, device="cuda") for _ in range(2))
        view, y = (t[shift:shift + 11 * cols].view(11, cols) for t in (buf, out))
        view.copy_(x[1:])
        f = p3d().pack3d_layer_norm_fwd(view, w, b, y=y, save_for_backward=True)
        assert torch.equal(y, want["y"]) and f["y"] is y
        assert bool((out[:shift] == 5.0).all()) and bool((out[shift + 11 * cols:] == 5.0).all())
        g = p3d().pack3d_layer_norm_bwd(dy[1:], view, w, f)
        for n in ("dx", "dweight", "dbias"):
            assert torch.equal(g[n], wantg[n]), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(20001, 128), (10001, 256), (6001, 512), (5001, 1024), (1501, 4096),
                                       (801, 8192), (301, 16384)])
def test_rows_of_four_pieces_a_thread_over_many_rows(dtype, rows, cols):
    # the most registers per thread: several rows for each group of threads, forward and backward
    run_and_check(*make(rows, cols, dtype, torch.float32, seed=12))
