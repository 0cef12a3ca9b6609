"""Gradients of fp16 layers (ozaki2_linear_grad) whose G = dY act'(Z) leaves fp16's range, against the formulas in 64 bits.

G is rounded to fp16 in units of a power of two u in which the largest finite |dY| is at least 2^14: an entry is off by 2^-11 of itself or by half
the subnormal step, 2^-25 u <= 2^-39 max|dY|, and none overflows. The rest as in test_gpu_linear: sums of binary32, slopes, and the result's own
rounding to fp16, whose subnormal half step is 2^-25."""
import math

import pytest
import torch

import rns_emulated_fp64_amd as oz
from layer_util import HALF, NAMES, U32, rounded_to, slope, slope_error
from test_gpu_linear import close, gen

pytestmark = pytest.mark.gpu

SMOOTH = ["gelu", "gelu_tanh", "silu"]


def check(got, dY, X, W, Z, name, rows=slice(None)):
    """Of the rows of dX that `rows` names, of dW and of dbias."""
    dX, dW, db = got
    z = Z.double()
    s = slope(name, z)
    g = dY.double() * s
    dg = dY.double().abs() * (slope_error(name, z) + U32 * s.abs())
    t, n = g.shape
    if db is not None:
        close(db, g.sum(0), dg.sum(0) + t * 2 * U32 * (g.abs() + dg).sum(0) + 2.0 ** -150, "dbias")
    dg = dg + HALF[torch.float16] * (g.abs() + dg) + 2.0 ** -39 * dY[torch.isfinite(dY)].abs().max().double()
    for out, a, da, b, terms, what in ((dX, g[rows], dg[rows], W, n, "dX"), (dW, g.t().contiguous(), dg.t().contiguous(), X, t, "dW")):
        if out is None:
            continue
        b = b.double().contiguous()
        want = a @ b
        tol = da @ b.abs() + terms * 2 * U32 * ((a.abs() + da) @ b.abs())
        close(out[rows] if what == "dX" else out, want, rounded_to(torch.float16, want, tol), what)


def operands(t, n, k, seed, z_at, size):
    g = gen(seed)
    X = torch.randn(t, k, generator=g, device="cuda").half()
    W = (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).half()
    Z = (torch.randn(t, n, generator=g, device="cuda") * 0.7 + z_at).half()
    dY = (torch.randn(t, n, generator=g, device="cuda") * size).half()
    return X, W, Z, dY


# few tokens, slices of a long k in either product, odd sizes, a narrow layer, large tiles
SIZES = [(1, 300, 512), (60, 200, 72), (509, 2051, 768), (2000, 130, 264), (7457, 28, 64), (300, 511, 1023), (8192, 300, 264)]


@pytest.mark.parametrize("t,n,k", SIZES)
@pytest.mark.parametrize("name", SMOOTH)
def test_small_gradients(t, n, k, name):
    for size in (1e-4, 1e-5, 2e-6):
        for z_at in (-4.0, 0.0):
            X, W, Z, dY = operands(t, n, k, t + n, z_at, size)
            check(oz.linear_grad(dY, X, W, Z, name), dY, X, W, Z, name)


def test_error_of_a_mean_loss_over_thousands_of_tokens():
    # by their norm: within 1.5 times what the roundings of G and of the result leave together, 2^-11 / sqrt(3) each at most of values that fp16
    # holds as normal numbers (X in hundreds, so that the results are)
    X, W, Z, dY = operands(8192, 256, 512, 1, -4.0, 1e-5)
    X = (X * 100).half()
    dX, dW, _ = oz.linear_grad(dY, X, W, Z, "silu")
    want = (dY.double() * slope("silu", Z.double())).t().contiguous() @ X.double()
    assert float((dW.double() - want).norm() / want.norm()) < 1.5 * 2.0 ** -11 * math.sqrt(2 / 3)


@pytest.mark.parametrize("name", SMOOTH)
def test_slopes_above_one_of_the_largest_gradients(name):
    # G is beyond fp16 where dX and dW are not
    X, W, Z, dY = operands(200, 136, 64, 2, 0.0, 1.0)
    Z[::2] = 1.4 if name != "silu" else 2.4  # slopes of 1.13, 1.13 and 1.10
    dY = (dY.sign() * 60000).half()
    X, W = (X / 256).half(), (W / 256).half()
    got = oz.linear_grad(dY, X, W, Z, name)
    assert all(torch.isfinite(v).all() for v in got)
    check(got, dY, X, W, Z, name)


def test_tokens_with_infinite_gradients_do_not_set_the_unit():
    X, W, Z, dY = operands(150, 200, 72, 3, -4.0, 1e-5)
    bad = dY.clone()
    bad[3, 5], bad[70], bad[149, 199] = math.inf, math.nan, -math.inf
    fine = [i for i in range(150) if i not in (3, 70, 149)]
    dX, _, _ = oz.linear_grad(bad, X, W, Z, "silu")
    assert not torch.isfinite(dX[[3, 70, 149]]).any()
    check((dX, None, None), torch.where(torch.isfinite(bad), bad, torch.zeros_like(bad)), X, W, Z, "silu", fine)


def test_ends_of_the_range():
    X, W, Z, dY = operands(40, 72, 64, 4, 0.0, 1.0)
    X, W = torch.ones_like(X), torch.ones_like(W)
    for value in (0.0, 2.0 ** -24, -(2.0 ** -24), 2.0 ** -14, 65504.0):
        g = torch.zeros_like(dY)
        g[7, 3] = value
        Z[7, 3] = 100.0  # a slope of 1
        dX, dW, db = oz.linear_grad(g, X, W, Z, "gelu")
        assert (dX[7] == value).all() and (dW[3] == value).all() and db[3] == value
        assert int((dX != 0).sum()) == (64 if value else 0) == int((dW != 0).sum())


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (True, True, False), (False, True, True)])
def test_each_gradient_alone(want):
    X, W, Z, dY = operands(300, 300, 96, 5, -4.0, 1e-5)
    whole = oz.linear_grad(dY, X, W, Z, "silu")
    got = oz.linear_grad(dY, X, W, Z, "silu", *want)
    for a, b, wanted in zip(got, whole, want):
        assert torch.equal(a, b) if wanted else a is None


def test_values_of_relu_and_none_are_not_scaled():
    # their G is dY's own values: integers give exact sums
    g = gen(6)
    X, W = (torch.randint(-8, 9, (x, 64), generator=g, device="cuda").half() for x in (130, 200))
    Z, dY = (torch.randint(-8, 9, (130, 200), generator=g, device="cuda").half() for _ in range(2))
    for name in ("none", "relu"):
        G = (dY.double() * slope(name, Z.double())).contiguous()
        dX, dW, db = oz.linear_grad(dY, X, W, Z, name)
        assert torch.equal(dX, (G @ W.double()).half()) and torch.equal(dW, (G.t().contiguous() @ X.double()).half())
        assert torch.equal(db, G.sum(0).float())


def test_replays_find_their_own_unit():
    t, n, k = 509, 300, 264
    X, W, Z, dY = operands(t, n, k, 7, -4.0, 1e-5)
    ws = torch.empty(oz.ozaki2_linear_grad_workspace_size(t, n, k), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        oz.linear_grad(dY, X, W, Z, "silu", workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = oz.linear_grad(dY, X, W, Z, "silu", workspace=ws)
    for seed, size in ((8, 1e-6), (9, 3.0), (10, 1e-4)):
        for a, b in zip((X, W, Z, dY), operands(t, n, k, seed, -3.0, size)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        again = [v.clone() for v in got]
        check(again, dY, X, W, Z, "silu")
        for a, b in zip(again, oz.linear_grad(dY, X, W, Z, "silu")):
            assert torch.equal(a, b)
