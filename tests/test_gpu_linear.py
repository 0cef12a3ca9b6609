"""16-bit layers with their epilogue (ozaki2_linear) and their gradients (ozaki2_linear_grad) against the formulas in 64 bits.

A binary32 sum of k products, in whatever order, is off by at most k steps (2^-23) of the sum of the products' magnitudes (the
products of 16-bit values are exact; every partial sum is below that sum of magnitudes, and the matrix cores may cut
where they do not round). Bias, activation and residual add what layer_util states, and the output's rounding half a step
of its type. Where inputs are small integers every sum is exact, and results are compared bit for bit."""
import pytest
import torch

import rns_emulated_fp64_amd as oz
from layer_util import HALF, NAMES, TINY, U32, act, act_error, rounded_to, slope, slope_error

pytestmark = pytest.mark.gpu

TILES = ("skinny", "s11", "s21", "s22", "s42", "p4", "p8", "any")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(t, n, k, dtype, seed, pad=0):
    g = gen(seed)
    X = torch.randn(t, k + pad, generator=g, device="cuda").to(dtype)[:, pad:]
    W = (torch.randn(n, k + pad, generator=g, device="cuda") / max(k, 1) ** 0.5).to(dtype)[:, pad:]
    bias = torch.randn(n, generator=g, device="cuda")
    residual = torch.randn(t, n, generator=g, device="cuda") * 2
    return X, W, bias, residual


def product(A, B):
    """A @ B.T in 64 bits, and the bound on the binary32 sums."""
    a, b = A.double().contiguous(), B.double().t().contiguous()
    return a @ b, A.shape[1] * 2 * U32 * (a.abs() @ b.abs())


def close(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def check(got, X, W, bias, name, residual):
    Y, Z = got
    z, dz = product(X, W)
    if bias is not None:
        dz = dz + U32 * (z.abs() + dz + bias.double().abs())
        z = z + bias.double()
    if Z is not None:
        close(Z, z, rounded_to(Z.dtype, z, dz), "Z")
    y, dy = act(name, z), act_error(name, z, dz)
    if residual is not None:
        dy = dy + U32 * (y.abs() + dy + residual.double().abs())
        y = y + residual.double()
    close(Y, y, rounded_to(Y.dtype, y, dy), "Y")


SHAPES = [(1, 1, 1), (1, 300, 4096), (3, 17, 15), (2, 33, 64), (16, 100, 300), (17, 333, 77), (31, 65, 272), (33, 129, 1000),
          (64, 257, 1024), (65, 66, 65), (100, 200, 304), (129, 127, 1040), (257, 300, 400), (300, 511, 1023), (700, 3001, 200)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer(t, n, k, dtype):
    X, W, bias, residual = operands(t, n, k, dtype, t + n + k)
    name = NAMES[(t + n + k) % 5]
    check(oz.linear(X, W), X, W, None, "none", None)
    check(oz.linear(X, W, bias, name, residual.to(dtype), want_pre=True), X, W, bias, name, residual.to(dtype))
    check(oz.linear(X, W, bias, name, residual, out_dtype=torch.float32, want_pre=True), X, W, bias, name, residual)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("t,n,k", [(1, 128, 512), (40, 130, 96), (300, 520, 256)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_activations(name, t, n, k, out):
    X, W, bias, residual = operands(t, n, k, torch.bfloat16, 3)
    X = X * 3  # pre-activations out to the tails
    for b, r in ((None, None), (bias, None), (None, residual.to(out)), (bias, residual.to(out))):
        check(oz.linear(X, W, b, name, r, out_dtype=out), X, W, b, name, r)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("t,n,k,pad", [(1, 40, 256, 0), (16, 300, 400, 0), (50, 700, 528, 8), (64, 64, 1024, 0), (130, 257, 384, 16),
                                       (300, 600, 272, 0), (513, 1030, 256, 0), (70, 90, 1001, 3), (300, 300, 129, 0)])
def test_every_tile(tile, t, n, k, pad, monkeypatch):
    # integers up to 8 in 16-bit values: sums are exact in binary32 and so the same from every kernel, split and order
    g = gen(t + n)
    X = torch.randint(-8, 9, (t, k + pad), generator=g, device="cuda").to(torch.float16)[:, pad:]
    W = torch.randint(-8, 9, (n, k + pad), generator=g, device="cuda").to(torch.float16)[:, pad:]
    bias = torch.randint(-50, 50, (n,), generator=g, device="cuda").float()
    residual = torch.randint(-50, 50, (t, n), generator=g, device="cuda").to(torch.float16)
    z = X.double().contiguous() @ W.double().t().contiguous() + bias.double()
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    Y, Z = oz.linear(X, W, bias, "relu", residual, want_pre=True)
    assert torch.equal(Z, z.to(torch.float16))
    assert torch.equal(Y, (z.clamp(min=0) + residual.double()).to(torch.float16))
    Y, Z = oz.linear(X, W, bias, "none", residual.float(), out_dtype=torch.float32, want_pre=True)
    assert torch.equal(Z, z.to(torch.float16))
    assert torch.equal(Y, (z + residual.double()).float())


@pytest.mark.parametrize("t,n,k", [(65, 70, 32768), (70, 130, 16384), (256, 128, 32768), (130, 100, 16385), (40, 200, 20000)])
def test_slices_of_k(t, n, k):
    # long and narrow: k cut into slices whose sums are joined
    X, W, bias, residual = operands(t, n, k, torch.bfloat16, 4)
    assert k % 8 or oz.ozaki2_linear_workspace_size(t, n, k) > 0
    check(oz.linear(X, W, bias, "gelu", residual.bfloat16(), want_pre=True), X, W, bias, "gelu", residual.bfloat16())


def test_runs_of_copied_weights():
    # rows that are no multiple of 16 bytes and more of them than one run copies
    t, n, k = 40, 5700, 20001
    X, W, bias, residual = operands(t, n, k, torch.bfloat16, 5)
    assert n > (96 << 20) // ((2 * k // 128 + 2) * 128)
    check(oz.linear(X, W, bias, "silu", residual.bfloat16(), want_pre=True), X, W, bias, "silu", residual.bfloat16())


@pytest.mark.parametrize("t,n,k", [(4, 60, 128), (20, 100, 256), (140, 300, 512), (600, 2100, 256)])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_rows_of_out_keep_their_gaps(t, n, k, out):
    X, W, bias, residual = operands(t, n, k, torch.float16, 6)
    wide = torch.full((t + 2, n + 3), 7.0, dtype=out, device="cuda")
    res = torch.zeros(t + 1, n + 5, dtype=out, device="cuda")
    res[1:, 2:n + 2] = residual
    got = oz.linear(X, W, bias, "silu", res[1:, 2:n + 2], out=wide[1:t + 1, 1:n + 1])
    assert got[0].data_ptr() == wide[1:, 1:].data_ptr()
    check(got, X, W, bias, "silu", residual.to(out))
    wide[1:t + 1, 1:n + 1] = 7.0
    assert (wide == 7.0).all()


def test_views():
    X, W, bias, residual = operands(40, 50, 256, torch.bfloat16, 7)
    residual = residual.bfloat16()
    want = oz.linear(X, W, bias, "gelu", residual)[0]
    assert torch.equal(oz.linear(X.t().contiguous().t(), W.t().contiguous().t(), bias, "gelu", residual)[0], want)
    assert torch.equal(oz.linear(X[::2], W, bias, "gelu", residual[::2])[0], want[::2])
    assert torch.equal(oz.linear(X, W, bias, "gelu", residual[:1].expand(40, -1))[0],
                       oz.linear(X, W, bias, "gelu", residual[:1].repeat(40, 1))[0])


def test_empty_sizes():
    X, W, bias, residual = operands(5, 7, 16, torch.bfloat16, 8)
    residual = residual.bfloat16()
    assert oz.linear(X[:0], W, bias)[0].shape == (0, 7)
    assert oz.linear(X, W[:0], bias[:0], "relu")[0].shape == (5, 0)
    Y, Z = oz.linear(X[:, :0], W[:, :0], bias, "relu", residual, want_pre=True)
    assert torch.equal(Z, bias.bfloat16().expand(5, 7))
    assert torch.equal(Y, (bias.clamp(min=0) + residual.float()).bfloat16())
    for t in (1, 100, 300):
        Y = oz.linear(torch.zeros(t, 0, device="cuda").half(), torch.zeros(300, 0, device="cuda").half())[0]
        assert Y.shape == (t, 300) and not Y.any()


def test_odd_values():
    # infinities and NaN of one token or one channel stay with it
    for t, n, k in ((3, 40, 64), (90, 80, 256), (300, 300, 128)):
        X, W, bias, residual = operands(t, n, k, torch.bfloat16, 9)
        X[1, 3] = float("nan")
        W[5, 7] = float("inf")
        for name in NAMES:
            Y = oz.linear(X, W, bias, name)[0]
            fine = torch.ones(t, n, dtype=torch.bool, device="cuda")
            fine[1] = fine[:, 5] = False
            assert torch.isfinite(Y[fine]).all()
            assert torch.isnan(Y[1]).all()
            assert not torch.isfinite(Y[:, 5][Y[:, 5] != 0]).any()
    # pre-activations far out: exactly 0 or z
    X = torch.tensor([[1e30], [-1e30], [300.0], [-300.0], [0.0]], device="cuda").bfloat16()
    W = torch.ones(40, 1, device="cuda").bfloat16()
    for name in NAMES[1:]:
        Y = oz.linear(X, W, None, name)[0]
        assert torch.equal(Y, X.clamp(min=0).expand(5, 40)), name


def test_refusals():
    X, W, bias, residual = operands(5, 7, 16, torch.bfloat16, 10)
    residual = residual.bfloat16()
    for bad in ((X.float(), W.float()), (X, W.half()), (X.cpu(), W)):
        with pytest.raises(TypeError):
            oz.linear(*bad)
    with pytest.raises(ValueError):
        oz.linear(X, W[:, :8])
    with pytest.raises(ValueError):
        oz.linear(X, W, activation="tanh")
    with pytest.raises(TypeError):
        oz.linear(X, W, out_dtype=torch.float16)
    for bad in (bias[:3], bias.bfloat16(), bias.cpu()):
        with pytest.raises(ValueError):
            oz.linear(X, W, bad)
    for bad in (residual[:3], residual.float(), residual.cpu()):
        with pytest.raises(ValueError):
            oz.linear(X, W, residual=bad)
    with pytest.raises(oz.Ozaki2Error):  # the residual in the output's place
        oz.linear(X, W, residual=residual, out=residual)
    with pytest.raises(ValueError):
        oz.linear_grad(residual, X, W, activation="silu")
    with pytest.raises(ValueError):
        oz.linear_grad(residual.half(), X, W)
    with pytest.raises(ValueError):
        oz.linear_grad(residual[:3], X, W)
    with pytest.raises(ValueError):
        oz.linear_grad(residual, X, W, Z=residual[:, :3], activation="silu")


# ---- gradients ---------------------------------------------------------------------
def check_grad(got, dY, X, W, Z, name):
    dX, dW, db = got
    dtype = X.dtype
    g = dY.double()
    if name != "none":
        z = Z.double()
        s = slope(name, z)
        # the slope's error, a product's rounding, then G's to its type for the two products
        dg = g.abs() * (slope_error(name, z) + U32 * s.abs())
        g = g * s
    else:
        dg = torch.zeros_like(g)
    t, n = g.shape
    if db is not None:
        close(db, g.sum(0), dg.sum(0) + t * 2 * U32 * (g.abs() + dg).sum(0) + TINY[torch.float32], "dbias")
    if name != "none":
        dg = dg + HALF[dtype] * (g.abs() + dg) + TINY[dtype]
    for out, a, da, b, terms, what in ((dX, g, dg, W.double(), n, "dX"), (dW, g.t().contiguous(), dg.t().contiguous(), X.double(), t, "dW")):
        if out is None:
            continue
        b = b.contiguous()
        tol = da @ b.abs() + terms * 2 * U32 * ((a.abs() + da) @ b.abs())
        want = a @ b
        close(out, want, rounded_to(dtype, want, tol), what)


def grad_operands(t, n, k, dtype, seed, pad=0):
    X, W, _, _ = operands(t, n, k, dtype, seed, pad)
    g = gen(seed + 1000)
    Z = (torch.randn(t, n + pad, generator=g, device="cuda") * 2).to(dtype)[:, pad:]
    dY = (torch.randn(t, n + pad, generator=g, device="cuda") * 0.1).to(dtype)[:, pad:]
    return X, W, Z, dY


GRADS = [(1, 1, 1), (1, 300, 512), (3, 17, 15), (16, 100, 304), (33, 129, 1000), (65, 66, 65), (128, 256, 256), (129, 264, 136),
         (200, 1030, 77), (257, 300, 400), (300, 511, 1023), (520, 520, 520), (1500, 64, 72), (2000, 130, 264), (7457, 28, 64),
         (5000, 8, 40), (4099, 1, 16), (3001, 513, 24)]


@pytest.mark.parametrize("t,n,k", GRADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients(t, n, k, dtype):
    X, W, Z, dY = grad_operands(t, n, k, dtype, t + n)
    name = NAMES[1 + (t + n) % 4]
    check_grad(oz.linear_grad(dY, X, W, Z, name), dY, X, W, Z, name)
    check_grad(oz.linear_grad(dY, X, W), dY, X, W, None, "none")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_gradients_of_views(name, pad):
    X, W, Z, dY = grad_operands(150, 200, 104, torch.bfloat16, 2, pad)
    check_grad(oz.linear_grad(dY, X, W, Z, name), dY, X, W, Z, name)
    check_grad(oz.linear_grad(dY[:1].expand(150, -1), X, W, Z, name), dY[:1].expand(150, -1), X, W, Z, name)


@pytest.mark.parametrize("tile", ["p4", "p8"])
def test_gradients_of_every_tile(tile, monkeypatch):
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    for t, n, k in ((60, 300, 256), (300, 520, 264), (1000, 256, 256)):
        X, W, Z, dY = grad_operands(t, n, k, torch.float16, 3)
        check_grad(oz.linear_grad(dY, X, W, Z, "gelu"), dY, X, W, Z, "gelu")


def test_each_gradient_alone():
    X, W, Z, dY = grad_operands(140, 200, 96, torch.bfloat16, 4)
    whole = oz.linear_grad(dY, X, W, Z, "silu")
    for i in range(3):
        want = [i == 0, i == 1, i == 2]
        got = oz.linear_grad(dY, X, W, Z, "silu", *want)
        for j in range(3):
            assert got[j] is None if j != i else torch.equal(got[j], whole[j])
    assert oz.linear_grad(dY, X, W, Z, "silu", False, False, False) == (None, None, None)


def test_gradients_of_empty_sizes():
    X, W, Z, dY = grad_operands(5, 7, 16, torch.bfloat16, 5)
    dX, dW, db = oz.linear_grad(dY[:0], X[:0], W, Z[:0], "relu")
    assert dX.shape == (0, 16) and dW.shape == (7, 16) and not dW.any() and db.shape == (7,) and not db.any()
    dX, dW, db = oz.linear_grad(dY[:, :0], X, W[:0], Z[:, :0], "relu")
    assert dX.shape == (5, 16) and not dX.any() and dW.shape == (0, 16) and db.shape == (0,)
    dX, dW, db = oz.linear_grad(dY, X[:, :0], W[:, :0], Z, "silu")
    assert dX.shape == (5, 0) and dW.shape == (7, 0)
    check_grad((None, None, db), dY, X, W, Z, "silu")


def test_slopes_at_the_ends():
    # Z that overflowed fp16, zeros, values far out: slopes of exactly 0 and 1, relu's 0 at 0
    z = torch.tensor([float("inf"), -float("inf"), 6e4, -6e4, 100.0, -100.0], device="cuda").half()
    Z = z[None, :].expand(4, 6).contiguous()
    dY = torch.ones(4, 6, device="cuda").half()
    X, W = torch.ones(4, 8, device="cuda").half(), torch.ones(6, 8, device="cuda").half()
    for name in NAMES[1:]:
        assert torch.equal(oz.linear_grad(dY, X, W, Z, name)[2].cpu(), torch.tensor([4.0, 0, 4, 0, 4, 0])), name
    zero = torch.zeros(4, 6, device="cuda").half()
    assert not oz.linear_grad(dY, X, W, zero, "relu")[2].any()
    assert torch.equal(oz.linear_grad(dY, X, W, zero, "silu")[2], torch.full((6,), 2.0, device="cuda"))


@pytest.mark.parametrize("name", NAMES[1:])
def test_gradients_against_differences(name):
    # d sum(dY * Y) along a direction, by central differences of the formula in 64 bits
    t, n, k = 40, 48, 32
    X, W, _, _ = operands(t, n, k, torch.bfloat16, 6)
    bias = torch.randn(n, generator=gen(7), device="cuda")
    dY = torch.randn(t, n, generator=gen(8), device="cuda").bfloat16()
    _, Z = oz.linear(X, W, bias, name, want_pre=True)
    dX, dW, db = oz.linear_grad(dY, X, W, Z, name)

    def loss(x, w, b):
        return (act(name, x @ w.t().contiguous() + b) * dY.double()).sum()

    x, w, b = X.double(), W.double(), bias.double()
    h = 1e-6
    for i, (grad, base) in enumerate(((dX, x), (dW, w), (db, b))):
        step = torch.randn(base.shape, generator=gen(9 + i), device="cuda", dtype=torch.float64)
        if name == "relu":  # keep away from the kink
            h = 1e-9
        up = [v + h * step if j == i else v for j, v in enumerate((x, w, b))]
        down = [v - h * step if j == i else v for j, v in enumerate((x, w, b))]
        slope_along = float((loss(*up) - loss(*down)) / (2 * h))
        got = float((grad.double() * step).sum())
        # Z and G are rounded to bf16, half a step of 2^-8 each: every term G of the sums is off by 2^-8 |G| and by
        # |act''| <= 1.2 times Z's 2^-8 |Z|; the gradient's own rounding is 2^-8 of it
        z = x @ w.t().contiguous() + b
        dg = dY.double().abs() * 2.0 ** -8 * (slope(name, z).abs() + (0 if name == "relu" else 1.2) * z.abs()) * 1.01
        terms = {0: dg @ w.abs(), 1: dg.t().contiguous() @ x.abs(), 2: dg.sum(0)}[i]
        # bf16 sums may flip the sign of a pre-activation next to 0 that relu cuts
        if name == "relu":
            flip = dY.double().abs() * (z.abs() < 1e-5)
            terms = terms + {0: flip @ w.abs(), 1: flip.t().contiguous() @ x.abs(), 2: flip.sum(0)}[i]
        tol = ((terms + 2.0 ** -8 * grad.double().abs()) * step.abs()).sum()
        assert abs(got - slope_along) <= float(tol) + 1e-4 * abs(slope_along), (i, got, slope_along, float(tol))


# ---- streams, graphs, sizes ------------------------------------------------------------
def test_streams_graphs_and_workspaces():
    t, n, k = 70, 130, 8192  # with slices
    X, W, bias, residual = operands(t, n, k, torch.bfloat16, 11)
    residual = residual.bfloat16()
    need = oz.ozaki2_linear_workspace_size(t, n, k)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    gws = torch.empty(oz.ozaki2_linear_grad_workspace_size(t, n, k), dtype=torch.uint8, device="cuda")

    def step():
        Y, Z = oz.linear(X, W, bias, "gelu", residual, want_pre=True, workspace=ws)
        return (Y, Z) + oz.linear_grad(Y, X, W, Z, "gelu", workspace=gws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (12, 13, 14):
        a, w, b, r = operands(t, n, k, torch.bfloat16, seed)
        X.copy_(a)
        W.copy_(w)
        bias.copy_(b)
        residual.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        again = [v.clone() for v in got]
        for x, y in zip(again, step()):
            assert torch.equal(x, y)
    # two streams at once, each with its workspace
    other = operands(t, n, k, torch.bfloat16, 15)
    ws2 = torch.empty_like(ws)
    want = oz.linear(X, W, bias, "gelu")[0], oz.linear(other[0], other[1], other[2], "silu")[0]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            got.append((oz.linear(X, W, bias, "gelu", workspace=ws)[0], want[0]))
        with torch.cuda.stream(streams[1]):
            got.append((oz.linear(other[0], other[1], other[2], "silu", workspace=ws2)[0], want[1]))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, y)


def test_cached_workspace():
    # the C forms without a workspace argument
    t, n, k = 70, 130, 8192
    X, W, _, _ = operands(t, n, k, torch.bfloat16, 16)
    Y, Z = oz.linear(X, W, None, "silu", want_pre=True)
    want = oz.linear_grad(Y, X, W, Z, "silu")
    y, z, dx, dw = torch.empty_like(Y), torch.empty_like(Z), torch.empty_like(X), torch.empty_like(W)
    s = torch.cuda.current_stream().cuda_stream
    p = [v.data_ptr() for v in (X, W, y, z, dx, dw)]
    assert oz.ozaki2_linear(t, n, k, p[0], k, p[1], k, oz.BF16, 0, 4, 0, 0, p[2], n, oz.BF16, p[3], n, s) == 0
    assert oz.ozaki2_linear_grad(t, n, k, p[2], n, p[0], k, p[1], k, oz.BF16, 4, p[3], n, p[4], k, p[5], k, 0, s) == 0
    for a, b in ((y, Y), (z, Z), (dx, want[0]), (dw, want[1])):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # outputs and inputs of more than 2^32 bytes
    t, n, k = 2200, 1 << 20, 16
    X, W, bias, _ = operands(t, n, k, torch.bfloat16, 17)
    Y, Z = oz.linear(X, W, bias, "relu", want_pre=True)
    rows = torch.tensor([0, 1, t // 2, t - 2, t - 1], device="cuda")
    check((Y[rows], Z[rows]), X[rows], W, bias, "relu", None)
    dX, dW, db = oz.linear_grad(Y, X, W, Z, "relu")
    dY = Y.double()
    dY = dY.mul_(Z > 0)
    cols = torch.tensor([0, 5, n // 2, n - 1], device="cuda")
    part = dY[:, cols].t().contiguous()
    want = part @ X.double()
    close(dW[cols], want, rounded_to(torch.bfloat16, want, t * 2 * U32 * (part.abs() @ X.double().abs())))
    want = dY[rows] @ W.double()
    close(dX[rows], want, rounded_to(torch.bfloat16, want, n * 2 * U32 * (dY[rows].abs() @ W.double().abs())))


def test_training_step_of_two_layers():
    # a layer with an activation and the loss of an output layer over it: the chain of gradients against 64-bit autograd
    t, d, m, v = 150, 64, 96, 500
    g = gen(18)
    X = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    W1 = (torch.randn(m, d, generator=g, device="cuda") / 8).bfloat16()
    b1 = torch.randn(m, generator=g, device="cuda") * 0.1
    W2 = (torch.randn(v, m, generator=g, device="cuda") / 5).bfloat16()
    y = torch.randint(v, (t,), generator=g, device="cuda")
    w = torch.full((t,), 1 / t, device="cuda")
    H, Z = oz.linear(X, W1, b1, "gelu", want_pre=True)
    loss, lse = oz.xent(H, W2, y)
    dH, dW2 = oz.xent_grad(H, W2, y, lse, w)
    dX, dW1, db1 = oz.linear_grad(dH, X, W1, Z, "gelu")
    leaves = [v.double().requires_grad_() for v in (X, W1, b1, W2)]
    x, w1, b, w2 = leaves
    z = act("gelu", x @ w1.t() + b) @ w2.t()
    ref = torch.nn.functional.cross_entropy(z, y, reduction="none")
    # H is off by half a step, 2^-8 relative, and so are its logits, in a random walk over m terms
    assert (loss.double() - ref.detach()).abs().max() < 0.05
    ref.mean().backward()
    # Z, H, dH and G are rounded to bf16 (2^-8 each, at most), and each result: below 5 half steps of its norm
    for got, want in zip((dX, dW1, db1, dW2), leaves):
        assert float((got.double() - want.grad).norm() / want.grad.norm()) < 5 * 2.0 ** -8
