"""The linear cross entropy (ozaki2_xent, ozaki2_i8xent) and its gradients (ozaki2_xent_grad) against 64 bits.

Tolerances. A logit is a binary32 sum of d products, in any order: off by at most
d u S, S = sum |x w|, u = 2^-24; the log of a sum of exponentials is off by no
more than its largest argument plus a few roundings of values up to
max|z| + log v, each u relative, and of the exponentials' sum (v additions of
positive terms in blocks of at most a few hundred in a row: 2^-15 is far above
256 u = 2^-16). So
    |lse - exact| <= d u S + 2^-15 + 8 u max|z|,   loss: twice that.
Gradients: G = g (p - [v = y]) has the error of its exponent's argument,
E = 2 (d u S + 8 u max|z|) + 2^-15, relative to p, and is rounded to 16 bits, half
a step h relative (2^-8 of bf16, 2^-11 of fp16 at a binade's start; fp16 adds
2^-25 of the largest |g| below its normal range). The products sum in binary32
and round once more. So per entry, with |.| taken entry by entry,
    |dX - exact| <= ((h + 2 E) |G| + (v u) |G| + c) |W| + h |dX| + tiny,
and the same for dW with |X|; c is fp16's absolute part. Numbers below the
smallest normal one of binary32, 2^-126, become zeros where they leave the
exponential and where they enter or leave the matrix cores (which is the hardware's
arithmetic, not a choice of the kernels), so with |g| <= 1 an entry of G may be off by
2^-126 twice, and an output by 2^-126: 2^-125 is added to c, 2^-126 to the whole."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
TILES = ("skinny", "s11", "s21", "s22", "s42", "p4", "p8", "any")
BOTH = [torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(t, v, d, dtype, seed=0, pad=0, skip=0.15):
    g = gen(seed)
    W = torch.zeros(v, d + pad, dtype=dtype, device="cuda")[:, :d]
    W.copy_(torch.randn(v, d, generator=g, device="cuda") * (1.5 / d ** 0.5))
    y = torch.randint(v, (t,), generator=g, device="cuda")
    X = torch.zeros(t, d + pad, dtype=dtype, device="cuda")[:, :d]
    X.copy_(torch.randn(t, d, generator=g, device="cuda") + W[y].float() * 5 * torch.rand(t, 1, generator=g, device="cuda"))
    y[torch.rand(t, generator=g, device="cuda") < skip] = -100
    grad = (torch.rand(t, generator=g, device="cuda") - 0.3) / t
    return X, W, y, grad


def exact(X, W, y, grad, sx=None, sw=None):
    """Loss, lse, dX, dW and the bounds that the docstring derives, in 64 bits on the CPU."""
    x, w = X.double().cpu(), W.double().cpu()
    if sx is not None:
        x, w = x * sx.double().cpu()[:, None], w * sw.double().cpu()[:, None]
    y, n, d = y.cpu(), len(x), x.shape[1]
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    kept = y != -100
    at = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(kept, lse - at, torch.zeros_like(lse))
    S = (x.abs() @ w.abs().t()).amax(1)
    arg = d * U * S + 8 * U * z.abs().amax(1)
    tol = arg + 2.0 ** -15
    out = {"loss": loss, "lse": lse, "tol": tol}
    if grad is not None:
        g = torch.where(kept, grad.double().cpu(), torch.zeros(n, dtype=torch.float64))
        p = torch.exp(z - lse[:, None])
        G = p.clone()
        G[torch.arange(n), y.clamp(min=0)] -= 1
        G, p = G * g[:, None], p * g.abs()[:, None]
        h, v = STEP[X.dtype], len(w)
        far = 2.0 ** -125 + h * G.abs() + 2 * (2 * arg + 2.0 ** -15)[:, None] * p + max(v, n) * U * G.abs()
        if X.dtype == torch.float16:
            far = far + 2.0 ** -25 * float(g.abs().max())
            far[g == 0] = 0
        dX, dW = G @ w, G.t() @ x
        out["dX"], out["dX_tol"] = dX, far @ w.abs() + h * dX.abs() + TINY[X.dtype]
        out["dW"], out["dW_tol"] = dW, far.t() @ x.abs() + h * dW.abs() + TINY[X.dtype]
    return out


def near(got, want, tol, what):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol * 1.01)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(off.max()))


def check(X, W, y, grad, e=None):
    e = e or exact(X, W, y, grad)
    loss, lse = oz.xent(X, W, y)
    near(lse, e["lse"], e["tol"], "lse")
    near(loss, e["loss"], 2 * e["tol"], "loss")
    assert (loss[y == -100] == 0).all()
    if grad is not None:
        dX, dW = oz.xent_grad(X, W, y, lse, grad)
        assert dX.dtype == dW.dtype == X.dtype
        near(dX, e["dX"], e["dX_tol"], "dX")
        near(dW, e["dW"], e["dW_tol"], "dW")
        assert not dX[y == -100].any()
        only_x = oz.xent_grad(X, W, y, lse, grad, want_dw=False)
        only_w = oz.xent_grad(X, W, y, lse, grad, want_dx=False)
        assert only_x[1] is None and only_w[0] is None
        assert torch.equal(only_x[0], dX) and torch.equal(only_w[1], dW)
    return loss, lse


SHAPES = [(1, 1, 1), (1, 2, 3), (1, 17, 8), (2, 100, 64), (5, 33, 130), (16, 1000, 100), (17, 333, 129), (40, 5000, 77),
          (64, 2000, 256), (65, 130, 64), (100, 1000, 128), (130, 257, 1024), (129, 4097, 136), (300, 3001, 200),
          (520, 1037, 512), (610, 3501, 128)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("t,v,d", SHAPES)
def test_loss_and_gradients(t, v, d, dtype):
    check(*operands(t, v, d, dtype, t + v + d))


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("t,v,d,pad", [(7, 300, 256, 0), (50, 700, 264, 8), (300, 600, 136, 8), (270, 1030, 256, 0),
                                       (70, 90, 131, 0)])
def test_every_tile(tile, t, v, d, pad, monkeypatch):
    X, W, y, grad = operands(t, v, d, torch.bfloat16, 3, pad)
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    check(X, W, y, grad)
    A, sa = oz.quantize_rows(X)
    B, sb = oz.quantize_rows(W)
    e = exact(A, B, y, None, sa, sb)
    loss, lse = oz.i8xent(A, B, sa, sb, y)
    near(lse, e["lse"], e["tol"], "lse")
    near(loss, e["loss"], 2 * e["tol"], "loss")


@pytest.mark.parametrize("t,v,k", [(1, 1, 1), (1, 999, 64), (12, 5001, 300), (33, 100, 1000), (70, 2000, 256),
                                   (300, 4097, 512), (520, 1037, 131)])
def test_int8_loss(t, v, k):
    X, W, y, _ = operands(t, v, k, torch.float16, t)
    A, sa = oz.quantize_rows(X)
    B, sb = oz.quantize_rows(W)
    e = exact(A, B, y, None, sa, sb)
    loss, lse = oz.i8xent(A, B, sa, sb, y)
    near(lse, e["lse"], e["tol"], "lse")
    near(loss, e["loss"], 2 * e["tol"], "loss")
    sa[::2] *= -1  # scales of either sign
    sb[::3] *= -1
    e = exact(A, B, y, None, sa, sb)
    loss, lse = oz.i8xent(A, B, sa, sb, y)
    near(lse, e["lse"], e["tol"], "lse")
    near(loss, e["loss"], 2 * e["tol"], "loss")


@pytest.mark.parametrize("tile", ("",) + TILES)
@pytest.mark.parametrize("t,v", [(3, 37), (40, 300), (300, 557), (300, 700)])
def test_int8_rows_of_scale_zero(t, v, tile, monkeypatch):
    # a row of zeros is quantised with scale 0 (and -0 is one too): its logits are all 0, so its loss is log v,
    # beside tiles that reach past the vocabulary's end
    X, W, y, _ = operands(t, v, 64, torch.bfloat16, t, skip=0)
    X[::2] = 0
    A, sa = oz.quantize_rows(X)
    B, sb = oz.quantize_rows(W)
    A[2::4] = 1  # values that the scale alone takes away
    sa[2::4] = -0.0
    e = exact(A, B, y, None, sa, sb)
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    loss, lse = oz.i8xent(A, B, sa, sb, y)
    near(lse, e["lse"], e["tol"], "lse")
    near(loss, e["loss"], 2 * e["tol"], "loss")


def test_loss_chain_of_quantised_layers():
    # as they are used together: a quantised layer, then the loss of an output layer and its gradients, and the
    # quantised form of that layer
    g = gen(4)
    X = torch.randn(200, 512, generator=g, device="cuda").bfloat16()
    q, s = oz.quantize_rows(torch.randn(768, 512, generator=g, device="cuda") / 512 ** 0.5)
    H = oz.i8linear(X, q, s, bias=torch.randn(768, generator=g, device="cuda"))
    qx, sx = oz.quantize_rows(X)
    ref = (qx.double() * sx.double()[:, None]) @ (q.double() * s.double()[:, None]).t().contiguous()
    W = (torch.randn(3000, 768, generator=g, device="cuda") / 768 ** 0.5).bfloat16()
    y = torch.randint(3000, (200,), generator=g, device="cuda")
    grad = torch.full((200,), 1 / 200, device="cuda")
    loss, _ = check(H, W, y, grad)
    A, sa = oz.quantize_rows(H)
    B, sb = oz.quantize_rows(W)
    quant, _ = oz.i8xent(A, B, sa, sb, y)
    # an int8 value is within half a step of what it stands for, so a logit moves by at most
    # sum (|h| sb / 2 + |w| sa / 2 + sa sb / 4)
    h, w = H.double().abs(), W.double().abs()
    most = h.sum(1)[:, None] * sb.double() / 2 + w.sum(1) * sa.double()[:, None] / 2 + 768 * sa.double()[:, None] * sb.double() / 4
    assert ((quant - loss).abs() <= 2 * most.amax(1) + 1e-3).all()
    assert ref.shape == H.shape


@pytest.mark.parametrize("dtype", BOTH)
def test_gradient_against_differences(dtype):
    # the loss at X +- step along a direction, in 64 bits, against dX; W likewise
    X, W, y, grad = operands(6, 50, 16, dtype, 8)
    _, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    g = gen(1)

    def total(x, w):
        z = x @ w.t().contiguous()
        loss = torch.logsumexp(z, 1) - z.gather(1, y.clamp(min=0)[:, None])[:, 0]
        return (loss * grad.double())[y != -100].sum()

    x, w = X.double(), W.double()
    for _ in range(4):
        u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        m = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        fx = (total(x + step * u, w) - total(x - step * u, w)) / (2 * step)
        fw = (total(x, w + step * m) - total(x, w - step * m)) / (2 * step)
        # each entry of the gradient within 2 steps of its type, relative to the largest
        assert abs(fx - (dX.double() * u).sum()) <= 4 * STEP[dtype] * (dX.double().abs().max() * u.abs().sum())
        assert abs(fw - (dW.double() * m).sum()) <= 4 * STEP[dtype] * (dW.double().abs().max() * m.abs().sum())


@pytest.mark.parametrize("t", [3, 64, 200])
def test_tokens_without_a_target(t):
    X, W, y, grad = operands(t, 500, 128, torch.bfloat16, 5)
    y[0], y[1], y[2] = -100, -100, 7
    loss, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    # what an ignored row holds is nobody's business: its loss is 0 and it adds nothing to dW
    X[0], X[1] = float("nan"), float("inf")
    loss2, lse2 = oz.xent(X, W, y)
    assert torch.equal(loss2, loss) and torch.equal(lse2[2:], lse[2:])
    again = oz.xent_grad(X, W, y, lse2, grad)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
    # nor what a row holds whose loss has no gradient
    grad[2] = 0
    base = oz.xent_grad(X, W, y, lse2, grad)
    X[2] = float("nan")
    again = oz.xent_grad(X, W, y, oz.xent(X, W, y)[1], grad)
    assert torch.equal(again[0], base[0]) and torch.equal(again[1], base[1]) and not again[0][2].any()
    # all of them ignored
    y[:] = -100
    loss, lse = oz.xent(X, W, y)
    assert not loss.any()
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    assert not dX.any() and not dW.any()
    # another ignored index, which may be one of the vocabulary
    X, W, y, grad = operands(t, 500, 128, torch.bfloat16, 5, skip=0)
    y[::2] = 3
    loss, _ = oz.xent(X, W, y, ignore_index=3)
    want, _ = oz.xent(X, W, y)
    assert (loss[::2] == 0).all() and torch.equal(loss[y != 3], want[y != 3])


@pytest.mark.parametrize("t", [2, 90])
def test_targets_out_of_range(t):
    X, W, y, grad = operands(t, 500, 128, torch.float16, 6, skip=0)
    want, lse0 = oz.xent(X, W, y)
    for bad in (500, -1, 2 ** 40, -2 ** 63):
        y2 = y.clone()
        y2[0] = bad
        loss, lse = oz.xent(X, W, y2)
        assert torch.isnan(loss[0]) and torch.equal(loss[1:], want[1:]) and torch.equal(lse, lse0)
        dX, dW = oz.xent_grad(X, W, y2, lse, grad)
        assert torch.isnan(dX[0]).all() and not torch.isnan(dX[1:]).any()
        A, sa = oz.quantize_rows(X)
        B, sb = oz.quantize_rows(W)
        assert torch.isnan(oz.i8xent(A, B, sa, sb, y2)[0][0])


def test_extreme_logits():
    # spreads that overflow exp on their own, equal logits, a vocabulary of one
    for scale in (0.0, 30.0, 300.0):
        X, W, y, grad = operands(70, 300, 64, torch.bfloat16, 7)
        X = (X.float() * scale).bfloat16()
        check(X, W, y, grad)
    X, W, y, grad = operands(9, 1, 64, torch.bfloat16, 7, skip=0)
    loss, lse = oz.xent(X, W, y)
    assert (loss.abs() <= 1e-5).all()


def test_infinite_logits():
    # entries at -inf take no part; a row of nothing else has lse -inf; +inf or NaN gives NaN
    for t in (4, 70):
        X = torch.ones(t, 16, dtype=torch.bfloat16, device="cuda")
        W = torch.randn(300, 16, generator=gen(2), device="cuda").bfloat16()
        W[5:200, 3] = float("-inf")
        y = torch.zeros(t, dtype=torch.int64, device="cuda")
        keep = torch.cat([torch.arange(5), torch.arange(200, 300)]).cuda()
        loss, lse = oz.xent(X, W, y)
        want, wlse = oz.xent(X, W[keep].contiguous(), y)
        assert (lse - wlse).abs().max() <= 2.0 ** -15 and (loss - want).abs().max() <= 2.0 ** -14
        W[:, 3] = float("-inf")
        assert (oz.xent(X, W, y)[1] == float("-inf")).all()
        W[:, 3] = 0
        W[17, 3] = float("nan")
        assert torch.isnan(oz.xent(X, W, y)[1]).all()


def test_fp16_small_gradients():
    # a mean over many tokens: g far below fp16's range, results within it
    X, W, y, _ = operands(300, 700, 128, torch.float16, 9, skip=0)
    grad = torch.full((300,), 2.0 ** -40, device="cuda")
    _, lse = oz.xent(X, W, y)
    big = oz.xent_grad(X, W, y, lse, torch.ones(300, device="cuda"))
    X32 = (X.float() * 1.0)
    assert X32.isfinite().all()
    small = oz.xent_grad(X, W, y, lse, grad)
    for a, b in zip(small, big):
        # the same sums, scaled by a power of two and rounded into fp16's subnormals
        assert torch.equal(a, (b.double() * 2.0 ** -40).half()) or ((a.double() - b.double() * 2.0 ** -40).abs() <= 2.0 ** -25).all()
    grad = torch.full((300,), 1e-3, device="cuda")
    e = exact(X, W, y, grad)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    near(dX, e["dX"], e["dX_tol"], "dX")
    near(dW, e["dW"], e["dW_tol"], "dW")


@pytest.mark.parametrize("dtype", BOTH)
def test_shared_and_strided_rows(dtype):
    X, W, y, grad = operands(40, 600, 192, dtype, 10, pad=24)
    e = exact(X, W, y, grad)
    check(X, W, y, grad, e)
    check(X.contiguous(), W.t().contiguous().t(), y, grad, e)
    # the same row for every token, and the same target
    one = X[:1].expand(40, -1)
    y = torch.full((40,), 5, dtype=torch.int64, device="cuda")
    check(one, W, y, grad)
    check(X[::2], W[::3], y[::2] % 200, grad[::2])


def test_pieces_of_the_vocabulary():
    # more tokens and entries than one piece of G holds: dX is summed over pieces
    t, v, d = 20000, 30000, 64
    assert t * v > 2 ** 28
    X, W, y, grad = operands(t, v, d, torch.bfloat16, 12)
    loss, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    rows = torch.cat([torch.arange(0, t, 997), torch.tensor([16383, 16384, t - 1])]).cuda()
    e = exact(X[rows], W, y[rows], grad[rows])
    near(lse[rows], e["lse"], e["tol"], "lse")
    near(loss[rows], e["loss"], 2 * e["tol"], "loss")
    near(dX[rows], e["dX"], e["dX_tol"], "dX")
    # columns of G for some entries, in 64 bits
    for at in (0, 12345, 13312, v - 1):
        z = X.double() @ W[at].double()
        G = torch.exp(z - lse.double()) - (y == at).double()
        G *= torch.where(y != -100, grad, torch.zeros_like(grad)).double()
        want = G @ X.double()
        tol = (2.0 ** -8 + 2.0 ** -13 + t * U) * (G.abs() @ X.double().abs()) + 2.0 ** -8 * want.abs()
        assert ((dW[at].double() - want).abs() <= tol).all()


def test_pieces_of_rows_that_are_copied():
    # rows of W that are not aligned, more than one copy holds
    t, v, d = 6, 33000, 4104
    X, W, y, grad = operands(t, v, d, torch.bfloat16, 16, pad=1)
    size = oz.ozaki2_xent_grad_workspace_size(t, v, d)
    assert 1 << 28 < size < 3 << 27
    check(X, W, y, grad)


@pytest.mark.parametrize("t", [3, 40, 300])
def test_weights_past_32_bits(t):
    # more than 2^32 bytes of W and of dW; 64 bits a slab at a time, with the docstring's bounds
    v, d = 540000, 4096
    W = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    g = gen(17)
    for at in range(0, v, 60000):
        W[at:at + 60000] = torch.randn(60000, d, generator=g, device="cuda") * (1.5 / d ** 0.5)
    X = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    y = torch.randint(v, (t,), generator=g, device="cuda")
    y[0] = v - 1
    grad = torch.rand(t, generator=g, device="cuda") / t
    loss, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    x = X.double()
    zs = [x @ W[at:at + 60000].double().t().contiguous() for at in range(0, v, 60000)]
    most = max(z.abs().max().item() for z in zs)
    sums = (x.abs().sum(1) * W.abs().max().double()).max().item()  # at least sum |x w|
    want = torch.logsumexp(torch.stack([torch.logsumexp(z, 1) for z in zs]), 0)
    tol = d * U * sums + 2.0 ** -15 + 8 * U * most
    assert ((lse.double() - want).abs() <= tol).all()
    E, h = 2 * (d * U * sums + 8 * U * most) + 2.0 ** -15, STEP[torch.bfloat16]
    sx, sx_abs = torch.zeros_like(x), torch.zeros_like(x)
    for i, z in enumerate(zs):
        slab = W[i * 60000:(i + 1) * 60000].double()
        G = torch.exp(z - want[:, None])
        mine = (y >= i * 60000) & (y < (i + 1) * 60000)
        G[mine, y[mine] - i * 60000] -= 1
        G *= grad.double()[:, None]
        P = G.abs() + (G + grad.double()[:, None] * (G < 0)).abs()  # |G| and the probability's own part of the target's
        sx += G @ slab
        sx_abs += P @ slab.abs()
        got = dW[i * 60000:(i + 1) * 60000].double()
        ref = G.t().contiguous() @ x
        bound = (h + 2 * E + t * U) * (P.t().contiguous() @ x.abs()) + h * ref.abs() + 2.0 ** -126
        assert ((got - ref).abs() <= bound).all(), i
    assert ((dX.double() - sx).abs() <= (h + 2 * E + v * U) * sx_abs + h * sx.abs() + 2.0 ** -126).all()


def test_streams_and_graph():
    X, W, y, grad = operands(80, 3001, 256, torch.bfloat16, 13)
    A, sa = oz.quantize_rows(X)
    B, sb = oz.quantize_rows(W)

    def step():
        loss, lse = oz.xent(X, W, y)
        return [loss, lse, *oz.xent_grad(X, W, y, lse, grad), *oz.i8xent(A, B, sa, sb, y)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        X.copy_(torch.randn(X.shape, generator=gen(r), device="cuda"))
        y.copy_(torch.randint(3001, y.shape, generator=gen(r), device="cuda"))
        A.copy_(torch.randint(-127, 128, A.shape, generator=gen(r), device="cuda", dtype=torch.int8))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r


def test_cached_workspace_form():
    X, W, y, grad = operands(80, 3001, 256, torch.bfloat16, 14)
    A, sa = oz.quantize_rows(X)
    B, sb = oz.quantize_rows(W)
    loss, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    qloss, qlse = oz.i8xent(A, B, sa, sb, y)
    n = lambda x: torch.zeros_like(x)  # noqa: E731
    a = [n(loss), n(lse), n(dX), n(dW), n(qloss), n(qlse)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    p = [x.data_ptr() for x in a]
    assert oz.ozaki2_xent(80, 3001, 256, X.data_ptr(), 256, W.data_ptr(), 256, oz.BF16, y.data_ptr(), -100, p[0], p[1],
                          s[0].cuda_stream) == 0
    assert oz.ozaki2_i8xent(80, 3001, 256, A.data_ptr(), 256, sa.data_ptr(), B.data_ptr(), 256, sb.data_ptr(),
                            y.data_ptr(), -100, p[4], p[5], s[1].cuda_stream) == 0
    assert oz.ozaki2_xent_grad(80, 3001, 256, X.data_ptr(), 256, W.data_ptr(), 256, oz.BF16, y.data_ptr(), -100,
                               lse.data_ptr(), grad.data_ptr(), p[2], 256, p[3], 256, s[0].cuda_stream) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in zip(a, [loss, lse, dX, dW, qloss, qlse]))


def test_no_tokens_and_pitched_outputs():
    X, W, y, grad = operands(5, 300, 64, torch.bfloat16, 15)
    loss, lse = oz.xent(X[:0], W, y[:0])
    assert loss.shape == lse.shape == (0,)
    dX, dW = oz.xent_grad(X[:0], W, y[:0], lse, grad[:0])
    assert dX.shape == (0, 64) and not dW.any()
    # no features: every logit is 0
    loss, lse = oz.xent(X[:, :0], W[:, :0], y)
    assert (lse - torch.log(torch.tensor(300.0))).abs().max() <= 2.0 ** -20
    # pitched outputs keep their gaps
    _, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    wx = torch.full((7, 70), 3.0, dtype=torch.bfloat16, device="cuda")
    ww = torch.full((302, 67), 3.0, dtype=torch.bfloat16, device="cuda")
    px, pw = wx[1:6, 2:66], ww[1:301, 1:65]
    size = oz.ozaki2_xent_grad_workspace_size(5, 300, 64)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    st = oz.ozaki2_xent_grad_ws(5, 300, 64, X.data_ptr(), 64, W.data_ptr(), 64, oz.BF16, y.data_ptr(), -100,
                                lse.data_ptr(), grad.data_ptr(), px.data_ptr(), 70, pw.data_ptr(), 67, ws.data_ptr(),
                                size, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(px, dX) and torch.equal(pw, dW)
    px[:], pw[:] = 3.0, 3.0
    assert (wx == 3.0).all() and (ww == 3.0).all()


def test_python_refusals():
    X, W, y, grad = operands(5, 30, 16, torch.bfloat16, 1)
    lse = torch.zeros(5, device="cuda")
    for bad in ((X.float(), W.float(), y), (X, W.half(), y), (X.cpu(), W, y), (X, W, y.int())):
        with pytest.raises(TypeError):
            oz.xent(*bad)
    for bad in ((X, W[:, :8], y), (X, W, y[:3]), (X[0], W, y), (X, W[:0], y), (X, W, y[:, None])):
        with pytest.raises(ValueError):
            oz.xent(*bad)
    with pytest.raises(ValueError):
        oz.xent_grad(X, W, y, lse.double(), grad)
    with pytest.raises(ValueError):
        oz.xent_grad(X, W, y, lse[:4], grad)
    with pytest.raises(TypeError):
        oz.i8xent(X, W, lse, lse, y)
    with pytest.raises(oz.Ozaki2Error) as e:
        oz.xent(X, W, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 2
