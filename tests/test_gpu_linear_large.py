"""Sizes at which the large tiles (256 x 256) run with more tiles than compute units, so that a block goes on from one
tile to the next while its stores are on their way: INT8 products and losses, and the gradients of many tokens, against
64 bits. And a quantised layer as part of a chain.

Tolerances of the gradients, per entry, u = 2^-24, h half a step of the type at a binade's start (2^-8 bf16, 2^-11 fp16),
S = sum |x w|: z is off by at most d u S, so p by E = 2 (2 (d u S + 8 u max|z|) + 2^-15) of itself; G by h of itself, or
2^-39 max|g| in fp16; sums over n entries by n u of the sum of magnitudes; the result by h of itself, or half the
smallest step of fp16."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ABS = {torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -39}  # of G, times max|g|
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("t,n,k", [(5100, 5100, 256), (4999, 6007, 400)])
def test_int8_product_of_many_tiles(t, n, k):
    g = gen(k)
    A = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sa = torch.rand(t, generator=g, device="cuda") + 0.01
    sb = torch.rand(n, generator=g, device="cuda") * 0.1 + 0.001
    bias = torch.randn(n, generator=g, device="cuda") * 50
    r = (A.double() @ B.double().t().contiguous()) * sa.double()[:, None] * sb.double()
    want = r + bias.double()
    # |sum| <= 2^14 k is exact in binary32 up to k = 1024; two products and the sum with the bias round once each
    tol = 1.01 * U * (2 * r.abs() + want.abs())
    C = oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32)
    assert ((C.double() - want).abs() <= tol).all()
    for dtype in (torch.bfloat16, torch.float16):
        assert torch.equal(oz.i8gemm(A, B, sa, sb, bias, out_dtype=dtype), C.to(dtype))


def test_int8_loss_of_many_tiles():
    t = v = 5100
    k = 256
    g = gen(1)
    A = torch.randint(-127, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (v, k), generator=g, device="cuda", dtype=torch.int8)
    sa = (torch.rand(t, generator=g, device="cuda") + 0.1) * 2.0 ** -9
    sb = (torch.rand(v, generator=g, device="cuda") + 0.1) * 2.0 ** -7
    y = torch.randint(v, (t,), generator=g, device="cuda")
    y[::7] = -100
    loss, lse = oz.i8xent(A, B, sa, sb, y)
    z = (A.double() @ B.double().t().contiguous()) * sa.double()[:, None] * sb.double()
    want = torch.logsumexp(z, 1)
    # the scales' products and the exponential's argument are off by at most 8 u max|z|, the sum by 2^-15
    tol = 2.0 ** -15 + 8 * U * z.abs().amax(1)
    assert ((lse.double() - want).abs() <= tol).all()
    kept = y != -100
    at = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    assert ((loss.double() - (want - at)).abs() <= 2 * tol)[kept].all() and not loss[~kept].any()


@pytest.mark.parametrize("t,v,d,dtype", [
    (8192, 600, 4096, torch.bfloat16),    # dX in one piece
    (8192, 600, 4096, torch.float16),
    (8200, 33000, 4096, torch.bfloat16),  # in two, dW in large tiles too
    (8200, 33000, 4096, torch.float16),
    (1270, 20000, 1024, torch.bfloat16),  # a short k: the loss and G in large tiles, dX and dW in small ones
])
def test_gradients_of_many_tokens(t, v, d, dtype):
    g = gen(v)
    W = (torch.randn(v, d, generator=g, device="cuda") * (1.5 / d ** 0.5)).to(dtype)
    y = torch.randint(v, (t,), generator=g, device="cuda")
    X = (torch.randn(t, d, generator=g, device="cuda") + W[y].float() * 4 * torch.rand(t, 1, generator=g, device="cuda")).to(dtype)
    y[::9] = -100
    grad = torch.rand(t, generator=g, device="cuda") + 0.25
    loss, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    assert not dX[y == -100].any()
    weight = torch.where(y != -100, grad, torch.zeros_like(grad)).double()
    floor = ABS[dtype] * grad.max().double()

    def within(got, want, tol):
        return ((got.double() - want).abs() <= 1.01 * (tol + HALF[dtype] * want.abs() + TINY[dtype])).all()

    # some tokens: their loss and their rows of dX
    rows = torch.unique(torch.cat([torch.arange(0, t, t // 97), torch.tensor([255, 256, t - 257, t - 1])])).cuda()
    x, w = X[rows].double(), W.double()
    z = x @ w.t().contiguous()
    want = torch.logsumexp(z, 1)
    arg = d * U * (x.abs() @ w.abs().t().contiguous()).amax(1) + 8 * U * z.abs().amax(1)
    assert ((lse[rows].double() - want).abs() <= arg + 2.0 ** -15).all()
    kept = y[rows] != -100
    at = z.gather(1, y[rows].clamp(min=0)[:, None])[:, 0]
    assert ((loss[rows].double() - (want - at)).abs() <= 2 * (arg + 2.0 ** -15))[kept].all()
    p = torch.exp(z - want[:, None])
    G = p.clone()
    G[torch.arange(len(rows), device="cuda"), y[rows].clamp(min=0)] -= 1
    G, p = G * weight[rows][:, None], p * weight[rows][:, None]
    far = (HALF[dtype] + v * U) * G.abs() + 2 * (2 * arg + 2.0 ** -15)[:, None] * p + floor
    far[weight[rows] == 0] = 0
    assert within(dX[rows], G @ w, far @ w.abs())
    # some entries of the vocabulary: their rows of dW, from every token's loss
    cols = torch.unique(torch.cat([torch.arange(0, v, v // 53), torch.tensor([255, 256, v - 257, v - 1]), y[1:9].cpu()])).cuda()
    x, w = X.double(), W[cols].double()
    z = x @ w.t().contiguous()
    S = x.abs() @ W.double().abs().amax(0)  # at least any sum |x w|
    arg = d * U * S + 8 * U * lse.double().abs() + 8 * U * z.abs().amax(1)
    p = torch.exp(z - lse.double()[:, None])  # (lse itself has been compared above)
    G = (p - (cols[None, :] == y[:, None]).double()) * weight[:, None]
    far = (HALF[dtype] + t * U) * G.abs() + 2 * (2 * arg + 2.0 ** -15)[:, None] * p * weight[:, None] + floor
    assert within(dW[cols], G.t().contiguous() @ x, far.t().contiguous() @ x.abs())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantised_layer_of_a_chain(dtype):
    # the layer whose output an output layer takes: its values, from the quantised operands and the bias
    g = gen(4)
    X = torch.randn(200, 512, generator=g, device="cuda").to(dtype)
    q, s = oz.quantize_rows(torch.randn(768, 512, generator=g, device="cuda") / 512 ** 0.5)
    bias = torch.randn(768, generator=g, device="cuda")
    H = oz.i8linear(X, q, s, bias=bias)
    qx, sx = oz.quantize_rows(X)
    r = (qx.double() * sx.double()[:, None]) @ (q.double() * s.double()[:, None]).t().contiguous()
    want = r + bias.double()
    # the sum is exact (127^2 * 512 < 2^24); two products and the sum with the bias round to binary32, the result to its type
    tol = U * (2 * r.abs() + want.abs())
    if dtype != torch.float32:
        tol = tol + HALF[dtype] * (want.abs() + tol) + TINY[dtype]
    assert H.dtype == dtype and ((H.double() - want).abs() <= 1.01 * tol).all()
