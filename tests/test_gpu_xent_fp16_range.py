"""Gradients of the linear cross entropy in fp16 (ozaki2_xent_grad) where the probabilities or the tokens' weights span
more than fp16 does, against 64 bits.

Tolerances, per entry, u = 2^-24, h = 2^-11 (half a step of fp16 at a binade's start), S = sum |x w|:
- z is a binary32 sum of d products in any order, off by at most d u S; with the roundings of the exponential's argument
  (up to 8 u max|z|) and of lse (2^-15 with its sum of exponentials) p is off by 2 (2 (d u S + 8 u max|z|) + 2^-15) of
  itself;
- G is rounded to fp16 relative to a power of two that is at least 2^-15 and at most 2^-14 of the largest |g|: half a
  step is h |G|, and below fp16's normal range 2^-25 of that power, at most 2^-39 max|g|;
- sums over n entries are off by n u of the sum of magnitudes, and the result by h of itself, or 2^-25 below fp16's
  normal range."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -11


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def confident(t, v, d, c, seed=0):
    """Tokens whose target stands out by c in logits beside which the others lie within a few units."""
    g = gen(seed)
    W = torch.randn(v, d, generator=g, device="cuda")
    W = (W / W.norm(dim=1, keepdim=True)).half()
    y = torch.randint(v // 2, (t,), generator=g, device="cuda")  # the upper half is nobody's target
    X = (c * W[y].float() + 1).half()
    return X, W, y


def check(X, W, y, grad):
    t, v, d = len(X), len(W), X.shape[1]
    _, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    x, w, g = X.double(), W.double(), grad.double()
    z = x @ w.t().contiguous()
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    G = p.clone()
    G[torch.arange(t, device="cuda"), y] -= 1
    G *= g[:, None]
    S = (x.abs() @ w.abs().t().contiguous()).amax(1)
    off = 2 * (2 * (d * U * S + 8 * U * z.abs().amax(1)) + 2.0 ** -15)
    far = (H + max(t, v) * U) * G.abs() + off[:, None] * p * g.abs()[:, None] + 2.0 ** -39 * g.abs().max()
    for got, want, tol, what in ((dX, G @ w, far @ w.abs(), "dX"),
                                 (dW, G.t().contiguous() @ x, far.t().contiguous() @ x.abs(), "dW")):
        tol = 1.01 * (tol + H * want.abs() + 2.0 ** -25)
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())
    return dX, dW


@pytest.mark.parametrize("c", [8, 16, 18, 20])
@pytest.mark.parametrize("t,grad", [(16, 4096.0), (96, 128.0), (300, 128.0)])
def test_confident_tokens_under_a_loss_scale(t, grad, c):
    X, W, y = confident(t, 3001, 128, c)
    _, dW = check(X, W, y, torch.full((t,), grad, device="cuda"))
    assert dW[1500:].any()


@pytest.mark.parametrize("t", [15, 64, 200])
def test_weights_of_tokens_over_many_binades(t):
    g = gen(t)
    W = (torch.randn(700, 96, generator=g, device="cuda") * (1.5 / 96 ** 0.5)).half()
    X = torch.randn(t, 96, generator=g, device="cuda").half()
    y = torch.randint(700, (t,), generator=g, device="cuda")
    grad = 2.0 ** (10 - torch.arange(t, device="cuda") % 15).float() * (1 + torch.rand(t, generator=g, device="cuda"))
    grad[::4] *= -1
    check(X, W, y, grad)


@pytest.mark.parametrize("t", [40, 130])
def test_small_weights_with_results_in_range(t):
    # g and G lie far below fp16's normal range, dW within it: X is large, and W as small as the logits ask for
    g = gen(t)
    W = (torch.randn(200, 64, generator=g, device="cuda") * (0.2 * 2.0 ** -10)).half()
    X = (torch.randn(t, 64, generator=g, device="cuda") * 2.0 ** 10).half()
    y = torch.randint(200, (t,), generator=g, device="cuda")
    grad = 2.0 ** -16 * (1 + torch.rand(t, generator=g, device="cuda"))
    _, dW = check(X, W, y, grad)
    assert (dW.abs() >= 2.0 ** -14).float().mean() > 0.5
    # the same in units of 2^-100 and 2^100: too small for fp16 altogether, and too large
    _, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad * 2.0 ** -100)
    assert not dX.any() and not dW.any()
    dX, dW = oz.xent_grad(X, W, y, lse, grad * 2.0 ** 100)
    assert torch.isinf(dX).float().mean() > 0.9 and torch.isinf(dW).float().mean() > 0.9
