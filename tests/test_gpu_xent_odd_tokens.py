"""Gradients of the linear cross entropy beside tokens and weights that are not numbers, or that have no place in the
loss: what is wrong with one token, or hidden from it, reaches no other."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu
BOTH = [torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(t, v, d, dtype, seed=0):
    g = gen(seed)
    W = (torch.randn(v, d, generator=g, device="cuda") * (1.5 / d ** 0.5)).to(dtype)
    X = torch.randn(t, d, generator=g, device="cuda").to(dtype)
    y = torch.randint(v, (t,), generator=g, device="cuda")
    return X, W, y


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("t", [20, 100, 600])
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan", "target"])
def test_a_token_that_is_not_a_number_leaves_the_others(t, bad, dtype):
    # results whose magnitudes fp16 holds, from weights of tokens that it does not
    X, W, y = operands(t, 500, 128, dtype, t)
    W = (W.float() * 2.0 ** -8).to(dtype)
    X = (X.float() * 2.0 ** 8).to(dtype)
    grad = 2.0 ** -6 * (1 + torch.rand(t, generator=gen(3), device="cuda")) * 2.0 ** (-torch.arange(t, device="cuda") % 9).float()
    _, lse = oz.xent(X, W, y)
    want = oz.xent_grad(X, W, y, lse, grad, want_dw=False)[0]
    at = torch.tensor([1, t - 1], device="cuda")  # (of no larger weight than others)
    if bad == "target":
        grad[at] = 2.0 ** 40
        y[at] = 500
    else:
        grad[at] = float(bad)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    rest = torch.ones(t, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert want[rest].isfinite().all() and (want[rest] != 0).float().mean() > 0.9
    assert torch.equal(dX[rest], want[rest])
    assert not dX[at].isfinite().any() and not dW.isfinite().any()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("t,v", [(6, 300), (100, 300), (300, 700), (600, 3000)])
def test_tokens_without_a_loss_beside_infinite_weights(t, v, dtype):
    # entries that a weight of -inf takes out of the vocabulary (their feature is 1 in every token): their rows of dW are 0
    # and their other features add nothing to dX, with ignored tokens and tokens of weight 0 beside the others
    X, W, y = operands(t, v, 64, dtype, t)
    X[:, 3] = 1
    keep = torch.ones(v, dtype=torch.bool, device="cuda")
    keep[5:v // 2] = False
    W[~keep, 3] = float("-inf")
    y %= 5
    grad = torch.rand(t, generator=gen(7), device="cuda") + 0.5
    y[::3] = -100
    grad[1::3] = 0
    _, lse = oz.xent(X, W, y)
    dX, dW = oz.xent_grad(X, W, y, lse, grad)
    assert not dW[~keep].any()
    assert dW[keep].isfinite().all()
    assert not dX[grad == 0][:, 4:].any() and not dX[y == -100][:, 4:].any()
    Wk = W[keep].contiguous()
    kX, kW = oz.xent_grad(X, Wk, y, oz.xent(X, Wk, y)[1], grad)
    # the same products from sums in another order: G and the sums agree to a step of the type, and so do the results
    # within two steps of each, relative to the magnitudes that they are sums of
    x, w, n = X.double(), Wk.double(), keep.sum()
    z = x @ w.t().contiguous()
    G = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    G[torch.arange(t, device="cuda"), y.clamp(min=0)] += 1
    G *= torch.where(y != -100, grad, torch.zeros_like(grad)).double()[:, None]
    step = torch.finfo(dtype).eps
    tol = 4 * step * (G @ w.abs()) + 2.0 ** -24
    cols = torch.arange(64, device="cuda") != 3
    assert ((dX.double() - kX.double()).abs() <= tol)[:, cols].all()
    tol = 4 * step * (G.t().contiguous() @ x.abs()) + 2.0 ** -24
    assert ((dW[keep].double() - kW.double()).abs() <= tol).all()
