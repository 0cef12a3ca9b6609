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
