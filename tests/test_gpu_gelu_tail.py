"""gelu and its slope relative to themselves, out to where they leave binary32: of values whose sums are exact (a bias alone).

gelu(z) = z Phi(z). In 32-bit results the kernel's Phi(-|z|) is off by at most 1e-6 of itself down to z = -13: the polynomial by 9e-8, its
eight roundings, of terms whose magnitudes add up to 1.3 times it, by 2.4e-7 at most, the reciprocal and its argument (with a
rounded constant) by 2.1e-7, times at most 1, since erfcx changes by less than its argument does, exponential 1.2e-7, what is put back into it
1.2e-7, products 1.2e-7. In 16-bit results the polynomial is off by 3e-5 and the exponential's argument, up to 122, by two half
steps and its constant's 1.4e-8: 122 ln 2 (1.2e-7 + 1.4e-8) = 1.14e-5; with the rest above 4.3e-5."""
import math

import pytest
import torch

import rns_emulated_fp64_amd as oz
from layer_util import HALF, TINY

pytestmark = pytest.mark.gpu

FINE, COARSE = 1e-6, 4.3e-5


def gelu(z):
    return z * torch.exp(torch.special.log_ndtr(z))


def bounds(want, dtype):
    """Of a result in `dtype`: the value's error and its rounding. (Phi(z) above 0 is 1 - Phi(-z), each off by less.)"""
    error = FINE if dtype == torch.float32 else COARSE
    return want.abs() * (error + 2.0 ** -24 + HALF[dtype] * (1 + 1e-3)) + TINY[dtype] + 2.0 ** -126 * 14


@pytest.mark.parametrize("t", [1, 20, 70, 300, 1100])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_gelu(t, out):
    z = torch.linspace(-13, 6, 2309, device="cuda")
    k = 64 if t < 1000 else 256
    dtype = torch.float16 if out == torch.float32 else out
    X, W = torch.zeros(t, k, dtype=dtype, device="cuda"), torch.zeros(len(z), k, dtype=dtype, device="cuda")
    want = gelu(z.double())
    Y = oz.linear(X, W, z, "gelu", out_dtype=out)[0]
    bad = ~((Y.double() - want).abs() <= bounds(want, out))
    assert not bad.any(), (z[bad.any(0)][:3], Y[:, bad.any(0)][0, :3], want[bad.any(0)][:3])
    # the same from int8 operands
    one = torch.ones(max(t, len(z)), device="cuda")
    C = oz.i8gemm(X.to(torch.int8), W.to(torch.int8), one[:t], one[:len(z)], z, out_dtype=out, activation="gelu")
    assert torch.equal(C, Y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_far_out(dtype):
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 40.0, -40.0, 1e19, -1e19, 3e38, -3e38, math.inf, float("nan")], device="cuda")
    X, W = torch.zeros(3, 8, dtype=dtype, device="cuda"), torch.zeros(len(z), 8, dtype=dtype, device="cuda")
    Y = oz.linear(X, W, z, "gelu", out_dtype=torch.float32)[0]
    want = torch.tensor([0.0, 0.0, 5e-31, -5e-31, 40.0, 0.0, 1e19, 0.0, 3e38, 0.0, math.inf], device="cuda")
    assert torch.allclose(Y[:, :-1], want.expand(3, -1), rtol=1e-6, atol=0) and torch.isnan(Y[:, -1]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_slope(dtype):
    # Phi(z) + z phi(z): the first off as in 16-bit results (and above 0, where it is 1 - Phi(-z), by a rounding of 1), the second by the
    # exponential and its argument, and three roundings of values below both
    z = torch.linspace(-12, 6, 2309, device="cuda").to(dtype)
    W = torch.zeros(len(z), 8, dtype=dtype, device="cuda")
    one = torch.ones(1, len(z), dtype=dtype, device="cuda")
    got = oz.linear_grad(one, W[:1], W, z[None, :], "gelu", False, False, True)[2].double()
    z = z.double()
    below, bell = torch.exp(torch.special.log_ndtr(z)), z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    bad = ~((got - below - bell).abs() <= below * COARSE + bell.abs() * 1.2e-5 + (below + bell.abs()) * 3 * 2.0 ** -24 + 2.0 ** -126 * 14)
    assert not bad.any(), (z[bad][:3], got[bad][:3], (below + bell)[bad][:3])
