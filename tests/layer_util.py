"""Activations of the layers and their slopes in 64 bits, and how far the kernels' binary32 forms may be off."""
import math

import torch

U32 = 2.0 ** -24  # half a step of binary32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step relative to the value
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the subnormal step
NAMES = ["none", "relu", "gelu", "gelu_tanh", "silu"]
#: The factor of z in gelu and its slope: 1.5e-7 of its polynomial, and about a dozen roundings of values
#: below 1 in its series, reciprocal and exponential.
GELU = 4e-7


def act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if name in ("gelu_tanh", "silu"):
        f, df = (z, torch.ones_like(z)) if name == "silu" else (
            2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2))
        return torch.sigmoid(f) + z * df * torch.sigmoid(f) * torch.sigmoid(-f)
    return torch.ones_like(z)


def act_error(name, z, dz):
    """Bound on |computed act(z + e) - act(z)| for |e| <= dz. No slope exceeds 1.2. The sigmoid's argument x carries the
    roundings of its polynomial and of the product with log2(e), 4 half steps of |x| at most, and sigmoid(x) (1 - sigmoid(x)) |x| <
    0.23; exponential, sum and reciprocal add 3 steps of binary32, the product with z half a one."""
    if name == "none":
        return dz
    if name == "relu":
        return dz
    if name == "gelu":
        return 1.2 * dz + (GELU + U32) * z.abs()
    return 1.2 * dz + z.abs() * (4 * U32 * 0.23 * 3 + 7 * U32)


def slope_error(name, z):
    """Bound on the computed slope's error at z: as act_error's, for a sigmoid, its complement and their products (|z f' s (1 - s)| < 0.5)."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    if name == "gelu":
        return torch.full_like(z, 2 * GELU)
    return torch.full_like(z, 4 * U32 * 3 + 24 * U32)


def rounded_to(dtype, value, tol):
    """Tolerance of a value within tol, rounded to dtype."""
    return tol + HALF[dtype] * (value.abs() + tol) + TINY[dtype]
