"""Workspaces of INT8 products with and without what follows them, without a GPU.

A product without an activation or a residual needs room for its own slices of k alone; the forms with them take that room too, and
ask for more only to cut k further."""
import random

import pytest

import rns_emulated_fp64_amd as oz

P = 1 << 20  # a pointer that is never followed

# bytes that the plain forms need: (t, n, k, i8gemm, i8linear)
SIZES = [(37, 4096, 11008, 0, 412416),
         (24, 4096, 14336, 786432, 1133824),
         (64, 5120, 13824, 0, 893184),
         (48, 8192, 28672, 0, 1382656),
         (17, 1024, 65536, 557056, 1673728),
         (96, 1500, 9000, 14504448, 14504960),
         (128, 512, 65536, 1048576, 9454080),
         (200, 3000, 20000, 0, 4020224),
         (37, 4096, 11001, 46025216, 46025472),
         (26, 22441, 4391, 100038144, 100038400),
         (8, 4096, 4096, 0, 0),
         (1024, 4992, 20001, 119373824, 119377920)]


@pytest.mark.parametrize("t,n,k,gemm,linear", SIZES)
def test_plain_products_need_their_own_slices_alone(t, n, k, gemm, linear):
    assert oz.ozaki2_i8gemm_workspace_size(t, n, k) == gemm
    assert oz.ozaki2_i8linear_workspace_size(t, n, k) == linear
    if gemm:
        call = (t, n, k, P, k, P, P, k, P, 0, P, n, oz.BF16)
        assert oz.ozaki2_i8gemm_ws(*call, P, gemm - 1) == 2
        act = (t, n, k, P, k, P, P, k, P, 0, 1, 0, 0, P, n, oz.BF16)
        assert oz.ozaki2_i8gemm_act_ws(*act, P, gemm - 1) == 2
    if linear:
        act = (t, n, k, P, k, oz.BF16, P, k, P, 0, 1, 0, 0, P, n, oz.BF16)
        assert oz.ozaki2_i8linear_act_ws(*act, P, linear - 1) == 2


def test_room_for_more_slices_is_never_less():
    assert oz.ozaki2_i8gemm_act_workspace_size(37, 4096, 11008) > 0  # (a plain product of these sizes needs none)
    rng = random.Random(1)
    for _ in range(3000):
        t, n, k = (int(2 ** rng.uniform(0, most)) for most in (13, 16, 17))
        assert oz.ozaki2_i8gemm_act_workspace_size(t, n, k) >= oz.ozaki2_i8gemm_workspace_size(t, n, k), (t, n, k)
        assert oz.ozaki2_i8linear_act_workspace_size(t, n, k) >= oz.ozaki2_i8linear_workspace_size(t, n, k), (t, n, k)
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, -1), (5, 5, 1 << 17), (1 << 31, 5, 5)):
        assert oz.ozaki2_i8gemm_act_workspace_size(*bad) == oz.ozaki2_i8linear_act_workspace_size(*bad) == 0
