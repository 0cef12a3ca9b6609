"""The quantising norm without a GPU: argument checks, which come before any HIP call."""
import rns_emulated_fp64_amd as oz

P = 1 << 20  # a pointer that is never followed


def test_refusals():
    #       t  k   X  ldx type     res ldr w  eps   Q  ldq scale sum lds
    good = (3, 16, P, 16, oz.FP16, P, 16, P, 1e-6, P, 16, P, P, 16)
    for i, bad in [(0, -1), (1, -1), (2, 0), (3, 15), (4, 3), (4, -1), (6, 15), (8, -1e-9), (8, float("nan")),
                   (8, float("inf")), (9, 0), (10, 15), (11, 0), (13, 15)]:
        assert oz.ozaki2_rmsnorm_quantize(*good[:i], bad, *good[i + 1:]) == -(i + 1), i
    assert oz.ozaki2_rmsnorm_quantize(1 << 31, *good[1:]) == 3
    k = 1 << 31
    assert oz.ozaki2_rmsnorm_quantize(3, k, P, k, oz.FP16, 0, 0, 0, 0.0, P, k, P, 0, 0) == 3
    # nothing to do; pitches of what is not there do not matter
    assert oz.ozaki2_rmsnorm_quantize(0, 16, 0, 16, oz.BF16, 0, 0, 0, 0.0, 0, 16, 0, 0, 0) == 0
