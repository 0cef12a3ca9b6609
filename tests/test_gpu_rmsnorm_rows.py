"""The quantising norm (ozaki2_rmsnorm_quantize) where its blocks go on from row to row: more rows than blocks for every kernel that has more
than one row per block, each row different, with the sum over an input too, whose rows behind are already on their way then. Results are
compared bit for bit, as in test_gpu_rmsnorm."""
import pytest
import torch

import rns_emulated_fp64_amd as oz
from test_gpu_rmsnorm import TYPES, check, formula, inputs

pytestmark = pytest.mark.gpu

# 64 threads (8192 blocks), 256 threads of one and of two vectors (2048), 512 of two and of four (1024), rows longer than the registers
SIZES = [(9001, 130), (20011, 33), (17003, 512), (4500, 1000), (2500, 2048), (2500, 2049), (4500, 4096), (1100, 8191), (2300, 5000),
         (1100, 8200), (1300, 16384), (1100, 17001)]


@pytest.mark.parametrize("t,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_more_rows_than_blocks(t, k, dtype):
    X, weight, residual = inputs(t, k, dtype, t + k)
    want = formula(X, weight, residual, 1e-6)
    check(oz.rmsnorm_quantize(X, weight, residual), want)
    check(oz.rmsnorm_quantize(X), formula(X, None, None, 1e-6), False)
    over = residual.clone()
    check(oz.rmsnorm_quantize(X, weight, over, sum_out=over), want)
    assert torch.equal(over, want[2])
    over = X.clone()
    check(oz.rmsnorm_quantize(over, weight, residual, sum_out=over), want)
    assert torch.equal(over, want[2])


@pytest.mark.parametrize("t,k", [(9001, 130), (4500, 1000), (2500, 4096), (1100, 8191), (1100, 8200)])
def test_a_row_of_nan_leaves_the_others(t, k):
    X, weight, residual = inputs(t, k, torch.bfloat16, t)
    bad = torch.arange(t, device="cuda") % 3 == 1
    X[bad, k // 2] = float("nan")
    q, scale, _ = oz.rmsnorm_quantize(X, weight, residual)
    wq, ws, _ = formula(X[~bad], weight, residual[~bad], 1e-6)
    assert torch.equal(q[~bad], wq) and torch.equal(scale[~bad], ws)
    assert torch.isnan(scale[bad]).all() and not q[bad].any()
