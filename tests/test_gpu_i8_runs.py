"""INT8 products whose rows are copied to aligned ones in more than one run of channels, the last one short and cut into
slices of k: exact results, and no byte written past the workspace that is asked for."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

# with scales of 1 the binary32 result is the integer sum itself, exact below 2^24 (here 400 * 8193)
SIZES = [(256, 12100, 8193), (26, 22441, 4391)]


def operands(t, n, k):
    g = torch.Generator(device="cuda").manual_seed(k)
    A = torch.randint(-20, 21, (t, k), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-20, 21, (n, k), generator=g, device="cuda", dtype=torch.int8)
    return A, B, torch.ones(t, device="cuda"), torch.ones(n, device="cuda")


def guarded(size, guard=1 << 20):
    return torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("t,n,k", SIZES)
def test_product_in_runs_stays_in_its_workspace(t, n, k):
    A, B, sa, sb = operands(t, n, k)
    size = oz.ozaki2_i8gemm_workspace_size(t, n, k)
    ws, C = guarded(size), torch.empty(t, n, device="cuda")
    st = oz.ozaki2_i8gemm_ws(t, n, k, A.data_ptr(), k, sa.data_ptr(), B.data_ptr(), k, sb.data_ptr(), None, C.data_ptr(),
                             n, oz.FP32, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(C.double(), A.double() @ B.double().t().contiguous())
    assert (ws[size:] == 0x5A).all()


@pytest.mark.parametrize("t,n,k", SIZES)
def test_layer_in_runs_stays_in_its_workspace(t, n, k):
    _, B, _, sb = operands(t, n, k)
    X = torch.randn(t, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    q, s = oz.quantize_rows(X)
    size = oz.ozaki2_i8linear_workspace_size(t, n, k)
    ws, C = guarded(size), torch.empty(t, n, device="cuda")
    st = oz.ozaki2_i8linear_ws(t, n, k, X.data_ptr(), k, oz.FP32, B.data_ptr(), k, sb.data_ptr(), None, C.data_ptr(), n,
                               oz.FP32, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(C, oz.i8gemm(q, B, s, sb, out_dtype=torch.float32))
    sums = q.double() @ B.double().t().contiguous()
    # the sum is exact in binary32 (below 127 * 20 * k < 2^25, so off by half a step of it at most), times the scale
    want = sums * s.double()[:, None]
    assert ((C.double() - want).abs() <= 2.02 * 2.0 ** -24 * want.abs()).all()
    assert (ws[size:] == 0x5A).all()
