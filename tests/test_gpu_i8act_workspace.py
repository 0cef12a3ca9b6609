"""INT8 products in workspaces of either size: a plain product in what its own slices need, one with an activation or a residual in that and
in the larger one, with the same bits, since the sums are integers, and not a byte outside."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

SIZES = [(37, 4096, 11008), (24, 1000, 14336), (17, 1024, 65536), (40, 700, 9001), (65, 130, 32768), (300, 520, 256)]


def operands(t, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.randint(-127, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = (torch.rand(x, generator=g, device="cuda") / k ** 0.5 for x in (t, n))
    residual = torch.randn(t, n, generator=g, device="cuda").bfloat16()
    X = torch.randn(t, k, generator=g, device="cuda").bfloat16()
    return A, B, sa, sb, residual, X


class Guarded:
    """So many bytes with 4 KiB of marks behind them."""

    def __init__(self, size):
        self.size = size
        self.all = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")

    def whole(self):
        return self.all[:self.size]

    def kept(self):
        return bool((self.all[self.size:] == 0xA5).all())


@pytest.mark.parametrize("t,n,k", SIZES)
def test_both_sizes(t, n, k):
    A, B, sa, sb, residual, X = operands(t, n, k, t + n)
    for plain, more, call in (
            (oz.ozaki2_i8gemm_workspace_size(t, n, k), oz.ozaki2_i8gemm_act_workspace_size(t, n, k),
             lambda **kw: oz.i8gemm(A, B, sa, sb, **kw)),
            (oz.ozaki2_i8linear_workspace_size(t, n, k), oz.ozaki2_i8linear_act_workspace_size(t, n, k),
             lambda **kw: oz.i8linear(X, B, sb, out_dtype=torch.bfloat16, **kw))):
        for finish in (dict(), dict(activation="relu"), dict(residual=residual), dict(activation="silu", residual=residual)):
            want = call(**finish)
            for size in (plain, more):
                ws = Guarded(size)
                assert torch.equal(call(workspace=ws.whole(), **finish), want) and ws.kept(), (size, finish)
            if plain > 0:
                with pytest.raises(oz.Ozaki2Error):
                    call(workspace=torch.empty(plain - 1, dtype=torch.uint8, device="cuda"), **finish)


def test_a_plain_product_of_few_rows_takes_no_workspace():
    t, n, k = 37, 4096, 11008
    A, B, sa, sb, _, _ = operands(t, n, k, 1)
    want = oz.i8gemm(A, B, sa, sb)
    C = torch.empty_like(want)
    s = torch.cuda.current_stream().cuda_stream
    args = (t, n, k, A.data_ptr(), k, sa.data_ptr(), B.data_ptr(), k, sb.data_ptr(), 0, C.data_ptr(), n, oz.BF16)
    assert oz.ozaki2_i8gemm_ws(*args, 0, 0, s) == 0
    assert torch.equal(C, want)
    # nor the cached one: captured into a graph, which a call that takes it must not be
    C.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert oz.ozaki2_i8gemm(*args, torch.cuda.current_stream().cuda_stream) == 0
    for _ in range(3):
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
