"""The quantising norm (ozaki2_rmsnorm_quantize) against its formula.

Squares, their sum and y are binary64 and y is rounded once to binary32, so the formula in torch's binary64, whose sum is
in another order, gives the same binary32 y but for one value in some 2^27 (two sums that differ by 2^-52 on either side
of a border). Codes and scales follow from y by the documented binary32 operations. So all three outputs are compared
bit for bit."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def formula(X, weight, residual, eps):
    """(q, scale, sum) for rows that are finite."""
    h = X.float()
    if residual is not None:
        h = h + residual.float()
    h64 = h.double()
    mean = (h64 * h64).sum(1, keepdim=True) / max(h.shape[1], 1) + eps
    up = torch.where(mean == 0, torch.zeros_like(mean), 1.0 / torch.sqrt(mean))
    y = (h64 * up * (1.0 if weight is None else weight.double())).float()
    top = y.abs().amax(1) if y.shape[1] else torch.zeros(len(y), device=y.device)
    to_code = torch.where(top >= 2.0 ** -120, (1.0 / top) * 127.0, torch.zeros_like(top))
    return torch.round(y * to_code[:, None]).to(torch.int8), top * (1.0 / 127.0), h.to(X.dtype)


def inputs(t, k, dtype, seed):
    g = gen(seed)
    X = (torch.randn(t, k, generator=g, device="cuda") * torch.exp(torch.randn(t, 1, generator=g, device="cuda"))).to(dtype)
    residual = (torch.randn(t, k, generator=g, device="cuda") * 2).to(dtype)
    weight = torch.randn(k, generator=g, device="cuda")
    return X, weight, residual


def check(got, want, has_sum=True):
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1], want[1])
    if has_sum:
        assert torch.equal(got[2], want[2])
    else:
        assert got[2] is None


# kernels of 64, 256 and 512 threads, rows longer than the registers
SIZES = [(1, 1), (3, 7), (2, 64), (5, 511), (4, 513), (1, 2048), (300, 2049), (257, 4096), (7, 4096), (2, 8191), (3, 8193),
         (2, 16384), (3, 16391), (2, 50000), (2300, 130), (4100, 33)]


@pytest.mark.parametrize("t,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(t, k, dtype):
    X, weight, residual = inputs(t, k, dtype, t + k)
    check(oz.rmsnorm_quantize(X, weight, residual, eps=1e-5), formula(X, weight, residual, 1e-5))
    check(oz.rmsnorm_quantize(X, weight), formula(X, weight, None, 1e-6), False)
    check(oz.rmsnorm_quantize(X), formula(X, None, None, 1e-6), False)


@pytest.mark.parametrize("dtype", TYPES)
def test_views_and_gaps(dtype):
    X, weight, residual = inputs(9, 707, dtype, 1)
    wide = torch.full((11, 710), 5.0, dtype=dtype, device="cuda")
    wide[1:10, 3:] = X
    want = formula(X, weight, residual, 1e-6)
    out = torch.full((11, 715), 7.0, dtype=dtype, device="cuda")
    got = oz.rmsnorm_quantize(wide[1:10, 3:], weight, residual.t().contiguous().t(), sum_out=out[1:10, 5:712])
    check(got, want)
    assert got[2].data_ptr() == out[1:10, 5:].data_ptr()
    out[1:10, 5:712] = 7.0
    assert (out == 7.0).all()
    check(oz.rmsnorm_quantize(X[:1].expand(9, -1), weight, residual), formula(X[:1].expand(9, -1), weight, residual, 1e-6))
    check(oz.rmsnorm_quantize(X[::2], weight, residual[::2]), tuple(v[::2] for v in want))


@pytest.mark.parametrize("k", [100, 4096, 20001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sum_in_place(k, dtype):
    X, weight, residual = inputs(6, k, dtype, 2)
    want = formula(X, weight, residual, 1e-6)
    over = residual.clone()
    check(oz.rmsnorm_quantize(X, weight, over, sum_out=over), want)
    assert torch.equal(over, want[2])
    over = X.clone()
    check(oz.rmsnorm_quantize(over, weight, residual, sum_out=over), want)


@pytest.mark.parametrize("k", [60, 4096, 17000])
def test_odd_rows(k):
    X, weight, residual = inputs(9, k, torch.float32, 3)
    X[0] = 0
    X[1] = 0
    X[1, k - 1] = 1e-30
    X[2] = 3e38  # the squares leave binary32, the norm does not
    X[3, k // 2] = float("inf")
    X[4, 0] = float("nan")
    X[5, k - 1] = -float("inf")
    X[6] *= 1e-44
    q, scale, total = oz.rmsnorm_quantize(X, weight, eps=0.0)
    fine = [0, 1, 2, 6, 7, 8]
    wq, ws, _ = formula(X[fine], weight, None, 0.0)
    assert torch.equal(q[fine], wq) and torch.equal(scale[fine], ws)
    assert scale[0] == 0 and not q[0].any()
    for r in (3, 4, 5):
        assert torch.isnan(scale[r]) and not q[r].any()
    # a sum that overflows binary32, and one of opposite infinities
    q, scale, total = oz.rmsnorm_quantize(X, weight, X)
    assert torch.isnan(scale[2]) and not q[2].any() and torch.isinf(total[2]).all()
    q, scale, total = oz.rmsnorm_quantize(X, weight, -X)
    assert torch.isnan(scale[3]) and scale[8] == 0 and not q.any() and not total[8].any()
    # weights: a zero, an infinity
    weight[1] = 0.0
    check(oz.rmsnorm_quantize(X[7:], weight), formula(X[7:], weight, None, 1e-6), False)
    weight[1] = float("inf")
    q, scale, _ = oz.rmsnorm_quantize(X[7:], weight)
    assert torch.isnan(scale).all() and not q.any()


def test_fp16_sum_that_overflows_its_type():
    X = torch.full((2, 640), 60000.0, dtype=torch.float16, device="cuda")
    q, scale, total = oz.rmsnorm_quantize(X, None, X)
    assert torch.isinf(total).all() and (q == 127).all()  # the norm is that of the binary32 sum
    check((q, scale, total), formula(X, None, X, 1e-6))


def test_empty():
    X, weight, residual = inputs(4, 16, torch.bfloat16, 4)
    q, scale, total = oz.rmsnorm_quantize(X[:0], weight, residual[:0])
    assert q.shape == (0, 16) and scale.shape == (0,) and total.shape == (0, 16)
    q, scale, total = oz.rmsnorm_quantize(X[:, :0], weight[:0], residual[:, :0])
    assert q.shape == (4, 0) and total.shape == (4, 0) and torch.equal(scale, torch.zeros(4, device="cuda"))


def test_refusals():
    X, weight, residual = inputs(4, 16, torch.bfloat16, 5)
    with pytest.raises(TypeError):
        oz.rmsnorm_quantize(X.double(), weight)
    with pytest.raises(TypeError):
        oz.rmsnorm_quantize(X.cpu(), weight)
    for bad in (residual.float(), residual[:3], residual.cpu()):
        with pytest.raises(ValueError):
            oz.rmsnorm_quantize(X, weight, bad)
    for bad in (weight[:5], weight.double(), weight.cpu()):
        with pytest.raises(ValueError):
            oz.rmsnorm_quantize(X, bad)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(oz.Ozaki2Error):
            oz.rmsnorm_quantize(X, weight, eps=eps)
    wide = torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda")
    for out in (residual[:, :8], residual.float(), residual.t().contiguous().t()):
        with pytest.raises(ValueError):
            oz.rmsnorm_quantize(X, weight, residual, sum_out=out)
    with pytest.raises(ValueError):  # shifted by a row
        oz.rmsnorm_quantize(wide[:4], weight, residual, sum_out=wide[1:])
    with pytest.raises(ValueError):  # one row for all
        oz.rmsnorm_quantize(wide[:1].expand(4, -1), weight, residual, sum_out=wide[:4])


def test_rows_past_32_bits():
    # offsets of rows beyond 2^32 bytes
    t, k = 2100000, 1056
    X = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")
    last, weight, _ = inputs(3, k, torch.bfloat16, 6)
    X[-3:] = last
    q, scale, _ = oz.rmsnorm_quantize(X, weight)
    wq, ws, _ = formula(last, weight, None, 1e-6)
    assert torch.equal(q[-3:], wq) and torch.equal(scale[-3:], ws) and not q[:-3].any()


def test_graph_and_streams():
    X, weight, residual = inputs(33, 4096, torch.bfloat16, 7)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        oz.rmsnorm_quantize(X, weight, residual)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = oz.rmsnorm_quantize(X, weight, residual)
    for seed in (8, 9, 10):
        a, w, b = inputs(33, 4096, torch.bfloat16, seed)
        X.copy_(a)
        weight.copy_(w)
        residual.copy_(b)
        graph.replay()
        check(got, formula(X, weight, residual, 1e-6))


def test_products_of_the_norm():
    # its outputs are a quantised layer's operands
    X, weight, residual = inputs(40, 512, torch.bfloat16, 11)
    W = torch.randn(96, 512, generator=gen(12), device="cuda")
    B, b_scale = oz.quantize_rows(W)
    q, scale, _ = oz.rmsnorm_quantize(X, weight, residual)
    wq, ws, _ = formula(X, weight, residual, 1e-6)
    C = oz.i8gemm(q, B, scale, b_scale, out_dtype=torch.float32)
    want = (wq.double() @ B.double().t().contiguous()) * ws.double()[:, None] * b_scale.double()
    # the sum's rounding and those of two products, half a step each
    assert ((C.double() - want).abs() <= 3.01 * 2.0 ** -24 * want.abs()).all()
