"""INT8 products with scales (ozaki2_i8gemm, ozaki2_i8linear, ozaki2_quantize_rows) against their formulas.

The int32 sums are exact, so the only roundings are, per entry: the sum to
binary32, two products and (with a bias) one sum. Each is off by at most half a
step, u = 2^-24 relative; the bias enters with its own magnitude, so the bound is
3 u |sum sa sb| + u (|sum sa sb| + |bias|) before the rounding to the output
type, which adds half of its step."""
import pytest
import torch

import rns_emulated_fp64_amd as oz

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -24}  # half a step, relative to the binade's top
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the subnormal step
TILES = ("skinny", "s11", "s21", "s22", "s42", "p4", "p8", "any")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(t, n, k, seed, pad_a=0, pad_b=0, ext=False):
    g = gen(seed)
    lo, hi = (-128, 128) if not ext else (-128, -127)
    A = torch.randint(lo, hi, (t, k + pad_a), generator=g, device="cuda", dtype=torch.int8)[:, :k]
    B = torch.randint(lo, hi, (n, k + pad_b), generator=g, device="cuda", dtype=torch.int8)[:, :k]
    sa = torch.rand(t, generator=g, device="cuda") + 0.01
    sb = torch.rand(n, generator=g, device="cuda") * 0.1 + 0.001
    bias = torch.randn(n, generator=g, device="cuda") * 50
    return A, B, sa, sb, bias


def sums(A, B):
    """Exact integer sums: every partial sum of products is below 2^53."""
    return A.double().contiguous() @ B.double().t().contiguous()


def check(C, S, sa, sb, bias):
    r = S * sa.double()[:, None] * sb.double()
    tol = 3 * U32 * r.abs()
    if bias is not None:
        tol = tol + U32 * (r.abs() + bias.double().abs())
        r = r + bias.double()
    tol = tol * 1.01  # second-order terms
    # half a step of the output type: at most HALF * 2 relative to the value
    tol = tol + 2 * HALF[C.dtype] * (r.abs() + tol) + TINY[C.dtype]
    top = torch.finfo(C.dtype).max
    fine = r.abs() < top
    bad = ((C.double() - r).abs() > tol) & fine
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


SHAPES = [(1, 1, 1), (1, 1, 5), (3, 17, 15), (1, 4096, 256), (2, 33, 64), (16, 100, 300), (17, 333, 77), (31, 65, 272),
          (33, 129, 1000), (64, 257, 1024), (65, 65, 65), (100, 200, 304), (129, 127, 1040), (256, 256, 256),
          (257, 300, 400), (300, 511, 2047), (700, 3001, 384), (700, 3000, 400)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_product(t, n, k, dtype):
    A, B, sa, sb, bias = operands(t, n, k, t * 7 + n * 3 + k)
    S = sums(A, B)
    check(oz.i8gemm(A, B, sa, sb, out_dtype=dtype), S, sa, sb, None)
    check(oz.i8gemm(A, B, sa, sb, bias, out_dtype=dtype), S, sa, sb, bias)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("t,n,k,pad", [(1, 40, 256, 0), (16, 300, 400, 0), (50, 700, 528, 16), (64, 64, 1024, 0),
                                       (130, 257, 384, 32), (300, 600, 272, 0), (513, 1030, 256, 0),
                                       (70, 90, 1001, 3), (300, 300, 129, 0)])
def test_every_tile_gives_the_same_bits(tile, t, n, k, pad, monkeypatch):
    A, B, sa, sb, bias = operands(t, n, k, k + t, pad, pad)
    monkeypatch.delenv("OZ2_LINEAR_TILE", raising=False)
    want = oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32)
    check(want, sums(A, B), sa, sb, bias)
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    for dtype in (torch.float32, torch.bfloat16):
        got = oz.i8gemm(A, B, sa, sb, bias, out_dtype=dtype)
        assert torch.equal(got, want.to(dtype))


def test_largest_inner_dimension_is_exact():
    # every product is 2^14, so the sum is as large as it gets
    k = 2 ** 17 - 1
    A, B, sa, sb, _ = operands(3, 20, k, 0, ext=True)
    one = torch.ones(3, device="cuda"), torch.ones(20, device="cuda")
    C = oz.i8gemm(A, B, *one, out_dtype=torch.float32)
    assert torch.equal(C, torch.full((3, 20), float(k * 2 ** 14), device="cuda"))
    C = oz.i8gemm(A[:1].repeat(100, 1), B, torch.ones(100, device="cuda"), one[1], out_dtype=torch.float32)
    assert torch.equal(C, torch.full((100, 20), float(k * 2 ** 14), device="cuda"))


@pytest.mark.parametrize("t,n,k", [(65, 70, 65536), (70, 130, 32768), (256, 128, 65536), (300, 200, 65552),
                                   (130, 100, 65537)])
def test_slices_of_k(t, n, k):
    # long and narrow: k cut into slices whose sums are joined
    A, B, sa, sb, bias = operands(t, n, k, 3)
    assert k % 16 or oz.ozaki2_i8gemm_workspace_size(t, n, k) > 0
    S = sums(A, B)
    for dtype in (torch.float32, torch.bfloat16):
        check(oz.i8gemm(A, B, sa, sb, bias, out_dtype=dtype), S, sa, sb, bias)


@pytest.mark.parametrize("t,n,k", [(4, 60, 128), (20, 100, 256), (140, 300, 512), (600, 2100, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_out_keep_their_gaps(t, n, k, dtype):
    A, B, sa, sb, bias = operands(t, n, k, 5)
    wide = torch.full((t + 2, n + 3), 7.0, dtype=dtype, device="cuda")
    out = wide[1:t + 1, 1:n + 1]
    got = oz.i8gemm(A, B, sa, sb, bias, out=out)
    assert got.data_ptr() == out.data_ptr()
    check(out, sums(A, B), sa, sb, bias)
    wide[1:t + 1, 1:n + 1] = 7.0
    assert (wide == 7.0).all()


def test_views_and_copies():
    A, B, sa, sb, _ = operands(40, 50, 256, 9)
    want = oz.i8gemm(A, B, sa, sb)
    assert torch.equal(oz.i8gemm(A.t().contiguous().t(), B, sa, sb), want)       # columns contiguous: copied
    assert torch.equal(oz.i8gemm(A[::2], B, sa[::2], sb), want[::2])             # every second row
    assert torch.equal(oz.i8gemm(A[:, 5:], B[:, 5:], sa, sb), oz.i8gemm(A[:, 5:].contiguous(), B[:, 5:].contiguous(), sa, sb))
    assert torch.equal(oz.i8gemm(A[:1].expand(40, -1), B, sa[:1].expand(40), sb), want[:1].expand(40, -1))  # a broadcast row


def test_empty_sizes():
    A, B, sa, sb, bias = operands(5, 7, 16, 1)
    assert oz.i8gemm(A[:0], B, sa[:0], sb).shape == (0, 7)
    assert oz.i8gemm(A, B[:0], sa, sb[:0]).shape == (5, 0)
    assert torch.equal(oz.i8gemm(A[:, :0], B[:, :0], sa, sb, bias, out_dtype=torch.float32), bias.expand(5, 7))
    for t in (1, 100, 300):
        z = torch.zeros(t, 0, dtype=torch.int8, device="cuda")
        w = torch.zeros(300, 0, dtype=torch.int8, device="cuda")
        C = oz.i8gemm(z, w, torch.ones(t, device="cuda"), torch.ones(300, device="cuda"))
        assert C.shape == (t, 300) and not C.any()
    q, s = oz.quantize_rows(torch.zeros(4, 0, device="cuda"))
    assert q.shape == (4, 0) and torch.equal(s, torch.zeros(4, device="cuda"))


def quantised(x):
    """The documented formula, one binary32 rounding per operation."""
    x = x.float()
    top = x.abs().amax(1)
    up = torch.where(top > 0, (1.0 / top) * torch.tensor(127.0, device=x.device), torch.zeros_like(top))
    scale = top * torch.tensor(1.0 / 127.0, dtype=torch.float32, device=x.device)
    return torch.round(x * up[:, None]).to(torch.int8), scale


@pytest.mark.parametrize("t,k", [(1, 1), (3, 7), (5, 64), (2, 4096), (17, 2049), (4, 8193), (3, 20000), (1000, 512),
                                 ((1 << 20) + 300, 5)])  # the last: more rows than blocks
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_rows(t, k, dtype):
    x = (torch.randn(t, k + 3, generator=gen(t + k), device="cuda") * torch.rand(t, 1, generator=gen(1), device="cuda")).to(dtype)
    for v in (x[:, :k], x[:, 3:]):  # the second at an odd offset
        q, s = oz.quantize_rows(v)
        qr, sr = quantised(v)
        assert torch.equal(q, qr) and torch.equal(s, sr)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_odd_values(dtype):
    # ties, extremes, zeros, subnormals, Inf and NaN rows
    x = torch.zeros(8, 300, dtype=dtype, device="cuda")
    x[0, :255] = torch.arange(-127, 128, device="cuda").to(dtype) * 0.5  # many exact halves
    x[0, 299] = 127.0
    x[1, 3] = torch.finfo(dtype).max
    x[1, 4] = -torch.finfo(dtype).max
    x[3, 5] = torch.finfo(dtype).tiny
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[6, 0] = -3.0
    x[7, 299] = float("-inf")
    q, s = oz.quantize_rows(x)
    ok = [0, 1, 2, 6]
    qr, sr = quantised(x[ok])
    assert torch.equal(q[ok], qr) and torch.equal(s[ok], sr)
    assert s[2] == 0 and not q[2].any()
    for r in (4, 5, 7):
        assert torch.isnan(s[r]) and not q[r].any()
    if torch.finfo(dtype).tiny < 2.0 ** -120:
        assert not q[3].any()
    else:
        assert q[3, 5] == 127


LINEAR = [(1, 64, 64), (1, 4096, 4096), (1, 9000, 1000), (2, 33, 77), (4, 500, 4096), (5, 40, 100), (8, 300, 5000),
          (8, 9000, 512), (16, 256, 256), (37, 1000, 333), (130, 257, 1024), (300, 600, 2048)]


@pytest.mark.parametrize("t,n,k", LINEAR)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_is_quantise_then_product(t, n, k, dtype):
    _, B, _, sb, bias = operands(1, n, k, t + n)
    X = (torch.randn(t, k, generator=gen(k), device="cuda") * 3).to(dtype)
    q, s = oz.quantize_rows(X)
    for b in (None, bias):
        got = oz.i8linear(X, B, sb, b)
        assert got.dtype == dtype
        assert torch.equal(got, oz.i8gemm(q, B, s, sb, b, out_dtype=dtype))
    wide = oz.i8linear(X, B, sb, bias, out_dtype=torch.float32)
    assert torch.equal(wide, oz.i8gemm(q, B, s, sb, bias, out_dtype=torch.float32))
    check(wide, sums(q, B), s, sb, bias)


@pytest.mark.parametrize("t", [1, 3, 40, 300])
def test_linear_non_finite_rows(t):
    _, B, _, sb, bias = operands(1, 300, 512, 2)
    X = torch.randn(t, 512, generator=gen(3), device="cuda")
    clean = oz.i8linear(X, B, sb, bias)
    X[0, 11] = float("nan")
    got = oz.i8linear(X, B, sb, bias)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], clean[1:])


def test_streams_and_graph():
    A, B, sa, sb, bias = operands(128, 512, 65536, 11)  # slices of k: a workspace
    X = torch.randn(3, 1024, generator=gen(5), device="cuda").bfloat16()
    X2 = torch.randn(40, 1024, generator=gen(6), device="cuda").bfloat16()
    W = operands(1, 700, 1024, 12)[1]
    sw = torch.rand(700, device="cuda")
    want = [oz.i8gemm(A, B, sa, sb, bias), oz.i8linear(X, W, sw), oz.i8linear(X2, W, sw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [oz.i8gemm(A, B, sa, sb, bias), oz.i8linear(X, W, sw), oz.i8linear(X2, W, sw)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [oz.i8gemm(A, B, sa, sb, bias), oz.i8linear(X, W, sw), oz.i8linear(X2, W, sw)]
    for r in range(4):
        A.copy_(torch.randint(-128, 128, A.shape, generator=gen(r), device="cuda", dtype=torch.int8))
        X.copy_(torch.randn(X.shape, generator=gen(r), device="cuda"))
        X2.copy_(torch.randn(X2.shape, generator=gen(r + 9), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = [oz.i8gemm(A, B, sa, sb, bias), oz.i8linear(X, W, sw), oz.i8linear(X2, W, sw)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r


def test_cached_workspace_form():
    # the C entry points without a workspace argument, interleaved on two streams
    A, B, sa, sb, bias = operands(128, 512, 65536, 13)
    want = oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32)
    outs = [torch.empty_like(want) for _ in range(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        st = oz.ozaki2_i8gemm(128, 512, 65536, A.data_ptr(), 65536, sa.data_ptr(), B.data_ptr(), 65536, sb.data_ptr(),
                              bias.data_ptr(), o.data_ptr(), 512, oz.FP32, streams[i % 2].cuda_stream)
        assert st == 0
    X = torch.randn(40, 1024, generator=gen(6), device="cuda")
    W = operands(1, 700, 1024, 12)[1]
    C = torch.empty(40, 700, device="cuda")
    torch.cuda.synchronize()
    st = oz.ozaki2_i8linear(40, 700, 1024, X.data_ptr(), 1024, oz.FP32, W.data_ptr(), 1024, torch.ones(700, device="cuda").data_ptr(),
                            None, C.data_ptr(), 700, oz.FP32, streams[0].cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert torch.equal(C, oz.i8linear(X, W, torch.ones(700, device="cuda")))


def test_offsets_past_32_bits():
    # rows of B more than 2^32 bytes apart, and an output whose elements lie past 2^31
    n, k, t = 70000, 65536, 33
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * n * k:
        pytest.skip("needs memory")
    B = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    rows = torch.tensor([0, 1, 32767, 65535, 65536, 65537, n - 1], device="cuda")
    B[rows] = torch.randint(-128, 128, (len(rows), k), generator=gen(0), device="cuda", dtype=torch.int8)
    A = torch.randint(-128, 128, (t, k), generator=gen(1), device="cuda", dtype=torch.int8)
    one = torch.ones(t, device="cuda"), torch.ones(n, device="cuda")
    for a, s in ((A, one[0]), (A[:3], one[0][:3])):
        C = oz.i8gemm(a, B, s, one[1], out_dtype=torch.float32)
        assert torch.equal(C[:, rows], sums(a, B[rows]).float())
        C[:, rows] = 0
        assert not C.any()


def test_python_refusals():
    A, B, sa, sb, bias = operands(5, 7, 16, 1)
    with pytest.raises(TypeError):
        oz.i8gemm(A.float(), B, sa, sb)
    with pytest.raises(TypeError):
        oz.i8gemm(A.cpu(), B, sa, sb)
    with pytest.raises(TypeError):
        oz.i8gemm(A, B, sa, sb, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        oz.i8gemm(A, B[:, :8], sa, sb)
    with pytest.raises(ValueError):
        oz.i8gemm(A, B, sa[:4], sb)
    with pytest.raises(ValueError):
        oz.i8gemm(A, B, sa.double(), sb)
    with pytest.raises(ValueError):
        oz.i8gemm(A, B, sa, sb, bias[:3])
    with pytest.raises(ValueError):
        oz.i8gemm(A, B, sa, sb, out=torch.empty(5, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        oz.i8gemm(A[0], B, sa, sb)
    with pytest.raises(oz.Ozaki2Error) as e:
        oz.i8gemm(*operands(128, 512, 65536, 1)[:4], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(oz.Ozaki2Error) as e:  # 2^17: the sums would leave int32
        z = torch.zeros(1, 2 ** 17, dtype=torch.int8, device="cuda")
        oz.i8gemm(z, z, torch.ones(1, device="cuda"), torch.ones(1, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(TypeError):
        oz.quantize_rows(A)
    with pytest.raises(TypeError):
        oz.i8linear(A, B, sb)
