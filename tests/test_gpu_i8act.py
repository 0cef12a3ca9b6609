"""INT8 products with activation and residual (ozaki2_i8gemm_act, ozaki2_i8linear_act).

The activation is taken of the value that the product without one would round: with a binary32 output that value is
known bit for bit, and what follows it is off by what layer_util states."""
import pytest
import torch

import rns_emulated_fp64_amd as oz
from layer_util import NAMES, U32, act, act_error, rounded_to

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(t, n, k, seed, pad=0):
    g = gen(seed)
    A = torch.randint(-128, 128, (t, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, pad:]
    B = torch.randint(-128, 128, (n, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, pad:]
    sa = torch.rand(t, generator=g, device="cuda") + 0.5
    sb = (torch.rand(n, generator=g, device="cuda") + 0.5) / (5000 * max(k, 1) ** 0.5)
    return A, B, sa, sb, torch.randn(n, generator=g, device="cuda"), torch.randn(t, n, generator=g, device="cuda")


def check(C, z, name, residual):
    z = z.double()
    y, dy = act(name, z), act_error(name, z, torch.zeros_like(z))
    if residual is not None:
        dy = dy + U32 * (y.abs() + dy + residual.double().abs())
        y = y + residual.double()
    bad = ~((C.double() - y).abs() <= rounded_to(C.dtype, y, dy))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


SHAPES = [(1, 1, 1), (1, 300, 4096), (3, 17, 15), (16, 100, 300), (31, 65, 272), (33, 129, 1000), (65, 65, 65), (129, 127, 1040),
          (257, 300, 400), (300, 511, 2047), (700, 3001, 384), (70, 130, 32768)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_product(t, n, k, dtype):
    A, B, sa, sb, bias, residual = operands(t, n, k, t + n + k)
    residual = residual.to(dtype)
    for b in (None, bias):
        z = oz.i8gemm(A, B, sa, sb, b, out_dtype=torch.float32)
        for name in NAMES if t < 64 else (NAMES[k % 5],):
            check(oz.i8gemm(A, B, sa, sb, b, out_dtype=dtype, activation=name), z, name, None)
            check(oz.i8gemm(A, B, sa, sb, b, out_dtype=dtype, activation=name, residual=residual), z, name, residual)


@pytest.mark.parametrize("tile", ["skinny", "s11", "s21", "s22", "s42", "p4", "p8", "any"])
@pytest.mark.parametrize("t,n,k,pad", [(1, 40, 256, 0), (16, 300, 400, 0), (50, 700, 528, 16), (64, 64, 1024, 0), (300, 600, 272, 0),
                                       (513, 1030, 256, 0), (70, 90, 1001, 3)])
def test_every_tile_gives_the_same_bits(tile, t, n, k, pad, monkeypatch):
    A, B, sa, sb, bias, residual = operands(t, n, k, k + t, pad)
    monkeypatch.delenv("OZ2_LINEAR_TILE", raising=False)
    want = {name: oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32, activation=name, residual=residual) for name in NAMES}
    check(want["gelu"], oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32), "gelu", residual)
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    for name in NAMES:
        assert torch.equal(oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32, activation=name, residual=residual), want[name])


@pytest.mark.parametrize("t,n,k", [(1, 64, 64), (1, 9000, 1000), (4, 500, 4096), (5, 40, 100), (8, 9000, 512), (16, 256, 256),
                                   (37, 1000, 333), (300, 600, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_layer_is_quantise_then_product(t, n, k, dtype):
    _, B, _, sb, bias, residual = operands(1, n, k, t + n)
    residual = torch.randn(t, n, generator=gen(5), device="cuda").to(dtype)
    X = (torch.randn(t, k, generator=gen(k), device="cuda") * 3).to(dtype)
    q, s = oz.quantize_rows(X)
    for name in NAMES:
        for r in (None, residual):
            got = oz.i8linear(X, B, sb, bias, activation=name, residual=r)
            assert torch.equal(got, oz.i8gemm(q, B, s, sb, bias, out_dtype=dtype, activation=name, residual=r))


def test_without_either_it_is_the_plain_product():
    A, B, sa, sb, bias, _ = operands(40, 90, 256, 6)
    C = torch.empty(40, 90, dtype=torch.bfloat16, device="cuda")
    st = oz.ozaki2_i8gemm_act(40, 90, 256, A.data_ptr(), 256, sa.data_ptr(), B.data_ptr(), 256, sb.data_ptr(), bias.data_ptr(), 0, 0, 0,
                              C.data_ptr(), 90, oz.BF16, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(C, oz.i8gemm(A, B, sa, sb, bias))


def test_gaps_views_and_runs():
    A, B, sa, sb, bias, residual = operands(140, 300, 512, 7)
    want = oz.i8gemm(A, B, sa, sb, bias, activation="silu", residual=residual.bfloat16())
    wide = torch.full((142, 305), 7.0, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros(150, 303, dtype=torch.bfloat16, device="cuda")
    res[3:143, 1:301] = residual
    oz.i8gemm(A, B, sa, sb, bias, activation="silu", residual=res[3:143, 1:301], out=wide[1:141, 3:303])
    assert torch.equal(wide[1:141, 3:303], want)
    wide[1:141, 3:303] = 7.0
    assert (wide == 7.0).all()
    # rows of an odd length, more channels than one run copies: the residual moves along
    t, n, k = 26, 6000, 20001
    A, B, sa, sb, bias, residual = operands(t, n, k, 8)
    z = oz.i8gemm(A, B, sa, sb, bias, out_dtype=torch.float32)
    check(oz.i8gemm(A, B, sa, sb, bias, activation="gelu_tanh", residual=residual.bfloat16()), z, "gelu_tanh", residual.bfloat16())


def test_refusals():
    A, B, sa, sb, bias, residual = operands(20, 30, 64, 9)
    X = torch.randn(20, 64, device="cuda").bfloat16()
    for call in (lambda **k: oz.i8gemm(A, B, sa, sb, **k), lambda **k: oz.i8linear(X, B, sb, **k)):
        with pytest.raises(ValueError):
            call(activation="swish")
        for bad in (residual, residual.bfloat16()[:3], residual.bfloat16().cpu()):  # float32 beside a bfloat16 result
            with pytest.raises(ValueError):
                call(residual=bad)
        out = residual.bfloat16()
        with pytest.raises(oz.Ozaki2Error):
            call(residual=out, out=out)


def test_block_of_a_quantised_model():
    # norm -> widening layer with activation -> narrowing layer onto the residual stream, captured into a graph
    t, d, m = 9, 512, 1400
    g = gen(10)
    stream_in = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    delta = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    norm = torch.rand(d, generator=g, device="cuda") + 0.5
    W1, s1 = oz.quantize_rows(torch.randn(m, d, generator=g, device="cuda") / 20)
    W2, s2 = oz.quantize_rows(torch.randn(d, m, generator=g, device="cuda") / 30)
    b1 = torch.randn(m, generator=g, device="cuda")

    def block():
        q, s, total = oz.rmsnorm_quantize(delta, norm, stream_in)
        h = oz.i8gemm(q, W1, s, s1, b1, out_dtype=torch.bfloat16, activation="silu")
        return h, total, oz.i8linear(h, W2, s2, residual=total)

    h, total, out = block()
    q, s, _ = oz.rmsnorm_quantize(delta, norm, stream_in)
    z = (q.double() @ W1.double().t().contiguous()) * s.double()[:, None] * s1.double() + b1.double()
    y = act("silu", z)
    # the product's three roundings and the bias's
    close = rounded_to(torch.bfloat16, y, act_error("silu", z, 4 * U32 * (z.abs() + b1.double().abs())))
    assert ((h.double() - y).abs() <= close).all()
    assert torch.equal(total, (stream_in.float() + delta.float()).bfloat16())
    check(out, oz.i8linear(h, W2, s2, out_dtype=torch.float32), "none", total)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    for seed in (1, 2, 3):
        delta.copy_(torch.randn(t, d, generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        again = [v.clone() for v in got]
        for a, b in zip(again, block()):
            assert torch.equal(a, b)
