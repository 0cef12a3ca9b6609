"""The sampler (ozaki2_sample) against its definition in 64 bits.

A weight is off by at most 2^-41 from its rounding and 2^-44.6 from the exponential, relative to the largest weight, which the sum is
no smaller than: a running sum of v of them by at most v 2^-40.8 of the whole. Where u, or a filter's bound, is further than
that from the sums next to it, the token has to be the definition's; rows where it is not are counted, and they
are few. The logarithm of the probability is a binary64 value rounded to binary32, with a sum off by as much."""
import math

import numpy as np
import pytest
import torch

import rns_emulated_fp64_amd as oz
from sample_util import reference

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def per_row(x, t):
    return x.tolist() if isinstance(x, torch.Tensor) else [x] * t


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, most_unsure=None, **kw):
    tokens, logs = oz.sample(logits, u, temperature, top_k, top_p, min_p, **kw)
    t, v = logits.shape
    settings = [per_row(x, t) for x in (temperature, top_k, top_p, min_p)]
    rows, us = logits.double().cpu().numpy(), u.tolist()
    unsure = 0
    slack = v * 2.0 ** -40.8
    for i in range(t):
        ref = reference(rows[i], us[i], *(s[i] for s in settings))
        if ref is None:
            assert tokens[i] == -1 and math.isnan(logs[i]), i
            continue
        index, sums, token, log, margin = ref
        if margin <= slack:
            unsure += 1
            assert 0 <= int(tokens[i]) < v and rows[i][int(tokens[i])] > -np.inf
            continue
        assert int(tokens[i]) == token, (i, int(tokens[i]), token, [s[i] for s in settings], us[i], margin)
        assert abs(float(logs[i]) - log) <= 2.0 ** -24 * abs(log) + 2 * slack + 1e-14, (i, float(logs[i]), log)
    assert unsure <= (max(2, t // 50) if most_unsure is None else most_unsure), unsure
    return tokens, logs


def inputs(t, v, dtype, seed, spread=2.0):
    g = gen(seed)
    z = torch.randn(t, v, generator=g, device="cuda") * spread + 6 * (torch.rand(t, v, generator=g, device="cuda") < 3e-4)
    z[torch.rand(t, v, generator=g, device="cuda") < 0.02] = -math.inf
    z[:, v // 2] = 1.0
    return z.to(dtype), torch.rand(t, generator=g, device="cuda", dtype=torch.float64)


# one block per row and several, ragged ends, rows that fit the list and rows that do not
SIZES = [(1, 1), (3, 2), (7, 100), (5, 4096), (4, 4097), (1, 8192), (2, 8193), (1, 50001), (3, 32000), (40, 9001), (600, 500),
         (1500, 70), (2, 300001)]
SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=0.0), dict(top_k=1), dict(top_k=50), dict(top_k=50, top_p=0.9),
            dict(top_p=0.9), dict(top_p=0.3), dict(top_p=0.999, temperature=1.5), dict(min_p=0.05), dict(min_p=1.0),
            dict(top_k=20, top_p=0.8, min_p=0.1, temperature=1.3), dict(top_k=6000), dict(top_k=6000, top_p=0.7),
            dict(top_p=0.0), dict(top_k=10 ** 9), dict(temperature=30.0, top_p=0.5), dict(temperature=0.01)]


@pytest.mark.parametrize("t,v", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_settings(t, v, dtype):
    logits, u = inputs(t, v, dtype, t + v)
    some = SETTINGS if v < 40000 and t < 100 else SETTINGS[::3]
    for s in some:
        check(logits, u, **s)


@pytest.mark.parametrize("dtype", TYPES)
def test_settings_per_row(dtype):
    t, v = 300, 3001
    logits, u = inputs(t, v, dtype, 1)
    g = gen(2)

    def uniform():
        return torch.rand(t, generator=g, device="cuda")

    temperature = torch.where(uniform() < 0.1, torch.zeros(t, device="cuda"), 0.2 + 2 * uniform())
    top_k = torch.randint(-2, 400, (t,), generator=g, device="cuda", dtype=torch.int32)
    top_p = 1.2 * uniform() - 0.1
    min_p = 0.2 * uniform() - 0.05
    check(logits, u, temperature, top_k, top_p, min_p)
    check(logits, u, temperature)
    check(logits, u, 0.9, top_k, 0.9)
    check(logits, u, temperature, 0, top_p, 0.01)
    # out of range or NaN in a vector: refused for that row alone
    temperature[5], temperature[6], top_p[7], min_p[8] = -1.0, float("nan"), float("nan"), float("nan")
    min_p[9], top_p[10] = 3.0, 7.0
    u[11] = float("nan")
    u[12], u[13], u[14] = -0.5, 1.0, float("inf")
    tokens, _ = check(logits, u, temperature, top_k, top_p, min_p)
    assert (tokens[[5, 6, 7, 8, 11]] == -1).all()


@pytest.mark.parametrize("v", [5000, 20000, 100000])
def test_equal_logits(v):
    # thousands of equal entries in one step: cuts inside them go by the index
    u = torch.rand(6, generator=gen(3), device="cuda", dtype=torch.float64)
    flat = torch.zeros(6, v, device="cuda")
    for s in (dict(), dict(top_k=4500), dict(top_k=v - 1), dict(top_p=0.37), dict(top_k=4999, top_p=0.5), dict(temperature=0.0),
              dict(temperature=float("inf"))):
        check(flat, u, most_unsure=6, **s)
        k = s.get("top_k", v)
        tokens, logs = oz.sample(flat, u, **s)
        if "top_p" not in s and s.get("temperature") != 0.0:
            # exact: all weights are 1
            assert torch.equal(tokens, (u * k).floor().long())
            assert torch.allclose(logs.double(), torch.full_like(u, -math.log(k)), rtol=1e-7)
    assert torch.equal(oz.sample(flat, u, temperature=0.0)[0], torch.zeros(6, dtype=torch.long, device="cuda"))
    # two levels, and zeros of both signs
    two = torch.zeros(6, v, device="cuda")
    two[:, ::2] = -0.0
    two[:, 1::7] = 1.0
    for s in (dict(top_k=v // 2), dict(top_k=v // 2 + 1, top_p=0.6), dict(top_p=0.9), dict(top_k=v // 7 - 3)):
        check(two, u, most_unsure=6, **s)


def test_long_flat_rows():
    # cuts among tens of thousands of entries that are close to each other, in 16 bits with many ties
    for dtype in TYPES:
        z = (torch.randn(8, 90001, generator=gen(4), device="cuda") * 0.003).to(dtype)
        u = torch.rand(8, generator=gen(5), device="cuda", dtype=torch.float64)
        for s in (dict(top_k=30000), dict(top_p=0.4), dict(top_k=50000, top_p=0.7), dict(top_p=0.9999), dict(min_p=0.997)):
            check(z, u, most_unsure=8, **s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("min_p", [1e-13, 1e-6, 0.003, 0.02, 0.1, 0.35, 0.9, 1.0])
def test_min_p_beside_the_other_filters(dtype, min_p):
    # min_p's border above, at and below those of a top_k and a top_p whose entries do not all fit a list
    z, u = inputs(6, 30000, dtype, 30)
    for s in (dict(), dict(top_k=3000), dict(top_k=9000), dict(top_k=400), dict(top_k=400, top_p=0.9), dict(top_p=0.95),
              dict(top_p=0.6), dict(top_p=0.999), dict(top_k=5000, top_p=0.9)):
        for temperature in (0.6, 1.7):
            check(z, u, temperature=temperature, min_p=min_p, most_unsure=2, **s)
    # just at the border of a filter: the weight of the entry where it cuts
    for k in (300, 3000):
        w = torch.exp(torch.sort(z.double(), dim=1, descending=True)[0][:, k - 1] - z.double().amax(1)).float()
        for m in (w, torch.nextafter(w, torch.zeros_like(w)), torch.nextafter(w, torch.ones_like(w))):
            check(z, u, top_k=k, min_p=m, most_unsure=6)
            check(z, u, top_p=0.97, min_p=m, most_unsure=6)


@pytest.mark.parametrize("t,v", [(2, 70000), (5, 131073), (100, 66000)])
def test_long_rows_on_several_blocks(t, v):
    # (with 131073 entries the bound of 7e-8 is up to a tenth of the sums' distances near a top_p of 0.99, 1e-6, on either side: a
    # row in six is unsure, so three of five are no surprise in twenty settings)
    for dtype in TYPES:
        z, u = inputs(t, v, dtype, v)
        for s in (dict(), dict(top_k=50, top_p=0.9), dict(top_k=4000), dict(top_p=0.95, temperature=1.5), dict(top_p=0.99, min_p=0.01),
                  dict(temperature=0.0), dict(top_k=4000, top_p=0.8)):
            check(z[:7], u[:7], most_unsure=4, **s)
    z[0, 5] = math.inf
    z[1] = -math.inf
    for s in SETTINGS[:8]:
        check(z[:7], u[:7], most_unsure=4, **s)


def test_equal_logits_and_min_p():
    z = torch.zeros(3, 70000, device="cuda")
    u = torch.tensor([0.1, 0.5, 0.9], device="cuda", dtype=torch.float64)
    for s in (dict(min_p=1.0), dict(min_p=0.5), dict(min_p=1.0, top_k=69999), dict(min_p=1.0, top_p=0.5)):
        check(z, u, most_unsure=3, **s)


def test_odd_rows():
    v = 9000
    for dtype in TYPES:
        z = torch.randn(9, v, generator=gen(6), device="cuda").to(dtype)
        u = torch.full((9,), 0.7, device="cuda", dtype=torch.float64)
        z[0] = -math.inf
        z[1, 17] = float("nan")
        z[2] = -math.inf
        z[2, 8999] = -3.0
        z[3, [5, 77, 8000]] = math.inf
        z[4] = math.inf
        z[5] = torch.finfo(dtype).max
        z[6] = torch.finfo(dtype).min
        z[6, 100] = torch.finfo(dtype).max
        z[7] = -math.inf
        z[7, 3], z[7, 4] = float("nan"), 1.0
        for s in SETTINGS:
            tokens, logs = check(z, u, most_unsure=9, **s)
            assert tokens[0] == -1 and tokens[1] == -1 and tokens[7] == -1
            assert tokens[2] == 8999 and logs[2] == 0 and tokens[6] == (100 if s.get("temperature") != math.inf else tokens[6])
            assert int(tokens[3]) in (5, 77, 8000)
        # NaN with its sign set
        z[8, 4000] = torch.tensor(-float("nan"), device="cuda")
        assert oz.sample(z, u)[0][8] == -1


def test_never_a_banned_token():
    v = 30000
    z = torch.full((200, v), -math.inf, device="cuda")
    allowed = torch.randperm(v, generator=gen(7), device="cuda")[:40]
    z[:, allowed] = torch.randn(200, 40, generator=gen(8), device="cuda")
    u = torch.linspace(0, 1, 200, device="cuda", dtype=torch.float64)
    for s in SETTINGS:
        tokens, _ = oz.sample(z, u, **s)
        assert torch.isin(tokens, allowed).all(), s


def test_ends_of_u():
    # 0 takes the first kept index, just below 1 the last
    z, _ = inputs(3, 20001, torch.float32, 9)
    for u in (0.0, 1.0 - 2.0 ** -53):
        for s in (dict(), dict(top_k=100), dict(top_p=0.9), dict(top_p=0.99, temperature=2.0), dict(min_p=0.01)):
            tokens, _ = oz.sample(z, torch.full((3,), u, device="cuda", dtype=torch.float64), **s)
            for i in range(3):
                index = reference(z[i].double().cpu().numpy(), u, s.get("temperature", 1.0), s.get("top_k", 0), s.get("top_p", 1.0),
                                  s.get("min_p", 0.0))[0]
                w = z[i].double()[torch.from_numpy(index).cuda()]
                real = index[((w - z[i].double().max()) / s.get("temperature", 1.0) > -28).cpu().numpy()]  # weights that do not round to 0
                assert int(tokens[i]) in ((real[0],) if u == 0 else index[-200:]), s


def test_frequencies():
    # the distribution itself: 200000 draws over 12 tokens
    z = torch.randn(1, 12, generator=gen(10), device="cuda")
    n = 200000
    u = torch.rand(n, generator=gen(11), device="cuda", dtype=torch.float64)
    tokens, logs = oz.sample(z.expand(n, 12), u, temperature=0.8)
    p = torch.softmax(z[0].double() / 0.8, 0)
    got = torch.bincount(tokens, minlength=12).double() / n
    # six standard deviations of a frequency
    assert ((got - p).abs() <= 6 * (p * (1 - p) / n).sqrt()).all()
    assert torch.allclose(logs.double(), p[tokens].log(), rtol=1e-6, atol=1e-9)


def test_same_tokens_however_rows_are_spread():
    # a row alone and among many
    z, u = inputs(520, 40000, torch.bfloat16, 12)
    for s in (dict(), dict(top_k=40), dict(top_p=0.95), dict(top_p=0.95, temperature=0.5)):
        tokens, logs = oz.sample(z, u, **s)
        for i in (0, 3, 519):
            one = oz.sample(z[i:i + 1], u[i:i + 1], **s)
            assert one[0] == tokens[i] and one[1] == logs[i]
        again = oz.sample(z, u, **s)
        assert torch.equal(again[0], tokens) and torch.equal(again[1], logs)


def test_views_and_alignment():
    z, u = inputs(6, 5003, torch.float16, 13)
    want = oz.sample(z, u, top_p=0.9)
    wide = torch.full((8, 5010), float("nan"), dtype=torch.float16, device="cuda")
    wide[1:7, 3:5006] = z
    for got in (oz.sample(wide[1:7, 3:5006], u, top_p=0.9), oz.sample(z.t().contiguous().t(), u, top_p=0.9)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = oz.sample(z[::2], u[::2], top_p=0.9)
    assert torch.equal(got[0], want[0][::2])


def test_empty():
    tokens, logs = oz.sample(torch.zeros(0, 5, device="cuda"), torch.zeros(0, device="cuda", dtype=torch.float64))
    assert tokens.shape == logs.shape == (0,) and tokens.dtype == torch.int64


def test_refusals():
    z, u = inputs(4, 50, torch.float32, 14)
    for bad in (z.double(), z.cpu()):
        with pytest.raises(TypeError):
            oz.sample(bad, u)
    for bad in (u.float(), u[:3], u.cpu()):
        with pytest.raises(ValueError):
            oz.sample(z, bad)
    with pytest.raises(ValueError):
        oz.sample(z[:, :0], u)
    for s in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_p=1.5), dict(top_p=-0.1), dict(min_p=2.0),
              dict(min_p=float("nan"))):
        with pytest.raises(oz.Ozaki2Error):
            oz.sample(z, u, **s)
    for s in (dict(temperature=u), dict(top_k=torch.zeros(4, device="cuda", dtype=torch.int64)), dict(top_p=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            oz.sample(z, u, **s)


def test_offsets_past_32_bits():
    t, v = 700, 4000000
    z = torch.zeros(t, v, dtype=torch.bfloat16, device="cuda")
    z[-1] = inputs(1, v, torch.bfloat16, 15)[0][0]
    u = torch.full((t,), 0.25, device="cuda", dtype=torch.float64)
    tokens, _ = oz.sample(z, u, top_p=0.9)
    want = oz.sample(z[-1:], u[-1:], top_p=0.9)[0]
    assert tokens[-1] == want[0]
    check(z[-1:], u[-1:], top_p=0.9, most_unsure=1)
    tokens, _ = oz.sample(z, u)
    assert (tokens[:-1] == v // 4).all()


def test_graph_and_streams():
    z, u = inputs(30, 12001, torch.float32, 16)
    temperature = torch.full((30,), 0.8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        oz.sample(z, u, temperature, 50, 0.9)
        oz.sample(z, u, temperature, 0, 0.99)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = oz.sample(z, u, temperature, 50, 0.9)
        b = oz.sample(z, u, temperature, 0, 0.99)
    for seed in (17, 18, 19):
        x, y = inputs(30, 12001, torch.float32, seed)
        z.copy_(x)
        u.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in a + b]
        want = oz.sample(z, u, temperature, 50, 0.9) + oz.sample(z, u, temperature, 0, 0.99)
        for v, w in zip(got, want):
            assert torch.equal(v, w)


def test_cached_workspace_on_two_streams():
    z, u = inputs(20, 30000, torch.float32, 20)
    want = oz.sample(z, u, top_p=0.9)[0], oz.sample(z, u, top_k=30)[0]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, w, (k, p) in zip(streams, want, ((0, 0.9), (30, 1.0))):
            out = torch.empty(20, dtype=torch.int64, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            assert oz.ozaki2_sample(20, 30000, z.data_ptr(), 30000, oz.FP32, u.data_ptr(), 1.0, 0, k, 0, p, 0, 0.0, 0, out.data_ptr(), 0,
                                    s.cuda_stream) == 0
            outs.append((out, w))
    torch.cuda.synchronize()
    for got, w in outs:
        assert torch.equal(got, w)


def test_a_step_of_decoding():
    # norm, quantised layers, output layer in fp32, and a token per sequence
    t, d, m, v = 5, 256, 700, 5001
    g = gen(21)
    x = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    delta = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    W1, s1 = oz.quantize_rows(torch.randn(m, d, generator=g, device="cuda") / 16)
    W2, s2 = oz.quantize_rows(torch.randn(d, m, generator=g, device="cuda") / 26)
    W = (torch.randn(v, d, generator=g, device="cuda") / 8).bfloat16()
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)

    def step():
        q, s, total = oz.rmsnorm_quantize(delta, None, x)
        h = oz.i8gemm(q, W1, s, s1, activation="silu")
        h = oz.i8linear(h, W2, s2, residual=total)
        logits, _ = oz.linear(h, W, out_dtype=torch.float32)
        return (logits,) + oz.sample(logits, u, 0.8, 40, 0.95)

    logits, tokens, logs = step()
    check(logits, u, 0.8, 40, 0.95)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (22, 23, 24):
        delta.copy_(torch.randn(t, d, generator=gen(seed), device="cuda"))
        u.copy_(torch.rand(t, generator=gen(seed), device="cuda", dtype=torch.float64))
        graph.replay()
        torch.cuda.synchronize()
        again = [v.clone() for v in got]
        for a, b in zip(again, step()):
            assert torch.equal(a, b)
