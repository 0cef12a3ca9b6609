"""The sampler's rows on several blocks (ozaki2_sample), whose common state is in a workspace, under streams, graphs and other calls, and more rows
than one launch takes. Each test asks for the workspace's size, which says how its rows go."""
import pytest
import torch

import rns_emulated_fp64_amd as oz
from test_gpu_sample import TYPES, check, gen, inputs

pytestmark = pytest.mark.gpu

# without filters; a cut that the list decides (top_k in one step, top_p in a window); rows that fit no list; min_p alone
SETTINGS = [dict(), dict(top_k=40), dict(top_k=3000), dict(top_k=50, top_p=0.9), dict(top_p=0.95), dict(top_p=0.95, temperature=0.5),
            dict(top_p=0.99, min_p=0.001), dict(min_p=0.02), dict(top_k=9000, top_p=0.8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("few,v", [(1, 70001), (20, 70001), (48, 66000), (60, 100003), (96, 100003)])
def test_same_tokens_however_rows_are_spread(dtype, few, v):
    many = 130
    assert oz.ozaki2_sample_workspace_size(few, v) > 0 and oz.ozaki2_sample_workspace_size(many, v) == 0
    z, u = inputs(many, v, dtype, v + few)
    for s in SETTINGS:
        tokens, logs = oz.sample(z, u, **s)
        one = oz.sample(z[:few], u[:few], **s)
        assert torch.equal(one[0], tokens[:few]) and torch.equal(one[1], logs[:few]), s


def test_settings_per_row_of_spread_rows():
    t, v = 40, 80011
    assert oz.ozaki2_sample_workspace_size(t, v) > 0
    z, u = inputs(t, v, torch.bfloat16, 1)
    g = gen(2)
    temperature = 0.4 + torch.rand(t, generator=g, device="cuda")
    temperature[::9] = 0.0
    top_k = torch.randint(-3, 5000, (t,), generator=g, device="cuda", dtype=torch.int32)
    top_p = 0.5 + 0.6 * torch.rand(t, generator=g, device="cuda")
    min_p = 0.02 * torch.rand(t, generator=g, device="cuda")
    check(z, u, temperature, top_k, top_p, min_p, most_unsure=8)


def test_cached_workspace_on_two_streams():
    t, v = 20, 70001
    assert oz.ozaki2_sample_workspace_size(t, v) > 0
    z, u = inputs(t, v, torch.float32, 3)
    settings = ((0, 0.9), (30, 1.0), (0, 1.0), (3000, 0.8))
    want = [oz.sample(z, u, top_k=k, top_p=p) for k, p in settings]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(24):
        s, (k, p) = streams[i % 2], settings[i % 4 if i < 12 else (i // 2) % 4]
        tokens = torch.empty(t, dtype=torch.int64, device="cuda")
        logs = torch.empty(t, dtype=torch.float32, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        assert oz.ozaki2_sample(t, v, z.data_ptr(), v, oz.FP32, u.data_ptr(), 1.0, 0, k, 0, p, 0, 0.0, 0, tokens.data_ptr(),
                                logs.data_ptr(), s.cuda_stream) == 0
        outs.append((tokens, logs, want[settings.index((k, p))]))
    torch.cuda.synchronize()
    for tokens, logs, w in outs:
        assert torch.equal(tokens, w[0]) and torch.equal(logs, w[1])


def test_graph_replays():
    t, v = 30, 70001
    need = oz.ozaki2_sample_workspace_size(t, v)
    assert need > 0
    z, u = inputs(t, v, torch.float32, 4)
    temperature = torch.full((t,), 0.8, device="cuda")
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def calls():
        # the same workspace from call to call, on one stream
        return [x for s in SETTINGS[:7] for x in oz.sample(z, u, **{"temperature": temperature, **s}, workspace=ws)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for seed in (5, 6, 7):
        for a, b in zip((z, u), inputs(t, v, torch.float32, seed)):
            a.copy_(b)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        again = [x.clone() for x in got]
        want = [x for s in SETTINGS[:7] for x in oz.sample(z, u, **{"temperature": temperature, **s})]
        for a, b in zip(again, want):
            assert torch.equal(a, b)
    check(z[:6], u[:6], 0.8, 50, 0.9)


def test_two_graphs_with_a_workspace_each():
    t, v = 9, 70001
    inputs_of = [inputs(t, v, torch.bfloat16, seed) for seed in (8, 9)]
    graphs, outs = [], []
    for z, u in inputs_of:
        oz.sample(z, u, top_p=0.9)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(oz.sample(z, u, top_p=0.9))
        graphs.append(graph)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (z, u), got in zip(inputs_of, outs):
            want = oz.sample(z, u, top_p=0.9)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_rows_than_a_launch():
    t, v = (1 << 20) + 700, 37
    assert oz.ozaki2_sample_workspace_size(t, v) == 0
    g = gen(10)
    z = torch.randn(t, v, generator=g, device="cuda") * 2
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    temperature = 0.5 + torch.rand(t, generator=g, device="cuda")
    top_k = torch.randint(0, 30, (t,), generator=g, device="cuda", dtype=torch.int32)
    top_p = 0.6 + 0.5 * torch.rand(t, generator=g, device="cuda")
    min_p = 0.1 * torch.rand(t, generator=g, device="cuda")
    tokens, logs = oz.sample(z, u, temperature, top_k, top_p, min_p)
    assert tokens.shape == (t,) and int(tokens.min()) >= 0 and int(tokens.max()) < v
    # rows on either side of the border between launches, against the definition and the whole call
    at = slice((1 << 20) - 400, t)
    got = check(z[at], u[at], temperature[at], top_k[at], top_p[at], min_p[at])
    assert torch.equal(got[0], tokens[at]) and torch.equal(got[1], logs[at])
