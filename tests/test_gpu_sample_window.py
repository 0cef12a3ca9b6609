"""top_p beside min_p where logits are clustered (ozaki2_sample against its definition in 64 bits).

The sampler estimates the step in which top_p cuts from counts per step, each entry taken for its step's middle. Entries that all lie near one
end of their steps shift that estimate by up to a step's width, so that the cut can lie outside the narrower windows, also
where min_p's own border is between the two. The rows here are such: one entry at the top, 1800 just below the start of step 10, 1900 just before
the end of step 40, top_p in the first cluster, min_p between them; then top_p, not min_p, says which entries of the first are
kept, and without it every log-probability would be off by 1e-3."""
import math

import numpy as np
import pytest
import torch

import rns_emulated_fp64_amd as oz
from test_gpu_sample import check, gen

pytestmark = pytest.mark.gpu

STEP = math.log(2) / 99.5  # of logits over temperature
# logits of the two clusters, values of all three types; at this temperature they are 10.02 and 40.96 steps below 0
NEAR, FAR, TEMPERATURE = -0.53125, -2.171875, 0.53125 / (10.02 * STEP)


def clustered(t, v, dtype, seed):
    """Rows of v entries, the clusters' at random places, -inf elsewhere."""
    g = gen(seed)
    z = torch.full((t, v), -math.inf, device="cuda")
    for i in range(t):
        at = torch.randperm(v, generator=g, device="cuda")[:3701]
        z[i, at[:1]], z[i, at[1:1801]], z[i, at[1801:]] = 0.0, NEAR, FAR
    return z.to(dtype), torch.rand(t, generator=g, device="cuda", dtype=torch.float64)


def share(cut):
    """A top_p that lies a fraction `cut` below what the top and the first cluster weigh."""
    near, far = 1800 * math.exp(NEAR / TEMPERATURE), 1900 * math.exp(FAR / TEMPERATURE)
    return (1 + near) / (1 + near + far) * (1 - cut)


# one block and several (where rows are few and longer than 65536 entries)
@pytest.mark.parametrize("t,v", [(4, 3701), (3, 9001), (2, 70001), (5, 140003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_min_p_between_the_cut_and_its_estimate(t, v, dtype):
    z, u = clustered(t, v, dtype, t + v)
    for cut in (0.0009, 0.0013, 0.0018, 0.0022, 0.0025):
        # min_p in the middle between the clusters, just above the far one, and right below and above the near one
        for steps in (25.0, 39.5, 11.5, 9.0, 45.0):
            check(z, u, TEMPERATURE, top_p=share(cut), min_p=2.0 ** (-steps / 99.5), most_unsure=0)
        check(z, u, TEMPERATURE, top_p=share(cut), most_unsure=0)


def test_settings_per_row_over_clusters():
    t, v = 120, 9001  # one block per row
    z, u = clustered(t, v, torch.float32, 1)
    top_p = torch.tensor([share(0.0008 + 0.00002 * i) for i in range(t)], device="cuda", dtype=torch.float32)
    min_p = torch.tensor([2.0 ** (-(8 + 0.3 * i) / 99.5) for i in range(t)], device="cuda", dtype=torch.float32)
    check(z, u, TEMPERATURE, top_p=top_p, min_p=min_p, most_unsure=0)


def test_a_long_row_over_many_steps():
    # 80% of the weight in one entry, some thousands spread over forty steps near 2^-20, and a quarter of a million right behind
    # them: the estimate is off by three steps and only the narrowest window has room for its entries
    rng = np.random.default_rng(0)
    step = np.concatenate([[0.0], rng.uniform(1950, 1990, 9186), np.full(267447, 1995.97)])
    z = torch.from_numpy(-step * STEP).float().cuda()
    z = z[torch.randperm(len(z), generator=gen(2), device="cuda")][None, :].expand(8, -1).contiguous()
    # (u in the top entry's share, wherever it lies among the others: the other weights are too close to the bound for a token)
    u = torch.linspace(0.25, 0.75, 8, device="cuda", dtype=torch.float64)
    for top_p in (0.79975, 0.8, 0.80025, 0.8005):
        for min_p in (1.1155e-6, 1.12e-6, 1.10e-6, 1.14e-6):
            check(z[:2], u[:2], top_p=top_p, min_p=min_p, most_unsure=0)
    tokens, logs = check(z, u, top_p=0.80025, min_p=1.1155e-6, most_unsure=0)
    # the same rows, one block each
    many = oz.sample(z[:1].expand(104, -1).contiguous(), u.repeat(13), top_p=0.80025, min_p=1.1155e-6)
    assert torch.equal(many[0], tokens.repeat(13)) and torch.equal(many[1], logs.repeat(13))
