"""The sampler without a GPU: argument checks, which come before any HIP call, its workspace, and the definition that the GPU tests
compare with on rows that can be worked out by hand."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import rns_emulated_fp64_amd as oz
from sample_util import reference

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

P = 1 << 20  # a pointer that is never followed


def test_refusals():
    #       t  v  l  ldl type     u  temp  ts k  ks top_p ps min_p ms tok log
    good = (3, 9, P, 9, oz.BF16, P, 1.0, 0, 5, 0, 0.9, 0, 0.1, 0, P, 0)
    for i, bad in [(0, -1), (1, -1), (1, 0), (2, 0), (3, 8), (4, 3), (4, -1), (5, 0), (6, -0.5), (6, float("nan")), (10, 1.5),
                   (10, -0.1), (10, float("nan")), (12, 1.1), (12, -0.1), (12, float("nan")), (14, 0)]:
        assert oz.ozaki2_sample(*good[:i], bad, *good[i + 1:]) == -(i + 1), (i, bad)
        assert oz.ozaki2_sample_ws(*good[:i], bad, *good[i + 1:], P, 1 << 30) == -(i + 1), (i, bad)
    v = 100000  # a few long rows need a workspace
    long = (3, v, P, v, *good[4:])
    need = oz.ozaki2_sample_workspace_size(3, v)
    assert oz.ozaki2_sample_ws(*long, 0, need) == -17
    assert oz.ozaki2_sample_ws(*long, P + 8, need) == -17
    assert oz.ozaki2_sample_ws(*long, P, need - 1) == 2
    # a vector's value is not looked at here, and the number beside it does not matter
    vectors = (3, v, P, v, oz.BF16, P, -1.0, P, 5, P, 7.0, P, 7.0, P, P, 0)
    assert oz.ozaki2_sample_ws(*vectors, P, need - 1) == 2
    assert oz.ozaki2_sample(1 << 31, *good[1:]) == 3
    v = 1 << 23
    assert oz.ozaki2_sample(3, v, P, v, *good[4:]) == 3
    assert oz.ozaki2_sample(0, 0, 0, 1, oz.FP32, 0, 1.0, 0, 0, 0, 1.0, 0, 0.0, 0, 0, 0) == 0


def test_workspace():
    one = oz.ozaki2_sample_workspace_size(1, 128000)
    assert 0 < one < 48 << 10 and oz.ozaki2_sample_workspace_size(96, 128000) <= 96 * one
    # a block per row needs none
    assert oz.ozaki2_sample_workspace_size(1, 32000) == oz.ozaki2_sample_workspace_size(1 << 20, 128000) == 0
    for bad in ((0, 5), (-1, 5), (5, 0), (5, -1), (1 << 31, 5), (5, 1 << 23)):
        assert oz.ozaki2_sample_workspace_size(*bad) == 0


def test_the_definition_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))

    def token(u, t=1.0, k=0, p=1.0, m=0.0):
        return reference(l, u, t, k, p, m)[2]

    assert [token(u) for u in (0.0, 0.09, 0.11, 0.49, 0.55, 0.65, 0.95, 1.0)] == [0, 0, 1, 1, 2, 3, 4, 4]
    assert [token(u, k=2) for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]
    assert [token(u, k=3) for u in (0.0, 0.2)] == [0, 1]  # of equal ones the first
    assert [token(u, p=0.65) for u in (0.0, 0.6)] == [1, 3]
    assert [token(u, p=0.75) for u in (0.0, 0.2)] == [0, 1]
    assert token(0.99, p=0.0) == token(0.0, t=0.0) == 1
    assert [token(u, m=0.5) for u in (0.0, 0.99)] == [1, 3]
    index = reference(l, 0.5, 0.5, 0, 1.0, 0.0)
    assert np.allclose(index[1], np.cumsum([1 / 16, 1, 1 / 16, 9 / 16, 1 / 16]))
    assert abs(reference(l, 0.2, 1.0, 2, 1.0, 0.0)[3] - np.log(4 / 7)) < 1e-12
    assert reference([np.nan, 1.0], 0.5, 1.0, 0, 1.0, 0.0) is None
    assert reference([-np.inf, -np.inf], 0.5, 1.0, 0, 1.0, 0.0) is None
    assert reference([np.inf, 1.0, np.inf], 0.6, 1.0, 0, 1.0, 0.0)[2] == 2


@pytest.mark.parametrize("source", ["sample.hip", "norm.hip"])
def test_kernels_keep_their_state_in_registers(source):
    """No spills, no packed FP32, and LDS for two of the sampler's blocks on a compute unit."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    src = os.path.join(ROOT, "rns_emulated_fp64_amd", "csrc", source)
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o", "-",
           "-Rpass-analysis=kernel-resource-usage", src]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    seen = 0
    for line in out.stderr.splitlines():
        m = re.search(r"remark:\s+(VGPRs Spill|ScratchSize|LDS Size)(?: \[[^\]]+\])?: (\d+)", line)
        if m:
            seen += 1
            assert int(m.group(2)) <= (80 << 10 if m.group(1) == "LDS Size" else 0), line
    assert seen > 20
    assert not re.search(r"\n\s+v_pk_(add|mul|fma)_f32", out.stdout)
