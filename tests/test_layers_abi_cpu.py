"""Layers with an epilogue and their gradients without a GPU: argument checks (which come before any HIP call), workspace
sizes, and what the compiler makes of their kernels."""
import os
import random
import re
import shutil
import subprocess

import pytest

import rns_emulated_fp64_amd as oz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
P = 1 << 20  # pointers that are never followed
R = 1 << 30


def with_arg(good, i, value):
    return good[:i] + (value,) + good[i + 1:]


def test_i8gemm_act_refusals():
    #       t  n  k   A  ldA sa B  ldb sb b  act res ldr C ldc type
    good = (4, 6, 16, P, 16, P, P, 16, P, 0, 1, R, 6, P, 6, oz.BF16)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 15), (5, 0), (6, 0), (7, 15), (8, 0), (10, -1), (10, 5), (11, P),
                   (11, P + 40), (12, 5), (13, 0), (14, 5), (15, 3), (15, -1)]:
        assert oz.ozaki2_i8gemm_act(*with_arg(good, i, bad)) == -(i + 1), (i, bad)
        assert oz.ozaki2_i8gemm_act_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), (i, bad)
    # the first argument that is wrong is named
    assert oz.ozaki2_i8gemm_act(*with_arg(with_arg(good, 10, 9), 2, -1)) == -3
    assert oz.ozaki2_i8gemm_act(*with_arg(with_arg(good, 14, 1), 10, 9)) == -11
    assert oz.ozaki2_i8gemm_act(1 << 31, *with_arg(good, 11, 0)[1:]) == 3
    assert oz.ozaki2_i8gemm_act(0, 6, 16, 0, 16, 0, 0, 16, 0, 0, 4, 0, 0, 0, 6, oz.FP32) == 0
    t, n, k = 128, 512, 65536
    need = oz.ozaki2_i8gemm_workspace_size(t, n, k)
    sliced = (t, n, k, P, k, P, P, k, P, 0, 2, 0, 0, P, n, oz.FP32)
    assert oz.ozaki2_i8gemm_act_ws(*sliced, 0, need) == -17
    assert oz.ozaki2_i8gemm_act_ws(*sliced, P + 64, need) == -17
    assert oz.ozaki2_i8gemm_act_ws(*sliced, P, need - 1) == 2


def test_i8linear_act_refusals():
    #       t  n  k   X  ldx xtype    B  ldb sb b  act res ldr C ldc type
    good = (9, 6, 16, P, 16, oz.FP16, P, 16, P, 0, 3, R, 6, P, 6, oz.BF16)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 15), (5, 7), (6, 0), (7, 15), (8, 0), (10, 5), (11, P), (12, 5), (13, 0),
                   (14, 5), (15, 3)]:
        assert oz.ozaki2_i8linear_act(*with_arg(good, i, bad)) == -(i + 1), (i, bad)
        assert oz.ozaki2_i8linear_act_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), (i, bad)
    need = oz.ozaki2_i8linear_workspace_size(9, 6, 16)
    assert oz.ozaki2_i8linear_act_ws(*good, 0, need) == -17
    assert oz.ozaki2_i8linear_act_ws(*good, P, need - 1) == 2
    # (with the residual's last byte right before the output, and its first right behind it)
    rows = 2 * 9 * 6
    assert oz.ozaki2_i8linear_act_ws(*with_arg(good, 11, P - rows), P, need - 1) == 2
    assert oz.ozaki2_i8linear_act_ws(*with_arg(good, 11, P - rows + 2), P, need - 1) == -12
    assert oz.ozaki2_i8linear_act_ws(*with_arg(good, 11, P + rows), P, need - 1) == 2


def test_linear_refusals():
    #       t  n  k   X  ldx W  ldw type     b  act res ldr Y  ldy ytype    Z  ldz
    good = (5, 9, 16, P, 16, P, 16, oz.BF16, 0, 4, R, 9, P, 9, oz.FP32, P, 9)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 15), (5, 0), (6, 15), (7, oz.FP32), (7, -1), (9, 5), (9, -1), (10, P), (11, 8),
                   (12, 0), (13, 8), (14, oz.FP16), (14, 7), (16, 8)]:
        assert oz.ozaki2_linear(*with_arg(good, i, bad)) == -(i + 1), (i, bad)
        assert oz.ozaki2_linear_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), (i, bad)
    t, n, k = 70, 130, 16384
    need = oz.ozaki2_linear_workspace_size(t, n, k)
    assert need > 0
    sliced = (t, n, k, P, k, P, k, oz.FP16, 0, 0, 0, 0, P, n, oz.FP16, 0, 0)
    assert oz.ozaki2_linear_ws(*sliced, 0, need) == -18
    assert oz.ozaki2_linear_ws(*sliced, P + 128, need) == -18
    assert oz.ozaki2_linear_ws(*sliced, P, need - 1) == 2
    for bad in ((1 << 29, 9, 16), (5, 1 << 23, 16), (5, 9, 1 << 29)):
        assert oz.ozaki2_linear_workspace_size(*bad) == 0
        big = (*bad, P, bad[2], P, bad[2], oz.BF16, 0, 0, 0, 0, P, bad[1], oz.BF16, 0, 0)
        assert oz.ozaki2_linear(*big) == 3
    assert oz.ozaki2_linear(0, 9, 16, 0, 16, 0, 16, oz.BF16, 0, 0, 0, 0, 0, 9, oz.BF16, 0, 0) == 0
    assert oz.ozaki2_linear(5, 0, 16, 0, 16, 0, 16, oz.BF16, 0, 0, 0, 0, 0, 1, oz.BF16, 0, 0) == 0


def test_linear_grad_refusals():
    #       t  n  k   dY ldd X  ldx W  ldw type    act Z  ldz dX lddx dW lddw db
    good = (5, 9, 16, P, 9, P, 16, P, 16, oz.FP16, 2, P, 9, P, 16, P, 16, P)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 8), (5, 0), (6, 15), (7, 0), (8, 15), (9, 2), (10, 5), (11, 0), (12, 8),
                   (14, 15), (16, 15)]:
        assert oz.ozaki2_linear_grad(*with_arg(good, i, bad)) == -(i + 1), (i, bad)
        assert oz.ozaki2_linear_grad_ws(*with_arg(good, i, bad), P, 1 << 40) == -(i + 1), (i, bad)
    need = oz.ozaki2_linear_grad_workspace_size(5, 9, 16)
    for part in ((False, True, True), (True, False, True), (False, False, True)):
        assert need > oz.ozaki2_linear_grad_workspace_size(5, 9, 16, *part) > 0
    assert oz.ozaki2_linear_grad_workspace_size(5, 9, 16, False, False, False) == 0
    assert oz.ozaki2_linear_grad_ws(*good, 0, need) == -19
    assert oz.ozaki2_linear_grad_ws(*good, P + 16, need) == -19
    assert oz.ozaki2_linear_grad_ws(*good, P, need - 1) == 2
    # nothing wanted, nothing done
    assert oz.ozaki2_linear_grad(5, 9, 16, 0, 9, 0, 16, 0, 16, oz.BF16, 1, 0, 9, 0, 0, 0, 0, 0) == 0
    for bad in ((1 << 29, 9, 16), (5, 1 << 22, 16), (5, 9, 1 << 22)):
        assert oz.ozaki2_linear_grad_workspace_size(*bad) == 0
        t, n, k = bad
        assert oz.ozaki2_linear_grad(t, n, k, P, n, P, k, P, k, oz.BF16, 0, 0, 0, P, k, P, k, 0) == 3


def up(v, to):
    return -(-v // to) * to


@pytest.mark.parametrize("tile", ["", "s22", "s42", "p4", "p8", "any"])
def test_every_run_has_room_for_its_planes(tile, monkeypatch):
    """Rows that are no multiple of 16 bytes go in runs of channels, each an aligned product of its own: its planes are
    what the workspace of that product alone is."""
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    rng = random.Random(2)
    for _ in range(1000):
        k = int(2 ** rng.uniform(7, 15)) | 1
        pitch = (up(2 * k, 128) // 128 | 1) * 128
        run = max((96 << 20) // pitch // 256 * 256, 256)
        n = run * rng.randint(0, 2) + int(2 ** rng.uniform(0, 10))
        t = int(2 ** rng.uniform(4.2, 13))
        run = min(run, n)
        planes = max(oz.ozaki2_linear_workspace_size(t, r, up(k, 8)) for r in (run, n % run) if r)
        assert oz.ozaki2_linear_workspace_size(t, n, k) >= up(t * pitch, 256) + up(run * pitch, 256) + planes, (t, n, k)


def test_kernels_keep_their_state_in_registers():
    """No spills; M0, which the tiles' copies set in one statement and use in the next, is written nowhere else; no packed FP32;
    and the LDS leaves room for as many blocks as the tiles count on."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    src = os.path.join(ROOT, "rns_emulated_fp64_amd", "csrc", "linear.hip")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o", "-",
           "-Rpass-analysis=kernel-resource-usage", src]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert out.returncode == 0, out.stderr[-2000:]
    kernels, cur = {}, None
    for line in out.stderr.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            cur = kernels.setdefault(m.group(1), {})
        m = re.search(r"remark:\s+([A-Za-z ]+?)(?: \[[^\]]+\])?: (\d+)", line)
        if m and cur is not None:
            cur[m.group(1).strip()] = int(m.group(2))
    assert len(kernels) > 20
    for name, r in kernels.items():
        assert r.get("VGPRs Spill", 0) == 0 and r.get("ScratchSize", 0) == 0, (name, r)
        if "k_tile_p" in name:
            assert r["Occupancy"] == (1 if r["LDS Size"] == 160 * 1024 else 2), (name, r)
    lines = out.stdout.splitlines()
    assert not [l for l in lines if re.match(r"\s+v_pk_(add|mul|fma)_f32", l)]
    starts = [i for i, l in enumerate(lines) if re.match(r"^_ZN3oz28k_tile_[ps]\S*:", l)]
    assert len(starts) >= 8
    for start in starts:
        end = next(i for i in range(start, len(lines)) if lines[i].startswith("\t.end_amdhsa_kernel") or ".Lfunc_end" in lines[i])
        in_asm = False
        for l in lines[start:end]:
            t = l.strip()
            if t.startswith(";;#ASMSTART"):
                in_asm = True
            elif t.startswith(";;#ASMEND"):
                in_asm = False
            elif re.match(r"^s_\w+\s+m0\b", t):
                assert in_asm, (lines[start], t)
