"""The INT8 products with scales and the linear cross entropy without a GPU: argument checks (which come before any
HIP call), workspace sizes, and what the compiler makes of their kernels."""
import os
import re
import shutil
import subprocess

import pytest

import rns_emulated_fp64_amd as oz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
P = 1 << 20  # a pointer that is never followed


def with_arg(good, i, value):
    return good[:i] + (value,) + good[i + 1:]


def test_i8gemm_refusals():
    #       t  n  k   A  lda sa B  ldb sb bias C ldc type
    good = (4, 6, 16, P, 16, P, P, 16, P, 0, P, 6, oz.BF16)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 15), (5, 0), (6, 0), (7, 15), (8, 0), (10, 0), (11, 5), (12, 3),
                   (12, -1)]:
        assert oz.ozaki2_i8gemm(*with_arg(good, i, bad)) == -(i + 1), i
        assert oz.ozaki2_i8gemm_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), i
    assert oz.ozaki2_i8gemm(*with_arg(with_arg(good, 2, 1 << 17), 4, 1 << 17)[:7], 1 << 17, *good[8:]) == 3
    assert oz.ozaki2_i8gemm(1 << 31, *good[1:]) == 3
    # empty products touch nothing
    assert oz.ozaki2_i8gemm(0, 6, 16, 0, 16, 0, 0, 16, 0, 0, 0, 6, oz.FP32) == 0
    assert oz.ozaki2_i8gemm(4, 0, 16, 0, 16, 0, 0, 16, 0, 0, 0, 1, oz.FP16) == 0
    # a product that needs a workspace
    t, n, k = 128, 512, 65536
    need = oz.ozaki2_i8gemm_workspace_size(t, n, k)
    assert need > 0
    sliced = (t, n, k, P, k, P, P, k, P, 0, P, n, oz.FP32)
    assert oz.ozaki2_i8gemm_ws(*sliced, 0, need) == -14
    assert oz.ozaki2_i8gemm_ws(*sliced, P + 64, need) == -14
    assert oz.ozaki2_i8gemm_ws(*sliced, P, need - 1) == 2


def test_i8linear_refusals():
    #       t  n  k   X  ldx xtype    B  ldb sb bias C ldc type
    good = (9, 6, 16, P, 16, oz.FP16, P, 16, P, 0, P, 6, oz.BF16)
    for i, bad in [(0, -1), (1, -1), (2, -1), (3, 0), (4, 15), (5, 7), (6, 0), (7, 15), (8, 0), (10, 0), (11, 5), (12, 3)]:
        assert oz.ozaki2_i8linear(*with_arg(good, i, bad)) == -(i + 1), i
        assert oz.ozaki2_i8linear_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), i
    need = oz.ozaki2_i8linear_workspace_size(9, 6, 16)
    assert need > 0 and oz.ozaki2_i8linear_workspace_size(1, 6, 16) == 0  # one row is quantised in the product
    assert oz.ozaki2_i8linear_ws(*good, 0, need) == -14
    assert oz.ozaki2_i8linear_ws(*good, P + 8, need) == -14
    assert oz.ozaki2_i8linear_ws(*good, P, need - 1) == 2
    assert oz.ozaki2_i8linear(0, 6, 16, 0, 16, 0, 0, 16, 0, 0, 0, 6, 0) == 0


def test_quantize_rows_refusals():
    good = (3, 8, P, 8, oz.FP32, P, 8, P)
    for i, bad in [(0, -1), (1, -1), (2, 0), (3, 7), (4, 9), (5, 0), (6, 7), (7, 0)]:
        assert oz.ozaki2_quantize_rows(*with_arg(good, i, bad)) == -(i + 1), i
    assert oz.ozaki2_quantize_rows(1 << 31, *good[1:]) == 3
    assert oz.ozaki2_quantize_rows(0, 8, 0, 8, 0, 0, 8, 0) == 0


def test_xent_refusals():
    #       t  v  d   X  ldx W  ldw type     y  ignore loss lse
    good = (5, 9, 16, P, 16, P, 16, oz.BF16, P, -100, P, P)
    for i, bad in [(0, -1), (1, -1), (1, 0), (2, -1), (3, 0), (4, 15), (5, 0), (6, 15), (7, oz.FP32), (7, -1), (8, 0),
                   (10, 0), (11, 0)]:
        assert oz.ozaki2_xent(*with_arg(good, i, bad)) == -(i + 1), i
        assert oz.ozaki2_xent_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), i
    need = oz.ozaki2_xent_workspace_size(5, 9, 16)
    assert need > 0
    assert oz.ozaki2_xent_ws(*good, 0, need) == -13
    assert oz.ozaki2_xent_ws(*good, P + 128, need) == -13
    assert oz.ozaki2_xent_ws(*good, P, need - 1) == 2
    assert oz.ozaki2_xent(1 << 31, *good[1:]) == 3
    assert oz.ozaki2_xent(0, 0, 16, 0, 16, 0, 16, 0, 0, 0, 0, 0) == 0


def test_i8xent_refusals():
    #       t  v  k   A  lda sa B  ldb sb y  ignore loss lse
    good = (5, 9, 16, P, 16, P, P, 16, P, P, -100, P, P)
    for i, bad in [(0, -1), (1, 0), (2, -1), (3, 0), (4, 15), (5, 0), (6, 0), (7, 15), (8, 0), (9, 0), (11, 0), (12, 0)]:
        assert oz.ozaki2_i8xent(*with_arg(good, i, bad)) == -(i + 1), i
        assert oz.ozaki2_i8xent_ws(*with_arg(good, i, bad), P, 1 << 30) == -(i + 1), i
    need = oz.ozaki2_i8xent_workspace_size(5, 9, 16)
    assert oz.ozaki2_i8xent_ws(*good, 0, need) == -14
    assert oz.ozaki2_i8xent_ws(*good, P, need - 1) == 2
    k = 1 << 17
    assert oz.ozaki2_i8xent(5, 9, k, P, k, P, P, k, P, P, -100, P, P) == 3


def test_xent_grad_refusals():
    #       t  v  d   X  ldx W  ldw type     y  ignore lse g dX lddx dW lddw
    good = (5, 9, 16, P, 16, P, 16, oz.FP16, P, -100, P, P, P, 16, P, 16)
    for i, bad in [(0, -1), (1, -1), (1, 0), (2, -1), (3, 0), (4, 15), (5, 0), (6, 15), (7, 2), (8, 0), (10, 0), (11, 0),
                   (13, 15), (15, 15)]:
        assert oz.ozaki2_xent_grad(*with_arg(good, i, bad)) == -(i + 1), i
        assert oz.ozaki2_xent_grad_ws(*with_arg(good, i, bad), P, 1 << 40) == -(i + 1), i
    need = oz.ozaki2_xent_grad_workspace_size(5, 9, 16)
    assert need > oz.ozaki2_xent_grad_workspace_size(5, 9, 16, want_dx=False) > 0
    assert oz.ozaki2_xent_grad_workspace_size(5, 9, 16, False, False) == 0
    assert oz.ozaki2_xent_grad_ws(*good, 0, need) == -17
    assert oz.ozaki2_xent_grad_ws(*good, P + 16, need) == -17
    assert oz.ozaki2_xent_grad_ws(*good, P, need - 1) == 2
    # nothing wanted, nothing done; a pitch of an output that is skipped does not matter
    assert oz.ozaki2_xent_grad(*good[:12], 0, 0, 0, 0) == 0


def test_limits():
    # sizes whose launches or row numbers would leave their range are refused, with workspaces of 0 bytes
    t, n = 1 << 29, 1 << 23
    gemm = (P, 16, P, P, 16, P, 0, P)
    assert oz.ozaki2_i8gemm(t, 6, 16, *gemm, 6, oz.BF16) == 3
    assert oz.ozaki2_i8gemm(4, n, 16, *gemm, n, oz.BF16) == 3
    assert oz.ozaki2_i8linear(t, 6, 16, P, 16, oz.BF16, *gemm[3:], 6, oz.BF16) == 3
    assert oz.ozaki2_i8linear(4, n, 16, P, 16, oz.BF16, *gemm[3:], n, oz.BF16) == 3
    assert oz.ozaki2_xent(5, n, 16, P, 16, P, 16, oz.BF16, P, -100, P, P) == 3
    assert oz.ozaki2_i8xent(5, n, 16, P, 16, P, P, 16, P, P, -100, P, P) == 3
    for a, b, d in ((t, 9, 16), (5, n, 16), (5, 9, 1 << 22)):
        assert oz.ozaki2_xent_grad(a, b, d, P, d, P, d, oz.FP16, P, -100, P, P, P, d, P, d) == 3
        assert oz.ozaki2_xent_grad_workspace_size(a, b, d) == 0
    assert oz.ozaki2_i8gemm_workspace_size(t, 6, 15) == oz.ozaki2_i8linear_workspace_size(9, n, 16) == 0
    assert oz.ozaki2_xent_workspace_size(5, n, 16) == oz.ozaki2_i8xent_workspace_size(5, n, 16) == 0


def test_workspace_sizes():
    # sizes grow with the problem, stay small beside the logits, and are 0 for what is refused
    big = oz.ozaki2_xent_workspace_size(8192, 128000, 4096)
    assert 0 < big <= 8192 * (128000 // 64 + 16) * 8  # 1/32 of the logits
    assert oz.ozaki2_xent_workspace_size(1 << 20, 128000, 4096) < 1 << 29  # tokens are taken in runs
    grad = oz.ozaki2_xent_grad_workspace_size(8192, 128000, 4096)
    assert grad < 3 << 30
    assert oz.ozaki2_xent_grad_workspace_size(65536, 128000, 4096) < 10 << 30
    for bad in ((-1, 5, 5), (5, -1, 5), (5, 5, -1), (1 << 31, 5, 5)):
        assert oz.ozaki2_i8gemm_workspace_size(*bad) == 0
        assert oz.ozaki2_i8linear_workspace_size(*bad) == 0
        assert oz.ozaki2_xent_workspace_size(*bad) == 0
        assert oz.ozaki2_xent_grad_workspace_size(*bad) == 0
    assert oz.ozaki2_i8gemm_workspace_size(5, 5, 1 << 17) == 0


def compiled(source, *more):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    src = os.path.join(ROOT, "rns_emulated_fp64_amd", "csrc", source)
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "--cuda-device-only", *more, src]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert out.returncode == 0, out.stderr[-2000:]
    return out


@pytest.mark.parametrize("source", ["products.hip", "xent.hip"])
def test_kernels_keep_their_state_in_registers(source):
    """No kernel spills to scratch: in the tiles' main loops a scratch load's counter wait would also wait for every
    copy in flight. Their LDS lets as many blocks share a compute unit as their design counts on."""
    out = compiled(source, "-c", "-Rpass-analysis=kernel-resource-usage", "-o", os.devnull)
    kernels, cur = {}, None
    for line in out.stderr.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            cur = kernels.setdefault(m.group(1), {})
        m = re.search(r"remark:\s+([A-Za-z ]+?)(?: \[[^\]]+\])?: (\d+)", line)
        if m and cur is not None:
            cur[m.group(1).strip()] = int(m.group(2))
    assert len(kernels) > 10
    for name, r in kernels.items():
        assert r.get("VGPRs Spill", 0) == 0 and r.get("ScratchSize", 0) == 0, (name, r)
        if "k_tile_p" in name:
            assert r["LDS Size"] in (160 * 1024, 80 * 1024), (name, r)
            assert r["Occupancy"] == (1 if r["LDS Size"] == 160 * 1024 else 2), (name, r)


@pytest.mark.parametrize("source", ["products.hip", "xent.hip"])
def test_m0_is_written_only_by_the_copies(source):
    """The tiles set M0 (the LDS address of a copy) in one inline-asm statement and issue the copy in the next, which
    is sound only if the compiler writes M0 nowhere in these kernels itself. And the file holds no packed FP32."""
    lines = compiled(source, "-S", "-o", "-").stdout.splitlines()
    assert not [l for l in lines if re.match(r"\s+v_pk_(add|mul|fma)_f32", l)]
    starts = [i for i, l in enumerate(lines) if re.match(r"^_ZN3oz28k_tile_[ps]\S*:", l)]
    assert len(starts) >= 8
    for start in starts:
        end = next(i for i in range(start, len(lines)) if "s_endpgm" in lines[i])
        in_asm, asm_writes = False, 0
        for l in lines[start:end]:
            t = l.strip()
            if t.startswith(";;#ASMSTART"):
                in_asm = True
            elif t.startswith(";;#ASMEND"):
                in_asm = False
            elif re.match(r"^s_\w+\s+m0\b", t):
                assert in_asm, (lines[start], t)
                asm_writes += 1
        assert asm_writes >= 4, lines[start]
