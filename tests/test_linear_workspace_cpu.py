"""Workspaces of products whose rows are copied to aligned ones, a run of channels at a time, without a GPU.

Such a product holds the copied rows of A, those of one run of B, and the planes of the slices of k. Every run, the last
and shorter one too, is an aligned product of its own and cuts k into as many slices as its own sizes ask for, so its
planes are what ozaki2_i8gemm_workspace_size gives for it alone."""
import random

import pytest

import rns_emulated_fp64_amd as oz


def up(v, to):
    return -(-v // to) * to


def needed(t, n, k, rows_of_a):
    """Bytes that the runs of a product of t > 16 rows with an odd k write."""
    pitch = (up(k, 128) // 128 | 1) * 128
    run = max((96 << 20) // pitch // 256 * 256, 256)
    run = min(run, n)
    planes = max(oz.ozaki2_i8gemm_workspace_size(t, r, up(k, 16)) for r in (run, n % run) if r)
    return (up(t * pitch, 256) if rows_of_a else 0) + up(run * pitch, 256) + planes


def quantised(t, k):
    return up(t * (up(k, 128) // 128 | 1) * 128, 256) + up(4 * t, 256)


@pytest.mark.parametrize("t,n,k", [(256, 12100, 8193), (26, 22441, 4391), (1024, 4992, 20001), (17, 600, 131071),
                                   (2048, 2 * 4864 + 70, 20001), (300, 700, 1001)])
def test_every_run_has_room_for_its_planes(t, n, k):
    assert oz.ozaki2_i8gemm_workspace_size(t, n, k) >= needed(t, n, k, True)
    assert oz.ozaki2_i8linear_workspace_size(t, n, k) >= quantised(t, k) + needed(t, n, k, False)


@pytest.mark.parametrize("tile", ["", "s22", "s42", "p4", "p8", "any"])
def test_random_sizes_with_a_short_last_run(tile, monkeypatch):
    monkeypatch.setenv("OZ2_LINEAR_TILE", tile)
    rng = random.Random(1)
    for _ in range(2000):
        k = int(2 ** rng.uniform(8, 17)) | 1
        run = max((96 << 20) // ((up(k, 128) // 128 | 1) * 128) // 256 * 256, 256)
        n = run * rng.randint(1, 3) + int(2 ** rng.uniform(0, 10))
        t = int(2 ** rng.uniform(4.2, 13))
        assert oz.ozaki2_i8gemm_workspace_size(t, n, k) >= needed(t, n, k, True), (t, n, k)
        assert oz.ozaki2_i8linear_workspace_size(t, n, k) >= quantised(t, k) + needed(t, n, k, False), (t, n, k)
