"""bench.py reports the GEMM's counted bytes only while the GEMM's source is the one that was counted."""
import json
import os

import bench


def test_the_counted_gemm_source_is_found():
    path = os.path.join(bench.ROOT, "profiles", "k_gemm_persistent_spread1.0_4096_n16_traffic.txt")
    with open(path) as f:
        assert bench.gemm_source_hash() == json.load(f)["gemm_code_sha256"]
