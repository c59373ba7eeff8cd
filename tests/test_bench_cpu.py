"""CPU: the profiled traffic that bench.py quotes belongs to the sources it names."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "mixture_experts_layer_top_amd", "csrc")


def test_traffic_hash_covers_the_gemm_it_was_taken_of():
    """Every file that holds a piece of the bf16 MFMA kernel or of the selection that orders its tiles."""
    named = {os.path.basename(f) for f in bench.TRAFFIC_SOURCES}
    assert all(os.path.exists(os.path.join(bench.ROOT, f)) for f in bench.TRAFFIC_SOURCES)
    for f in os.listdir(CSRC):
        text = open(os.path.join(CSRC, f)).read()
        if re.search(r"\bstruct MfmaTile\b|\bvoid gemm_mfma_bf16\(|\bvoid select_block\(|\bint pop_tile_two_class\(", text):
            assert f in named, f


def test_traffic_files_hold_what_the_bench_reads():
    for workload in ("kimi_prefill", "mixtral_prefill"):
        path = os.path.join(bench.ROOT, "profiles", f"gate_up_gemm_{workload}_traffic.md")
        text = open(path).read()
        assert re.search(r"^traffic_bytes_per_launch: \d+$", text, re.M)
        assert re.search(r"^kernel_source_sha256_16: [0-9a-f]{16}$", text, re.M)
