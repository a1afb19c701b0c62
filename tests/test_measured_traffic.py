"""The DRAM traffic that bench.py reports was measured on the kernel sources that are there."""
import os

import bench


def test_the_captured_traffic_is_of_these_sources():
    csrc = os.path.join(bench.ROOT, "dense_gqa_decoder_gb300", "csrc")
    got, sha = bench.traffic_from_profiles([os.path.join(csrc, f) for f in ("k2_mega.cu", "k2_common.cuh", "k2_kernels.h")],
                                           "mega_decode")
    assert got is not None, f"no capture of source_sha={sha} in profiles/traffic.txt"
