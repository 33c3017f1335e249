"""The benchmark reports the fused GEMMs' memory traffic only while the committed counters are
those of the sources in the tree: they are, and every header of the kernels' code counts."""

import os
import re

import bench


def test_recorded_traffic_is_of_these_sources():
    assert bench.recorded_traffic() is not None, "retake the counters of profiles/gemm_nf4_workload2_traffic.md"


def test_every_header_of_the_kernels_counts():
    root = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "bit_quantized_lora_nf4_amd", "csrc")
    text = open(os.path.join(root, "gemm.hip")).read()
    used = set(re.findall(r'#include "(\w+\.h)"', text)) - {"qlora_internal.h"}  # declarations alone
    assert used == {os.path.basename(p) for p in bench.GEMM_SOURCES if p.endswith(".h")}
