"""The committed DRAM traffic figures belong to the kernels as they are: bench.py drops a figure whose
sources have changed since its capture, and the roofline of that workload loses its traffic."""
import glob
import os
import re

import pytest

import bench

SUMMARIES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "gateup_swiglu_*.md")))


@pytest.mark.parametrize("path", SUMMARIES, ids=os.path.basename)
def test_traffic_figure_is_of_these_sources(path):
    txt = open(path, encoding="utf-8").read()
    if not re.search(r"^traffic_(bytes_per_launch|per_algorithmic_byte):", txt, re.M):
        pytest.skip("no figure")
    workload = re.match(r"gateup_swiglu_(.*)\.md", os.path.basename(path))[1]
    sources = [f.strip() for f in re.search(r"^kernel_sources:\s*(.+)$", txt, re.M)[1].split(",")]
    traffic, where = bench._profiled_traffic(workload, tuple(sources), 10 ** 9)
    assert traffic is not None and traffic > 0, where

