"""Kernels that hand registers from one warpgroup to another ask the compiler for what they are launched with, and get
it (ptxas's report; no GPU): with any other count the host refuses every call of them."""
import os
import re
import subprocess

import pytest

from generative_recommender_ranking_gb300 import build as bld

SPLIT = {"scaled.cu": r"k_scaled", "dense_tc.cu": r"k_denseILNS_7DenseOpE2E"}  # (DenseOp 2: kDglu)


def test_no_other_source_splits_registers():
    using = {os.path.basename(f) for f in bld._sources() if "more_registers<" in open(f).read()}
    assert using == set(SPLIT)


@pytest.mark.parametrize("source", sorted(SPLIT))
def test_kernels_get_the_registers_that_they_split(source):
    path = os.path.join(bld.CSRC, source)
    assert "__maxnreg__" in open(path).read()
    cmd = [bld._nvcc(), *bld.ARCH, "-O3", "-std=c++17", "-I", bld.INCLUDE, "-I", bld.CSRC, "-Xptxas", "-v", "-c", path, "-o",
           os.devnull]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    counts = re.findall(r"Function properties for (\S+)\n.*\n.*?Used (\d+) registers", log)
    counts = {name: int(n) for name, n in counts if re.search(SPLIT[source], name)}
    assert len(counts) >= 2 and set(counts.values()) == {96}, counts  # 640 threads
