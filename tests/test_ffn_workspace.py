"""Parts of the summed axis that the feed-forward products ask a workspace for: as many as the header allows (no GPU; the
rules are called as the library has them)."""
import subprocess

import pytest

from generative_recommender_ranking_gb300 import build as bld

MAIN = r"""
#include <cstdio>
#include <initializer_list>
namespace recattn {
int dense_splits(int M, int N, int kblocks, double block_us, int num_sms);
int dense32_splits(int M, int N, int kblocks, int num_sms);
}
int main() {
  const int blocks[] = {1, 2, 3, 7, 16, 64, 304, 1000, 5001, 33000000};
  for (int sms : {8, 132, 152})
    for (int m = 8; m <= 140000; m = m * 3 / 2 + 1)
      for (int n = 8; n <= 70000; n = n * 2 + 1)
        for (int k : blocks)
          printf("%d %d %d %d %d %d %d\n", sms, m, n, k, recattn::dense_splits(m, n, k, 0.4, sms),
                 recattn::dense_splits(m, n, k, 0.5, sms), recattn::dense32_splits(m, n, k, sms));
}
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    import glob
    import os
    bld.build()
    d = tmp_path_factory.mktemp("splits")
    (d / "main.cpp").write_text(MAIN)
    objects = sorted(glob.glob(os.path.join(bld.OUT_DIR, "*.o")))
    subprocess.run([bld._nvcc(), *bld.ARCH, "-std=c++17", "-o", str(d / "main"), str(d / "main.cpp"), *objects], check=True,
                   capture_output=True)
    out = subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_parts_are_within_the_documented_bounds(splits):
    for sms, m, n, k, bf16, e4m3, fp32 in splits:
        assert 1 <= bf16 <= min(64, k) and 1 <= e4m3 <= min(64, k), (sms, m, n, k)
        assert 1 <= fp32 <= max(1, min(sms // 2, k // 4)), (sms, m, n, k)
    # the bounds are reached, so the header's figures are not larger than they need be
    assert max(s[4] for s in splits) == 64
    assert max(s[6] for s in splits if s[0] == 152) == 76
