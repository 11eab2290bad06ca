"""The kernels' sources hold nothing that no call reaches (no GPU)."""
import glob
import os
import re

from generative_recommender_ranking_gb300 import build as bld


def test_every_device_function_has_a_caller():
    text = "\n".join(re.sub(r"//[^\n]*", "", open(f).read()) for f in sorted(glob.glob(os.path.join(bld.CSRC, "*.cu*"))))
    names = set(re.findall(r"__forceinline__[\w\s:<>,]*?\b(\w+)\(", text)) | set(re.findall(r"__noinline__[\w\s:<>,]*?\b(\w+)\(", text))
    assert len(names) > 50
    alone = sorted(n for n in names if len(re.findall(rf"\b{n}\b", text)) < 2)
    assert not alone, alone
