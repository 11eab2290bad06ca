"""Every helper of the PTX header is called by some kernel, and those of pairs of CTAs have one form (no GPU)."""
import os
import re

from generative_recommender_ranking_gb300 import build as bld


def _text():
    return {os.path.basename(f): re.sub(r"//.*", "", open(f).read()) for f in bld._sources() + bld._headers()}


def test_every_ptx_helper_is_called():
    text = _text()
    helpers = set(re.findall(r"__forceinline__ [\w ]+?\b(\w+)\(", text["ptx_sm103.cuh"]))
    assert len(helpers) > 40
    everything = "\n".join(text.values())
    unused = [h for h in sorted(helpers) if len(re.findall(r"\b%s\b" % h, everything)) < 2]
    assert not unused, unused


def test_pairs_have_one_form():
    """The two-CTA helpers have no single-CTA branch, which no kernel would take."""
    for name, src in _text().items():
        assert "CG == 1" not in src and not re.search(r"template <[^>]*\bint CG\b", src), name
