"""How the pipelined kernels leave a wait that gives up, read from their sources (no GPU): such a wait
cannot be made to run out in a kernel at work."""
import glob
import os
import re

import pytest

from generative_recommender_ranking_gb300 import build as bld

SOURCES = sorted(glob.glob(os.path.join(bld.CSRC, "*.cu")))


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, at):
    """The text of the braces that open at or after `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced")


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_waits_of_whole_warps_are_voted_on(path):
    """bounded_wait answers each lane for itself, so it stands in single-thread code alone: a branch of
    one lane, or a wrapper that such code calls."""
    text = code(path)
    for m in re.finditer(r"\bbounded_wait\(", text):
        before = text[:m.start()]
        line = before[before.rfind("\n") + 1:]
        wrapper = re.search(r"bool (wait_bar|bw_wait)\([^{}]*\{\s*return $", before)
        one_lane = any(m.start() < h.start() + len(block(text, h.start())) + 40 and h.start() < m.start()
                       for h in re.finditer(r"if \(lane == 0\) \{", text))
        assert wrapper or one_lane or "if (threadIdx.x == " in line, (os.path.basename(path), line.strip())
    # the wrappers' own whole-warp forms vote
    for name, body in re.findall(r"bool (\w+_warp)\([^{}]*\)\s*(\{[^}]*\})", text):
        assert "bounded_wait_warp(" in body, name


def test_scoring_waits_for_its_copies():
    """The few-row scoring kernel's loading thread waits for its last copies after its loop, however that
    ended: consumers that gave up on a tile write their outputs over the stages it lands in."""
    text = code(os.path.join(bld.CSRC, "score.cu"))
    loader = block(text, text.index("if (warp == kScoreWarps)"))
    at = loader.index("for (")  # the tiles
    loop = block(loader, at)
    assert "tma_load_2d(" in loop and "tma_load_2d(" not in loader.replace(loop, "")
    after = loader[loader.index(loop) + len(loop):]
    drain = re.search(r"for \(int j = max\(0, k - (\w+)\); j < k; \+\+j\)\s*bounded_drain\(s_full \+ j % \1, \(j / \1\) & 1, ", after)
    assert drain and drain.group(1) == "kScoreStages"
    # those waits cover every copy that may still be in flight: all but the ones whose stage was refilled
    for n in range(20):
        for stages in (2, 3, 4):
            last_use = {j % stages: (j // stages) & 1 for j in range(n)}
            assert {j % stages: (j // stages) & 1 for j in range(max(0, n - stages), n)} == last_use
