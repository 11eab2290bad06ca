"""The bf16 backward's range of softmax scales: it keeps the rows' constants in the scores' unit."""
import numpy as np
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def run(scale, dtype="bf16", lens=(200, 1, 130), d=64):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    T = int(off[-1])
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(T, 2, d, generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda() for _ in range(4))
    t, ty = torch.arange(T, device="cuda"), torch.full((T,), W.HIST, dtype=torch.int8, device="cuda")
    o, dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, q, k, v))
    lse = torch.empty(T, 2, device="cuda")
    p = bd.make_params(2, d, dtype=dtype, use_rope=False, hist_bidirectional=True, softmax_scale=scale)
    with bd.rec_attn_plan(p, off, torch.from_numpy(off).cuda(), t, ty) as plan:
        bd.rec_attn_fwd(plan, q, k, v, o, lse)
        try:
            bd.rec_attn_bwd(plan, q, k, v, o, lse, do, dq, dk, dv)
        except bd.RecAttnError as e:
            return e.code, None
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    # scores of next to nothing: every key of a request has the same weight, and dV_j = mean_i dO_i
    want = torch.cat([do[a:b].double().mean(0, keepdim=True).expand(int(b - a), -1, -1) for a, b in zip(off[:-1], off[1:])])
    return bd.OK, float((dv.double() - want).norm() / want.norm())


@pytest.mark.parametrize("scale", [1e-37, 1e-31, 1e31, 3e38])
def test_outside(scale):
    assert run(scale) == (bd.ERR_UNSUPPORTED, None)
    assert run(scale, "fp32")[0] == bd.OK


@pytest.mark.parametrize("scale", [2e-30, 1e-10])
def test_smallest(scale):
    """P is rounded to bf16 once (2^-9 of it), dV once: 2^-8 and some."""
    code, err = run(scale)
    assert code == bd.OK and err <= 2 * 2.0 ** -8
