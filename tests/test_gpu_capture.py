"""What the calls on plans and caches with shared heads refuse on a capturing stream leaves nothing
in the graph: a copy from the call's own memory, or a kernel over the caller's tensors, would run
again with every replay."""
import ctypes

import numpy as np
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W

pytestmark = pytest.mark.gpu
HK = 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def captured(call):
    """(status of call() on a capturing stream, nodes it left in the graph)."""
    torch.zeros(1, device="cuda")
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph, nodes = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()
    st = ctypes.c_void_p(stream.cuda_stream)
    assert cu.cuStreamBeginCapture_v2(st, 0) == 0
    try:
        call(stream)
        code = bd.OK
    except bd.RecAttnError as e:
        code = e.code
    assert cu.cuStreamEndCapture(st, ctypes.byref(graph)) == 0  # the capture is still valid
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(nodes)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    return code, nodes.value


@pytest.fixture(scope="module")
def case():
    """A small batch on a plan with shared heads, its forward done, and a gradient's worth of tensors."""
    w = W.mtgr(batch=2, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=8)
    t = gu.device_inputs(w)
    t["k"], t["v"] = t["k"][:, :HK].contiguous(), t["v"][:, :HK].contiguous()
    t["lse"] = torch.empty(t["q"].shape[:2], device="cuda")
    t["o"], t["do"] = torch.empty_like(t["q"]), torch.randn_like(t["q"])
    t["w"] = w
    with bd.rec_attn_plan_grouped(gu.params_for(w), HK, t["off_h"], t["off_d"], t["t"], t["ty"]) as plan:
        t["plan"] = plan
        bd.rec_attn_fwd(plan, t["q"], t["k"], t["v"], t["o"], t["lse"])
        torch.cuda.synchronize()
        yield t


def test_what_is_captured_is_counted(case):
    x, w = torch.randn(40, 64, device="cuda"), torch.ones(1, 64, device="cuda")
    y = torch.empty_like(x)
    bd.rec_attn_layernorm_fwd(x, w, None, y)
    assert captured(lambda s: bd.rec_attn_layernorm_fwd(x, w, None, y, stream=s)) == (bd.OK, 1)


def test_compressed_forward(case):
    c, w = case, case["w"]
    from test_gpu_compress import _hist_ranges
    hb, hl = _hist_ranges(w)
    segs = [(64, 1), (-1, 2)]
    n = int(bd.rec_attn_compress_lengths(w.offsets, hb, hl, segs)[-1])
    x = torch.full((n,) + c["q"].shape[1:], 7.0, dtype=torch.bfloat16, device="cuda")
    t, ty = torch.full((n,), -7, device="cuda"), torch.full((n,), 7, dtype=torch.int8, device="cuda")
    call = lambda s=None: bd.rec_attn_fwd_compress(c["plan"], c["q"], c["k"], c["v"], hb, hl, segs, x, t, ty, stream=s)
    assert captured(call) == (bd.ERR_UNSUPPORTED, 0)
    torch.cuda.synchronize()
    assert (x == 7).all() and (t == -7).all() and (ty == 7).all()
    call()  # the same call outside the capture is taken
    torch.cuda.synchronize()
    assert bd.rec_attn_device_status(c["plan"]) == bd.OK and torch.isfinite(x).all() and not (t == -7).any()


def test_fused_backward(case):
    c = case
    f = dict(out_gate=torch.randn_like(c["q"]), k_norm_weight=torch.ones(HK, c["k"].shape[2], device="cuda"))
    o, lse = torch.empty_like(c["o"]), torch.empty_like(c["lse"])
    bd.rec_attn_fwd_fused(c["plan"], c["q"], c["k"], c["v"], o, lse, **f)
    torch.cuda.synchronize()
    outs = dict(dout_gate=torch.full_like(c["q"], 7.0), dk_norm_weight=torch.full_like(f["k_norm_weight"], 7.0))
    dq, dk, dv = (torch.full_like(c[x], 7.0) for x in "qkv")
    call = lambda s=None: bd.rec_attn_bwd_fused(c["plan"], c["q"], c["k"], c["v"], o, lse, c["do"], dq, dk, dv, stream=s, **f,
                                                **outs)
    assert captured(call) == (bd.ERR_UNSUPPORTED, 0)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in (dq, dk, dv, *outs.values()))
    call()  # the same call outside the capture is taken
    torch.cuda.synchronize()
    assert bd.rec_attn_device_status(c["plan"]) == bd.OK
    assert all(torch.isfinite(x).all() and not (x == 7).all() for x in (dq, dk, dv, *outs.values()))


def test_the_other_calls(case):
    c, w = case, case["w"]
    dq, dk, dv = (torch.empty_like(c[x]) for x in "qkv")
    gate = torch.ones_like(c["q"])
    f32 = bd.make_params(8, 64, dtype="fp32")
    q1, k1, o1 = c["q"][:2].float(), c["k"][:2].float(), torch.empty_like(c["q"][:2]).float()
    hist = (w.offsets, c["t"], c["ty"], c["k"].float(), c["v"].float(), 1)
    cands = np.arange(len(w.offsets), dtype=np.int64)
    with bd.rec_attn_cache_create_grouped(f32, HK, *hist) as cache:
        for call in (
                lambda s: bd.rec_attn_plan_grouped(gu.params_for(w), HK, c["off_h"], c["off_d"], c["t"], c["ty"], stream=s),
                lambda s: bd.rec_attn_cache_create_grouped(f32, HK, *hist, stream=s),
                lambda s: bd.rec_attn_cache_score(cache, cands, c["t"], q1, k1, k1, o1, stream=s),
                lambda s: bd.rec_attn_fwd(c["plan"], c["q"], c["k"], c["v"], c["o"], c["lse"], stream=s),
                lambda s: bd.rec_attn_fwd_fused(c["plan"], c["q"], c["k"], c["v"], c["o"], c["lse"], stream=s,
                                                out_gate=gate),
                lambda s: bd.rec_attn_bwd(c["plan"], c["q"], c["k"], c["v"], c["o"], c["lse"], c["do"], dq, dk, dv, stream=s)):
            assert captured(call) == (bd.ERR_UNSUPPORTED, 0)
