"""Attention whose query heads share key/value heads in groups (rec_attn_plan_grouped,
rec_attn_cache_create_grouped) vs the fp64 oracle run with the shared heads repeated: the
output of a query head is the ungrouped one over its group's keys and values, and dk, dv are
the ungrouped gradients summed over the group.

Tolerances: the roundings are those of the ungrouped kernels (Q', K', P, O, dS and the
gradients in bf16, each at most 2^-8 relative, 2^-9 rms; sums over the group are fp32), so
the bounds are those tests' bounds: outputs max-abs 2e-2 and mean-abs 2e-3 (bf16), 1e-4
(fp32); gradients 1e-2 relative Frobenius and 2e-2 of the largest value (bf16), 1e-5 and
1e-4 (fp32).  The sum over a group's G heads adds their independent errors in quadrature, as
it adds the gradients themselves, so the relative bound does not change with G."""
import numpy as np
import pytest
import torch

import gpu_util as gu
import oracle
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


# name: (workload, key/value heads)
CASES = {
    "cadet_h4_kv2": (lambda: W.cadet(batch=3, n_pairs=150), 2),
    "sort_h8_kv1": (lambda: W.sort(batch=2, n_hist=400, n_cand=40, window=96), 1),
    "sort_h6_kv2": (lambda: W.sort(batch=2, n_hist=261, n_cand=30, window=50, heads=6), 2),
    "mtgr_h8_kv4": (lambda: W.mtgr(batch=3, hist=(150, 300), rt=(20, 60), cand=(10, 30)), 4),
    "mtgr_h5_kv5": (lambda: W.mtgr(batch=2, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=5), 5),
    "window_h8_kv2": (lambda: W.tm20k("window", batch=1, n_hist=3000), 2),
    "cadet_d128_h4_kv1": (lambda: W.cadet(batch=3, n_pairs=150, heads=4, head_dim=128), 1),
    "mtgr_d128_h6_kv3": (lambda: W.mtgr(batch=2, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=6, head_dim=128), 3),
    "many_items_h4_kv2": (lambda: W.cadet(batch=96, n_pairs=150), 2),
    "tiny_fp32_h2_kv1": (lambda: W.tiny_fp32(batch=3, n_hist=200, n_cand=20), 1),
    "one_token_h8_kv2": (lambda: W.sort(batch=3, n_special=0, n_hist=1, n_cand=0, heads=8), 2),
    "tile_edges_h8_kv2": (lambda: W.sort(batch=2, n_special=0, n_hist=128, n_cand=1, heads=8), 2),
}


def grouped(w, hk):
    """The workload with its first hk key/value heads, and with them repeated for the oracle."""
    k, v = np.ascontiguousarray(w.k[:, :hk]), np.ascontiguousarray(w.v[:, :hk])
    g = w.num_heads // hk
    rep = W.Workload(**{**w.__dict__, "k": np.repeat(k, g, axis=1), "v": np.repeat(v, g, axis=1)})
    return W.Workload(**{**w.__dict__, "k": k, "v": v}), rep


def group_sum(x, hk):
    return x.reshape(x.shape[0], hk, -1, x.shape[2]).sum(2)


def plan_of(w, hk, tens, keep=-1, **over):
    return bd.rec_attn_plan_grouped(gu.params_for(w, **over), hk, tens["off_h"], tens["off_d"], tens["t"], tens["ty"],
                                    keep_user_queries=keep)


def nan(x):
    return torch.full_like(x, float("nan"))


def check_out(w, got, ref, what):
    x = gu.to_f64(got)
    assert np.isfinite(x).all(), what
    err = np.abs(x - ref)
    if w.dtype == "bf16":
        assert err.max() <= gu.BF16_MAX_ABS and err.mean() <= gu.BF16_MEAN_ABS, (what, err.max(), err.mean())
    else:
        assert err.max() <= gu.FP32_MAX_ABS, (what, err.max())


def check_grad(w, got, ref, what):
    x = gu.to_f64(got)
    assert np.isfinite(x).all(), what
    rel = np.linalg.norm(x - ref) / max(np.linalg.norm(ref), 1e-30)
    mx = np.max(np.abs(x - ref))
    rt, mt = (1e-2, 2e-2) if w.dtype == "bf16" else (1e-5, 1e-4)
    if np.max(np.abs(ref)) < 1e-6:  # a row with a single visible key: dq and dk vanish
        assert mx <= 1e-3, (what, mx)
    else:
        assert rel <= rt and mx <= mt * np.max(np.abs(ref)), (what, rel, mx)


def device_like(w, a):
    return gu.device_inputs(W.Workload(**{**w.__dict__, "q": a}))["q"]


def upstream(w, seed=11):
    g = np.random.default_rng(seed).standard_normal(w.q.shape).astype(np.float32)
    return W.round_to_bf16_bits(g) if w.dtype == "bf16" else g


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name):
    make, hk = CASES[name]
    w, rep = grouped(make(), hk)
    tens = gu.device_inputs(w)
    g_host = upstream(w)
    dout = device_like(w, g_host)
    out, dq = nan(tens["q"]), nan(tens["q"])
    dk, dv = nan(tens["k"]), nan(tens["k"])
    lse = torch.full((w.total_tokens, w.num_heads), float("nan"), device="cuda")
    with plan_of(w, hk, tens) as plan:
        bd.rec_attn_fwd(plan, tens["q"], tens["k"], tens["v"], out, lse)
        bd.rec_attn_bwd(plan, tens["q"], tens["k"], tens["v"], out, lse, dout, dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    op = gu.oracle_params(w)
    ref, ref_lse = oracle.attention(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, with_lse=True)
    check_out(w, out, ref, "out")
    fin = np.isfinite(ref_lse)
    got_lse = lse.cpu().numpy()
    assert (np.isfinite(got_lse) == fin).all()
    assert np.abs(got_lse[fin] - ref_lse[fin]).max() <= (5e-2 if w.dtype == "bf16" else 1e-4)
    rq, rk, rv = oracle.attention_bwd(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, g_host)
    for what, got, r in (("dq", dq, rq), ("dk", dk, group_sum(rk, hk)), ("dv", dv, group_sum(rv, hk))):
        check_grad(w, got, r, what)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_key_head_per_query_head_is_the_plain_plan(dtype):
    w = W.mtgr(batch=3, hist=(150, 300), rt=(20, 60), cand=(10, 30)) if dtype == "bf16" else W.tiny_fp32(batch=3)
    tens = gu.device_inputs(w)
    got = {}
    for how in ("plain", "grouped"):
        plan = (bd.rec_attn_plan(gu.params_for(w), tens["off_h"], tens["off_d"], tens["t"], tens["ty"])
                if how == "plain" else plan_of(w, w.num_heads, tens))
        with plan:
            out = nan(tens["q"])
            lse = torch.empty((w.total_tokens, w.num_heads), device="cuda")
            bd.rec_attn_fwd(plan, tens["q"], tens["k"], tens["v"], out, lse)
            grads = [nan(out) for _ in range(3)]
            bd.rec_attn_bwd(plan, tens["q"], tens["k"], tens["v"], out, lse, device_like(w, upstream(w)), *grads)
            torch.cuda.synchronize()
            got[how] = [out, lse, *grads]
    for a, b in zip(got["plain"], got["grouped"]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name,keep", [("sort_h8_kv1", 130), ("mtgr_h8_kv4", 0), ("cadet_d128_h4_kv1", 40),
                                       ("tiny_fp32_h2_kv1", 70)])
def test_query_pruned(name, keep):
    make, hk = CASES[name]
    w, rep = grouped(make(), hk)
    tens = gu.device_inputs(w)
    rows = oracle.kept_rows(w.offsets, w.types, keep)
    pruned = np.ones(w.total_tokens, dtype=bool)
    pruned[rows] = False
    g_host = upstream(w)
    dout = device_like(w, g_host)
    dout[torch.from_numpy(pruned).cuda()] = 1e4  # finite garbage at pruned rows
    out, dq, dk, dv = nan(tens["q"]), nan(tens["q"]), nan(tens["k"]), nan(tens["k"])
    lse = torch.full((w.total_tokens, w.num_heads), float("nan"), device="cuda")
    with plan_of(w, hk, tens, keep) as plan:
        bd.rec_attn_fwd(plan, tens["q"], tens["k"], tens["v"], out, lse)
        bd.rec_attn_bwd(plan, tens["q"], tens["k"], tens["v"], out, lse, dout, dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    op = gu.oracle_params(w)
    ref = oracle.attention(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, rows=rows)
    check_out(w, out[torch.from_numpy(rows).cuda()], ref, "out")
    assert torch.isnan(out[torch.from_numpy(pruned).cuda()].float()).all()  # pruned rows stay as they were
    g_ref = g_host.copy()
    g_ref[pruned] = 0
    rq, rk, rv = oracle.attention_bwd(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, g_ref)
    for what, got, r in (("dq", dq, rq), ("dk", dk, group_sum(rk, hk)), ("dv", dv, group_sum(rv, hk))):
        check_grad(w, got, r, what)


@pytest.mark.parametrize("name", ["sort_h6_kv2", "mtgr_d128_h6_kv3", "tiny_fp32_h2_kv1"])
@pytest.mark.parametrize("use_rope", [True, False])
def test_fused_steps(name, use_rope):
    make, hk = CASES[name]
    w, rep = grouped(make(), hk)
    w.rope["use_rope"] = rep.rope["use_rope"] = use_rope
    G, H, d, T = w.num_heads // hk, w.num_heads, w.head_dim, w.total_tokens
    rng = np.random.default_rng(5)
    io = (lambda a: W.round_to_bf16_bits(a.astype(np.float32))) if w.dtype == "bf16" else (lambda a: a.astype(np.float32))
    qw, kw = (1 + 0.2 * rng.standard_normal((h, d)).astype(np.float32) for h in (H, hk))
    qg, kg, og = (io(rng.standard_normal((T, h, d))) for h in (H, hk, H))
    dev = {n: device_like(w, a) for n, a in (("q_gate", qg), ("k_gate", kg), ("out_gate", og))}
    dev["q_norm_weight"], dev["k_norm_weight"] = torch.from_numpy(qw).cuda(), torch.from_numpy(kw).cuda()
    tens = gu.device_inputs(w)
    g_host = upstream(w)
    dout = device_like(w, g_host)
    out = nan(tens["q"])
    lse = torch.empty((T, H), device="cuda")
    grads = {"dq": nan(out), "dk": nan(tens["k"]), "dv": nan(tens["k"]), "dq_gate": nan(out), "dk_gate": nan(tens["k"]),
             "dout_gate": nan(out), "dq_norm_weight": nan(dev["q_norm_weight"]), "dk_norm_weight": nan(dev["k_norm_weight"])}
    with plan_of(w, hk, tens) as plan:
        bd.rec_attn_fwd_fused(plan, tens["q"], tens["k"], tens["v"], out, lse, None, norm_eps=1e-6, **dev)
        bd.rec_attn_bwd_fused(plan, tens["q"], tens["k"], tens["v"], out, lse, dout, grads["dq"], grads["dk"],
                              grads["dv"], None, norm_eps=1e-6, **dev,
                              **{n: x for n, x in grads.items() if n not in ("dq", "dk", "dv")})
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    f = oracle.Fused(q_norm_w=qw.astype(np.float64), k_norm_w=np.repeat(kw, G, axis=0).astype(np.float64), norm_eps=1e-6,
                     q_gate=qg, k_gate=np.repeat(kg, G, axis=1), out_gate=og)
    op = gu.oracle_params(w)
    check_out(w, out, oracle.attention(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, fused=f), "out")
    ref = oracle.attention_bwd_fused(op, w.offsets, w.t, w.types, rep.q, rep.k, rep.v, f, g_host)
    for n in ("dk", "dv", "dk_gate"):
        ref[n] = group_sum(ref[n], hk)
    ref["dk_norm_w"] = ref["dk_norm_w"].reshape(hk, G, d).sum(1)
    rt, mt = (1e-2, 2e-2) if w.dtype == "bf16" else (1e-4, 1e-3)
    for n, got in grads.items():
        r = ref[{"dq_norm_weight": "dq_norm_w", "dk_norm_weight": "dk_norm_w"}.get(n, n)]
        x = got.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(x).all(), n
        rel, mx = np.linalg.norm(x - r) / np.linalg.norm(r), np.max(np.abs(x - r))
        assert rel <= rt and mx <= mt * np.max(np.abs(r)), (n, rel, mx)


def test_compression_epilogue():
    w, rep = grouped(W.tm20k("window", batch=2, n_hist=700), 2)
    tens = gu.device_inputs(w)
    segments = [(256, 1), (-1, 8)]
    hb, hl = np.zeros(2, dtype=np.int64), np.full(2, 700, dtype=np.int64)
    off = bd.rec_attn_compress_lengths(tens["off_h"], hb, hl, segments)
    out = torch.empty_like(tens["q"])
    xs = [torch.full((int(off[-1]), w.num_heads, w.head_dim), float("nan"), dtype=out.dtype, device="cuda") for _ in range(2)]
    ts = [torch.zeros(int(off[-1]), dtype=torch.int64, device="cuda") for _ in range(2)]
    ys = [torch.zeros(int(off[-1]), dtype=torch.int8, device="cuda") for _ in range(2)]
    with plan_of(w, 2, tens) as plan:
        bd.rec_attn_fwd(plan, tens["q"], tens["k"], tens["v"], out)
        bd.rec_attn_fwd_compress(plan, tens["q"], tens["k"], tens["v"], hb, hl, segments, xs[0], ts[0], ys[0])
        bd.rec_attn_compress(tens["off_h"], hb, hl, segments, out.view(out.shape[0], -1), tens["t"], tens["ty"],
                             xs[1].view(xs[1].shape[0], -1), ts[1], ys[1])
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    assert torch.equal(ts[0], ts[1]) and torch.equal(ys[0], ys[1])
    # eight outputs of at most ~4 in size, rounded before (second) or after (first) their sum
    assert (xs[0].float() - xs[1].float()).abs().max() <= 8 * 4 * 2**-8
