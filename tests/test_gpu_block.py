"""The operators together, as a model uses them: layer norm by token type, projections, attention
with shared key/value heads, its gradient and the layer norm's; and the same layer's candidates
scored against the cached history.  Against the same layer in 64 bits (the fp64 oracle for the
attention), and the calls that a graph capture refuses.

Tolerances (relative Frobenius): every tensor handed on is rounded to bf16, off by at most 2^-8
of each value; a projection with random weights and the averages of the attention leave a
relative error as it is.  Output: six roundings on the way (y; q, k, v; Q', K'; P; O; out), so
6 * 2^-8 = 2.4e-2.  Gradients: ten (y; q, k, v; Q', K'; P; O; dout; dS; dq, dk, dv; dy; dx), so
10 * 2^-8 = 3.9e-2.  A gain's and a bias's gradient is a sum of those over rows: the same."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gpu_util as gu
import oracle
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W

pytestmark = pytest.mark.gpu
OUT, GRAD = 6 * 2.0 ** -8, 10 * 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


CASES = {
    "d64": (lambda: W.mtgr(batch=3, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=8), 2, 512),
    "d64_one_token": (lambda: W.mtgr(batch=2, hist=(1, 1), rt=(0, 0), cand=(1, 1), heads=8), 4, 512),
    "d128": (lambda: W.mtgr(batch=2, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=6, head_dim=128), 2, 520),
    "many_candidates": (lambda: W.mtgr(batch=2, hist=(700, 900), rt=(20, 60), cand=(300, 400), heads=8), 1, 512),
}


class Block:
    """x -> layer norm by type -> q, k, v -> attention -> output projection."""

    def __init__(self, name):
        make, self.hk, self.width = CASES[name]
        self.w = w = make()
        g = torch.Generator().manual_seed(5)
        T, H, d, wd = w.total_tokens, w.num_heads, w.head_dim, self.width
        self.tens = gu.device_inputs(w)
        rnd = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).cuda()
        self.x = (rnd(T, wd) * 1.5 + 0.25).bfloat16()
        self.gain, self.bias = 1 + 0.1 * rnd(4, wd), 0.1 * rnd(4, wd)
        self.wq, self.wk, self.wv = (rnd(wd, h * d, scale=wd ** -0.5).bfloat16() for h in (H, self.hk, self.hk))
        self.wo = rnd(H * d, wd, scale=(H * d) ** -0.5).bfloat16()
        self.dy = rnd(T, wd).bfloat16()

    def norm_and_project(self, x, ty):
        w, y = self.w, torch.full_like(x, float("nan"))
        bd.rec_attn_layernorm_fwd(x, self.gain, self.bias, y, types=ty, eps=EPS)
        shape = lambda t, h: t.view(x.shape[0], h, w.head_dim)
        return y, shape(y @ self.wq, w.num_heads), shape(y @ self.wk, self.hk), shape(y @ self.wv, self.hk)

    def train(self):
        w, t = self.w, self.tens
        y, q, k, v = self.norm_and_project(self.x, t["ty"])
        nan = lambda a: torch.full_like(a, float("nan"))
        o, dq, dk, dv, dx = nan(q), nan(q), nan(k), nan(v), nan(self.x)
        dgain, dbias = nan(self.gain), nan(self.bias)
        lse = torch.empty(q.shape[:2], device="cuda")
        flat = lambda a: a.reshape(a.shape[0], -1)
        with bd.rec_attn_plan_grouped(gu.params_for(w), self.hk, t["off_h"], t["off_d"], t["t"], t["ty"]) as plan:
            bd.rec_attn_fwd(plan, q, k, v, o, lse)
            out = flat(o) @ self.wo
            do = (self.dy @ self.wo.t()).view_as(o)
            bd.rec_attn_bwd(plan, q, k, v, o, lse, do, dq, dk, dv)
            dn = torch.cat([flat(dq), flat(dk), flat(dv)], 1) @ torch.cat([self.wq, self.wk, self.wv], 1).t()
            bd.rec_attn_layernorm_bwd(self.x, self.gain, dn, dx, dgain, dbias, types=t["ty"], eps=EPS)
            torch.cuda.synchronize()
            assert bd.rec_attn_device_status(plan) == bd.OK
        return {"o": flat(o), "out": out, "dx": dx, "dgain": dgain, "dbias": dbias}

    def reference(self):
        w, G = self.w, self.w.num_heads // self.hk
        x, gain, bias, wq, wk, wv, wo, dy = (a.double().cpu().numpy() for a in (
            self.x, self.gain, self.bias, self.wq, self.wk, self.wv, self.wo, self.dy))
        T, d, ty = w.total_tokens, w.head_dim, w.types.astype(np.int64)
        m = x.mean(1, keepdims=True)
        r = 1 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + EPS)
        n = (x - m) * r
        y = n * gain[ty] + bias[ty]
        q, k, v = (y @ a for a in (wq, wk, wv))
        q = q.reshape(T, -1, d)
        k, v = (np.repeat(a.reshape(T, self.hk, d), G, 1) for a in (k, v))
        q, k, v, do = (a.astype(np.float32) for a in (q, k, v, (dy @ wo.T).reshape(q.shape)))  # the oracle's input type
        op = gu.oracle_params(w)
        o = oracle.attention(op, w.offsets, w.t, w.types, q, k, v)
        dq, dk, dv = oracle.attention_bwd(op, w.offsets, w.t, w.types, q, k, v, do)
        shared = lambda a: a.reshape(T, self.hk, G, d).sum(2).reshape(T, -1)
        dn = dq.reshape(T, -1) @ wq.T + shared(dk) @ wk.T + shared(dv) @ wv.T
        u = dn * gain[ty]
        dx = r * (u - u.mean(1, keepdims=True) - n * (u * n).mean(1, keepdims=True))
        dgain, dbias = np.zeros_like(gain), np.zeros_like(bias)
        np.add.at(dgain, ty, dn * n)
        np.add.at(dbias, ty, dn)
        o = o.reshape(T, -1)
        return {"o": o, "out": o @ wo, "dx": dx, "dgain": dgain, "dbias": dbias}


def close(got, ref, tol, what):
    x = got.double().cpu().numpy()
    assert np.isfinite(x).all(), what
    err = np.linalg.norm(x - ref) / max(np.linalg.norm(ref), 1e-30)
    assert err <= tol, (what, err)


@pytest.mark.parametrize("name", list(CASES))
def test_layer_forward_and_backward(name):
    b = Block(name)
    got, ref = b.train(), b.reference()
    for what in ref:
        close(got[what], ref[what], OUT if what in ("o", "out") else GRAD, what)
    again = b.train()
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("name", list(CASES))
def test_layer_candidates_against_the_cached_history(name):
    """The candidates' rows of the layer, from a cache of the other rows' keys and values."""
    b = Block(name)
    w = b.w
    cand = w.types == W.CAND
    req = np.repeat(np.arange(len(w.offsets) - 1), np.diff(w.offsets))
    count = lambda m: np.concatenate([[0], np.cumsum(np.bincount(req[m], minlength=len(w.offsets) - 1))]).astype(np.int64)
    rows = {c: torch.from_numpy(np.flatnonzero(cand == c)).cuda() for c in (True, False)}
    ty, t = b.tens["ty"], b.tens["t"]
    _, _, k, v = b.norm_and_project(b.x[rows[False]], ty[rows[False]])
    _, qc, kc, vc = b.norm_and_project(b.x[rows[True]], ty[rows[True]])
    coff = count(cand)
    out = torch.full_like(qc, float("nan"))
    with bd.rec_attn_cache_create_grouped(gu.params_for(w), b.hk, count(~cand), t[rows[False]], ty[rows[False]], k, v,
                                          int(np.diff(coff).max())) as cache:
        bd.rec_attn_cache_score(cache, coff, t[rows[True]], qc, kc, vc, out)
        torch.cuda.synchronize()
        assert bd.rec_attn_cache_device_status(cache) == bd.OK
    close(out.flatten(1), b.reference()["o"][cand], OUT, "scored")


@pytest.mark.parametrize("cands", [1, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_another_request_do_not_reach_the_candidates(d, cands):
    """NaN and infinities in one request's cached keys and values, and in one candidate's, stay
    with that request and that candidate, wherever the requests end within a tile."""
    hist, H, Hk = [130, 5, 64, 129], 8, 2
    hoff = np.concatenate([[0], np.cumsum(hist)]).astype(np.int64)
    coff = np.arange(5, dtype=np.int64) * cands
    g = torch.Generator().manual_seed(3)
    new = lambda n, h: torch.randn(n, h, d, generator=g).bfloat16().cuda()
    k, v = new(hoff[-1], Hk), new(hoff[-1], Hk)
    q, kc, vc = new(coff[-1], H), new(coff[-1], Hk), new(coff[-1], Hk)
    t = torch.arange(int(hoff[-1]), device="cuda")
    tc = torch.full((int(coff[-1]),), 10_000, device="cuda")
    ty = torch.full((int(hoff[-1]),), W.HIST, dtype=torch.int8, device="cuda")
    outs = []
    for poison in (False, True):
        if poison:
            k[130:135], v[130:135] = float("nan"), float("inf")
            q[3 * cands], vc[0] = float("nan"), float("inf")
        out = torch.zeros_like(q)
        with bd.rec_attn_cache_create_grouped(bd.make_params(H, d), Hk, hoff, t, ty, k, v, cands) as cache:
            bd.rec_attn_cache_score(cache, coff, tc, q, kc, vc, out)
            torch.cuda.synchronize()
        outs.append(out)
    clean = torch.ones(int(coff[-1]), dtype=torch.bool, device="cuda")
    clean[cands:2 * cands] = False
    clean[3 * cands], clean[0] = False, False
    assert torch.equal(outs[0][clean], outs[1][clean]) and torch.isfinite(outs[1][clean]).all()
    assert not torch.isfinite(outs[1][~clean]).any()


def test_capture_refuses_what_reads_host_memory_later():
    """Planning, cache creation and the calls on a grouped plan are refused on a capturing stream;
    the capture stays valid and holds what it could take."""
    b = Block("d64")
    w, t = b.w, b.tens
    _, q, k, v = b.norm_and_project(b.x, t["ty"])
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse, y = torch.empty(q.shape[:2], device="cuda"), torch.zeros_like(b.x)
    plan_args = (gu.params_for(w), b.hk, t["off_h"], t["off_d"], t["t"], t["ty"])
    f32 = bd.make_params(w.num_heads, 64, dtype="fp32")
    k32, q32 = k.float(), q[:1].float()
    with bd.rec_attn_plan_grouped(*plan_args) as plan, bd.rec_attn_cache_create_grouped(
            f32, b.hk, w.offsets, t["t"], t["ty"], k32, k32, 1) as cache:
        bd.rec_attn_fwd(plan, q, k, v, o, lse)
        torch.cuda.synchronize()
        coff = np.minimum(np.arange(len(w.offsets)), 1).astype(np.int64)
        o32 = torch.empty_like(q32)
        calls = [
            lambda: bd.rec_attn_plan_grouped(*plan_args),
            lambda: bd.rec_attn_cache_create_grouped(gu.params_for(w), b.hk, w.offsets, t["t"], t["ty"], k, v, 4),
            lambda: bd.rec_attn_cache_score(cache, coff, t["t"], q32, k32[:1], k32[:1], o32),
            lambda: bd.rec_attn_fwd(plan, q, k, v, o, lse),
            lambda: bd.rec_attn_bwd(plan, q, k, v, o, lse, q, dq, dk, dv),
        ]
        codes, graph = [], torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call in calls:
                try:
                    call()
                    codes.append(bd.OK)
                except bd.RecAttnError as e:
                    codes.append(e.code)
            bd.rec_attn_layernorm_fwd(b.x, b.gain, b.bias, y, types=t["ty"], eps=EPS)
        assert codes == [bd.ERR_UNSUPPORTED] * len(calls)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(y)
        bd.rec_attn_layernorm_fwd(b.x, b.gain, b.bias, want, types=t["ty"], eps=EPS)
        assert torch.equal(y, want)
        for call in calls[2:]:
            call()
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK


@pytest.mark.parametrize("call", ["bd.rec_attn_layernorm_fwd(x, w, None, dx)", "bd.rec_attn_layernorm_bwd(x, w, dy, dx, dw, db)",
                                  "bd.rec_attn_cache_score(cache, [0, n], t[:n], q, k, k, o)"])
def test_first_call_of_a_process_may_be_captured(call):
    """What a call sets up once (a workspace pool, kernel attributes) is then set up during the
    capture."""
    code = f"""
import torch
from generative_recommender_ranking_gb300 import binding as bd
dev, n = "cuda", 70
x, dy, w = torch.randn(300, 512, device=dev), torch.randn(300, 512, device=dev), torch.ones(1, 512, device=dev)
dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w)
q, k = torch.randn(n, 8, 64, device=dev).bfloat16(), torch.randn(n, 2, 64, device=dev).bfloat16()
kh, t, o = torch.randn(5000, 2, 64, device=dev).bfloat16(), torch.arange(5000, device=dev), torch.zeros_like(q)
if "score" in {call!r}:
    cache = bd.rec_attn_cache_create_grouped(bd.make_params(8, 64), 2, [0, 5000], t, torch.ones(5000, dtype=torch.int8, device=dev),
                                             kh, kh, n)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    {call}
g.replay()
torch.cuda.synchronize()
outs = (dx, dw, db, o)
got = [a.clone() for a in outs]
for a in outs:
    a.zero_()
{call}
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, got)) and sum(float(a.float().abs().sum()) for a in outs) > 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_layernorm_takes_tensors_of_the_current_device_only():
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(1, 64, device="cuda")
    y = torch.empty_like(x)
    bd.rec_attn_layernorm_fwd(x, w, None, y)  # the same call with device tensors is taken
    for bad in ((x.cpu(), w, None, y), (x, w.cpu(), None, y), (x, w, None, y.cpu()), (x.cpu(), w.cpu(), None, y.cpu())):
        with pytest.raises(bd.RecAttnError) as e:
            bd.rec_attn_layernorm_fwd(*bad)
        assert e.value.code == bd.ERR_INVALID_ARG


@pytest.mark.parametrize("name,lens,H,Hk,d", [
    ("parts", [5000], 4, 1, 64), ("whole_groups", list(range(4200, 4700, 50)), 4, 1, 64), ("d128", [4500, 4224], 4, 2, 128),
    ("edges", [4096, 4097, 4223], 2, 1, 64)])
def test_items_of_many_tiles(name, lens, H, Hk, d):
    """Causal rows of more than 32 tiles, alone and with the heads of a group in one item, against
    64 bits: gradients to 1e-2 relative Frobenius and 2e-2 of the largest value (the bounds of the
    ungrouped gradients), the output to 2e-2 and 2e-3 on average."""
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    T, G = int(off[-1]), H // Hk
    g = torch.Generator(device="cuda").manual_seed(7)
    new = lambda h: torch.randn(T, h, d, generator=g, device="cuda").bfloat16()
    q, k, v, do = new(H), new(Hk), new(Hk), new(H)
    t = torch.arange(T, device="cuda") * 60
    ty = torch.full((T,), W.HIST, dtype=torch.int8, device="cuda")
    o, dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, q, k, v))
    lse = torch.empty(T, H, device="cuda")
    with bd.rec_attn_plan_grouped(bd.make_params(H, d, use_rope=False), Hk, off, torch.from_numpy(off).cuda(), t, ty) as plan:
        bd.rec_attn_fwd(plan, q, k, v, o, lse)
        bd.rec_attn_bwd(plan, q, k, v, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    ref = [torch.empty(x.shape, dtype=torch.float64, device="cuda") for x in (o, dq, dk, dv)]
    for b in range(len(lens)):
        r = slice(int(off[b]), int(off[b + 1]))
        blind = torch.ones(lens[b], lens[b], dtype=torch.bool, device="cuda").triu(1)
        for hk in range(Hk):
            K, V = k[r, hk].double(), v[r, hk].double()
            sums = [torch.zeros_like(K), torch.zeros_like(V)]
            for h in range(hk * G, (hk + 1) * G):
                Q, dO = q[r, h].double(), do[r, h].double()
                P = torch.softmax((Q @ K.t() * d ** -0.5).masked_fill(blind, -float("inf")), 1)
                O = P @ V
                dS = P * (dO @ V.t() - (dO * O).sum(1, keepdim=True)) * d ** -0.5
                ref[0][r, h], ref[1][r, h] = O, dS @ K
                sums[0] += dS.t() @ Q
                sums[1] += P.t() @ dO
            ref[2][r, hk], ref[3][r, hk] = sums
    err = (o.double() - ref[0]).abs()
    assert err.max() <= gu.BF16_MAX_ABS and err.mean() <= gu.BF16_MEAN_ABS
    for what, got, want in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[1:]):
        diff = got.double() - want
        rel, top = float(diff.norm() / want.norm()), float(diff.abs().max() / want.abs().max())
        assert rel <= 1e-2 and top <= 2e-2, (what, rel, top)


F32 = {
    # lengths, heads, key/value heads, head_dim, mask
    "groups_in_parts_d64": ([700, 0, 63, 64, 65, 129], 8, 1, 64, {}),
    "groups_of_three_d32": ([190, 1, 257], 6, 2, 32, dict(use_delay=True, delay_s=1800)),
    "window_d64": ([300, 500], 4, 2, 64, dict(window=70)),
    "whole_groups_d32": ([40] * 200, 4, 2, 32, dict(hist_bidirectional=True)),
    "no_rotation_d64": ([128, 192], 2, 1, 64, dict(use_rope=False)),
}


@pytest.mark.parametrize("name", list(F32))
def test_fp32_shared_heads_at_tile_edges(name):
    """fp32 forward and backward with shared heads, lengths around the kernels' 64 rows, special tokens,
    events and candidates, an empty request, with and without parts of the groups: the fp32 bounds
    (outputs 1e-4; gradients 1e-5 relative Frobenius and 1e-4 of the largest value)."""
    lens, H, Hk, d, mask = F32[name]
    rng = np.random.default_rng(9)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    T, G = int(off[-1]), H // Hk
    t = np.concatenate([1_700_000_000 + np.cumsum(rng.integers(1, 2000, size=n)) for n in lens]).astype(np.int64)
    ty = np.concatenate([np.array(([W.GLOBAL] * 3 + [W.HIST] * n + [W.RT] * (n // 8) + [W.CAND] * (n // 9))[-n:] if n else [], dtype=np.int8)
                         for n in lens])
    new = lambda h: rng.standard_normal((T, h, d)).astype(np.float32)
    q, k, v, do = new(H), new(Hk), new(Hk), new(H)
    params = {"use_delay": False, **mask}
    dev = lambda a: torch.from_numpy(a).cuda()
    Q, K, V, DO = dev(q), dev(k), dev(v), dev(do)
    o, dq, dk, dv = (torch.full_like(x, float("nan")) for x in (Q, Q, K, V))
    lse = torch.full((T, H), float("nan"), device="cuda")
    with bd.rec_attn_plan_grouped(bd.make_params(H, d, dtype="fp32", **params), Hk, off, dev(off), dev(t), dev(ty)) as plan:
        bd.rec_attn_fwd(plan, Q, K, V, o, lse)
        bd.rec_attn_bwd(plan, Q, K, V, o, lse, DO, dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    op = oracle.Params(H, d, **params)
    kr, vr = np.repeat(k, G, 1), np.repeat(v, G, 1)
    ref, ref_lse = oracle.attention(op, off, t, ty, q, kr, vr, with_lse=True)
    rq, rk, rv = oracle.attention_bwd(op, off, t, ty, q, kr, vr, do)
    assert np.abs(o.double().cpu().numpy() - ref).max() <= gu.FP32_MAX_ABS
    fin, got = np.isfinite(ref_lse), lse.cpu().numpy()
    assert (np.isfinite(got) == fin).all() and np.abs(got[fin] - ref_lse[fin]).max() <= 1e-4
    shared = lambda a: a.reshape(T, Hk, G, d).sum(2)
    for what, x, want in (("dq", dq, rq), ("dk", dk, shared(rk)), ("dv", dv, shared(rv))):
        diff = x.double().cpu().numpy() - want
        assert np.linalg.norm(diff) <= 1e-5 * np.linalg.norm(want), what
        assert np.abs(diff).max() <= 1e-4 * np.abs(want).max(), what
