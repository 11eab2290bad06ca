"""fp32 attention: a key or value that is not finite reaches the rows that see its key, and no others
(a candidate's, the other candidates of its request; an old event's, the rows whose window has left
it).  The rows that do not see it keep every bit of the same call on finite inputs."""
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


CASES = {
    # requests of (special, history, events, candidates), heads, key/value heads, head_dim, mask
    "candidates_d64": ([(2, 100, 0, 90), (0, 1, 0, 3)], 4, 2, 64, {}),
    "events_d32": ([(1, 70, 60, 70)], 2, 1, 32, {}),
    "window_d64": ([(0, 300, 0, 1), (3, 129, 0, 20)], 2, 2, 64, dict(window=40)),
    "delay_d32": ([(0, 260, 0, 5)], 2, 2, 32, dict(use_delay=True, delay_s=3600)),
}


def batch(name):
    reqs, H, Hk, d, mask = CASES[name]
    rng = np.random.default_rng(4)
    ty = [np.repeat(np.array([W.GLOBAL, W.HIST, W.RT, W.CAND], dtype=np.int8), r) for r in reqs]
    off = np.concatenate([[0], np.cumsum([len(x) for x in ty])]).astype(np.int64)
    T = int(off[-1])
    t = np.concatenate([1_700_000_000 + np.cumsum(rng.integers(1, 2000, size=len(x))) for x in ty]).astype(np.int64)
    dev = lambda a: torch.from_numpy(a).cuda()
    q, k, v = (dev(rng.standard_normal((T, h, d)).astype(np.float32)) for h in (H, Hk, Hk))
    params = {"use_delay": False, **mask}
    seen = [oracle.mask_block(oracle.Params(H, d, **params), t[a:b], np.concatenate(ty)[a:b], 0, b - a, 0, b - a)
            for a, b in zip(off[:-1], off[1:])]
    return off, dev(t), dev(np.concatenate(ty)), q, k, v, Hk, bd.make_params(H, d, dtype="fp32", **params), seen


# (key, value) of the poisoned rows
POISON = {"value_inf": (None, float("inf")), "value_nan": (None, float("nan")), "key_nan": (float("nan"), None),
          "both": (float("inf"), float("-inf"))}


@pytest.mark.parametrize("poison", list(POISON))
@pytest.mark.parametrize("name", list(CASES))
def test_forward(name, poison):
    off, t, ty, q, k, v, hk, params, seen = batch(name)
    bad = []  # a few keys of every request
    for (a, b), s in zip(zip(off[:-1], off[1:]), seen):
        n = b - a
        bad += [a + j for j in {0, n // 3, n - 1, max(0, n - 4)} if not s[:n, j].all()]
    reached = np.zeros(int(off[-1]), dtype=bool)
    for j in bad:
        r = int(np.searchsorted(off, j, side="right")) - 1
        reached[off[r]:off[r + 1]] |= seen[r][:off[r + 1] - off[r], j - off[r]].astype(bool)
    assert bad and reached.any() and not reached.all()
    outs = []
    for p in (False, True):
        if p:
            for x, value in zip((k, v), POISON[poison]):
                if value is not None:
                    x[bad] = value
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        with bd.rec_attn_plan_grouped(params, hk, off, torch.from_numpy(off).cuda(), t, ty) as plan:
            bd.rec_attn_fwd(plan, q, k, v, out, lse)
            torch.cuda.synchronize()
            assert bd.rec_attn_device_status(plan) == bd.OK
        outs.append((out, lse))
        if hk == params.num_heads:  # the same without a mask table
            out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
            bd.rec_attn_fwd_noalloc(params, off, torch.from_numpy(off).cuda(), t, ty, q, k, v, out, lse)
            torch.cuda.synchronize()
            assert torch.equal(out[~torch.from_numpy(reached).cuda()], outs[-1][0][~torch.from_numpy(reached).cuda()])
    clean = torch.from_numpy(~reached).cuda()
    assert torch.isfinite(outs[1][0][clean]).all()  # (the lse of a row that sees no key is -inf)
    for a, b in zip(*outs):
        assert torch.equal(a[clean], b[clean])
    assert not torch.isfinite(outs[1][0][~clean]).all(-1).any()


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("d", [32, 64])
def test_scoring(d, grouped):
    """One candidate's pair, and another request's history."""
    hist, cands, H = [130, 5, 64], 70, 4
    hk = 2 if grouped else H
    hoff = np.concatenate([[0], np.cumsum(hist)]).astype(np.int64)
    coff = np.arange(len(hist) + 1, dtype=np.int64) * cands
    g = torch.Generator().manual_seed(3)
    new = lambda n, h: torch.randn(int(n), h, d, generator=g).cuda()
    k, v = new(hoff[-1], hk), new(hoff[-1], hk)
    q, kc, vc = new(coff[-1], H), new(coff[-1], hk), new(coff[-1], hk)
    t, tc = torch.arange(int(hoff[-1]), device="cuda"), torch.full((int(coff[-1]),), 10_000, device="cuda")
    ty = torch.full((int(hoff[-1]),), W.HIST, dtype=torch.int8, device="cuda")
    params, outs = bd.make_params(H, d, dtype="fp32"), []
    for poison in (False, True):
        if poison:
            k[130:135], v[130:135] = float("nan"), float("inf")
            vc[3], kc[3] = float("nan"), float("inf")
        out = torch.zeros_like(q)
        hist_args = (hoff, t, ty, k, v, cands)
        with (bd.rec_attn_cache_create_grouped(params, hk, *hist_args) if grouped
              else bd.rec_attn_cache_create(params, *hist_args)) as cache:
            bd.rec_attn_cache_score(cache, coff, tc, q, kc, vc, out)
            torch.cuda.synchronize()
        outs.append(out)
    clean = torch.ones(int(coff[-1]), dtype=torch.bool, device="cuda")
    clean[3], clean[cands:2 * cands] = False, False
    assert torch.isfinite(outs[1][clean]).all() and torch.equal(outs[0][clean], outs[1][clean])
    assert not torch.isfinite(outs[1][~clean]).all(-1).any()


def test_pruned_queries():
    """Queries that a plan does not compute may hold anything."""
    off, t, ty, q, k, v, hk, params, _ = batch("candidates_d64")
    kept, outs = (ty == W.CAND).cpu(), []
    for poison in (False, True):
        if poison:
            q[~kept.cuda()] = float("nan")
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        with bd.rec_attn_plan_grouped(params, hk, off, torch.from_numpy(off).cuda(), t, ty, keep_user_queries=0) as plan:
            bd.rec_attn_fwd(plan, q, k, v, out, lse)
            torch.cuda.synchronize()
        outs.append((out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and (outs[0][0][~kept.cuda()] == 0).all()
