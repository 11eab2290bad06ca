"""Candidates scored against a cached history whose key/value heads are shared by groups of
query heads (rec_attn_cache_create_grouped, rec_attn_cache_score) vs the fp64 oracle over
[history, candidates] with the shared heads repeated.

Tolerances: the roundings of the ungrouped path (Q', K', P and O in bf16), so its bounds:
max-abs 2e-2 and mean-abs 2e-3 (bf16), 1e-4 (fp32); lse: a score carries at most
2 * 2^-8 * scale * sum |q k|, below 5e-2 for these inputs (bf16), 1e-4 (fp32)."""
import numpy as np
import pytest
import torch

import gpu_util as gu
import oracle
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DAY = 86400


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def to_dev(a, dtype):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16) if dtype == "bf16" else torch.from_numpy(a).cuda()


class Batch:
    """Requests [history | candidates] with histories and candidate counts as given."""

    def __init__(self, hist, cands, heads, kv, d, dtype="bf16", seed=0, rt=0, special=0, scale=1.0, **params):
        rng = np.random.default_rng(seed)
        self.hist, self.cands, self.H, self.Hk, self.d, self.dtype = hist, cands, heads, kv, d, dtype
        self.hoff = np.concatenate([[0], np.cumsum(hist)]).astype(np.int64)
        self.coff = np.concatenate([[0], np.cumsum(cands)]).astype(np.int64)
        io = W.round_to_bf16_bits if dtype == "bf16" else (lambda a: a)
        new = lambda n, h: io((scale * rng.standard_normal((n, h, d))).astype(np.float32))
        Th, Nc = int(self.hoff[-1]), int(self.coff[-1])
        self.k, self.v = new(Th, kv), new(Th, kv)
        self.qc, self.kc, self.vc = new(Nc, heads), new(Nc, kv), new(Nc, kv)
        t, ty, tc = [], [], []
        for n, c in zip(hist, cands):
            s = 1_700_000_000 + int(rng.integers(0, 10 * DAY)) + np.cumsum(rng.integers(1, 3000, size=n + 1))
            t.append(s[:n])
            r, g = min(rt, n), min(special, max(n - rt, 0))
            ty.append(np.array([W.GLOBAL] * g + [W.HIST] * (n - g - r) + [W.RT] * r))
            tc.append(s[n] - rng.integers(0, 1500 * r + 1, size=c))
        self.t, self.tc = np.concatenate(t).astype(np.int64), np.concatenate(tc).astype(np.int64)
        self.ty = np.concatenate(ty).astype(np.int8)
        self.params = params

    def cache(self, max_cands=None):
        return bd.rec_attn_cache_create_grouped(
            bd.make_params(self.H, self.d, dtype=self.dtype, **self.params), self.Hk, self.hoff,
            torch.from_numpy(self.t).cuda(), torch.from_numpy(self.ty).cuda(), to_dev(self.k, self.dtype),
            to_dev(self.v, self.dtype), max_cands or max(1, max(self.cands)))

    def device(self):
        return (torch.from_numpy(self.tc).cuda(), to_dev(self.qc, self.dtype), to_dev(self.kc, self.dtype),
                to_dev(self.vc, self.dtype))

    def score(self, cache, with_lse=True, stream=None):
        tc, q, k, v = self.device()
        out = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:2], float("nan"), device="cuda") if with_lse else None
        bd.rec_attn_cache_score(cache, self.coff, tc, q, k, v, out, lse)
        torch.cuda.synchronize()
        return out, lse

    def reference(self):
        G = self.H // self.Hk
        off = self.hoff + self.coff
        T = int(off[-1])
        q = np.zeros((T, self.H, self.d), dtype=self.qc.dtype)
        k, v = q.copy(), q.copy()
        t, ty = np.zeros(T, dtype=np.int64), np.full(T, W.CAND, dtype=np.int8)
        rows = []
        for b in range(len(self.hist)):
            h0, h1, c0, c1, o = self.hoff[b], self.hoff[b + 1], self.coff[b], self.coff[b + 1], off[b]
            n, c = int(h1 - h0), int(c1 - c0)
            k[o:o + n], v[o:o + n] = np.repeat(self.k[h0:h1], G, 1), np.repeat(self.v[h0:h1], G, 1)
            t[o:o + n], ty[o:o + n] = self.t[h0:h1], self.ty[h0:h1]
            q[o + n:o + n + c] = self.qc[c0:c1]
            k[o + n:o + n + c], v[o + n:o + n + c] = np.repeat(self.kc[c0:c1], G, 1), np.repeat(self.vc[c0:c1], G, 1)
            t[o + n:o + n + c] = self.tc[c0:c1]
            rows += list(range(o + n, o + n + c))
        op = oracle.Params(self.H, self.d, **{"use_delay": False, **self.params})
        return oracle.attention(op, off, t, ty, q, k, v, rows=np.array(rows, dtype=np.int64), with_lse=True)

    def check(self, out, lse):
        ref, ref_lse = self.reference()
        x = gu.to_f64(out)
        assert np.isfinite(x).all()
        err = np.abs(x - ref)
        if self.dtype == "bf16":
            assert err.max() <= gu.BF16_MAX_ABS and err.mean() <= gu.BF16_MEAN_ABS, (err.max(), err.mean())
        else:
            assert err.max() <= gu.FP32_MAX_ABS, err.max()
        if lse is not None:
            y = lse.cpu().numpy()
            fin = np.isfinite(ref_lse)
            assert (np.isfinite(y) == fin).all()
            assert np.abs(y[fin] - ref_lse[fin]).max() <= (5e-2 if self.dtype == "bf16" else 1e-4)


CASES = {
    "one_of_one": dict(hist=[1], cands=[1], heads=8, kv=2, d=64),
    "one_token": dict(hist=[1023], cands=[1], heads=8, kv=2, d=64),
    "empty_history": dict(hist=[0, 5, 0], cands=[3, 2, 1], heads=8, kv=2, d=64),
    "no_candidates": dict(hist=[300, 77, 130], cands=[0, 5, 0], heads=8, kv=2, d=64),
    "tile_edges": dict(hist=[127, 128, 129, 255, 256, 257, 63, 64, 65], cands=[1] * 9, heads=4, kv=1, d=64),
    "ragged": dict(hist=[700, 33, 2049, 512], cands=[17, 90, 1, 33], heads=8, kv=2, d=64, rt=50),
    "group_of_three": dict(hist=[400, 91], cands=[11, 40], heads=6, kv=2, d=64, rt=20),
    "group_of_five_d128": dict(hist=[400, 91], cands=[7, 3], heads=5, kv=1, d=128, rt=9),
    "one_head_each": dict(hist=[300, 515], cands=[9, 2], heads=4, kv=4, d=64),
    "group_of_32": dict(hist=[200, 1000], cands=[3, 1], heads=32, kv=1, d=64),
    "long_history": dict(hist=[20000], cands=[2], heads=8, kv=2, d=64),
    "single_tokens_d128": dict(hist=[3000, 1500, 2999], cands=[1, 1, 1], heads=8, kv=2, d=128),
    "hundreds": dict(hist=[1500, 700], cands=[300, 129], heads=8, kv=2, d=64, rt=60),
    "hundreds_d128": dict(hist=[900], cands=[200], heads=4, kv=2, d=128, rt=60),
    "no_rotation": dict(hist=[333, 200], cands=[8, 4], heads=8, kv=2, d=64, use_rope=False),
    "delay": dict(hist=[600, 300], cands=[20, 5], heads=8, kv=2, d=64, rt=100, use_delay=True, delay_s=3600),
    "delay_hides_all": dict(hist=[200, 50], cands=[4, 3], heads=8, kv=2, d=64, use_delay=True, delay_s=1 << 40),
    "large_scores": dict(hist=[513], cands=[4], heads=8, kv=2, d=64, scale=3.0, use_rope=False),
    "fp32": dict(hist=[300, 0, 45], cands=[7, 2, 1], heads=4, kv=2, d=32, dtype="fp32", rt=30),
    "fp32_d64": dict(hist=[257], cands=[3], heads=6, kv=3, d=64, dtype="fp32"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_oracle(name):
    b = Batch(**CASES[name])
    with b.cache() as cache:
        out, lse = b.score(cache)
        again, _ = b.score(cache, with_lse=False)
        assert bd.rec_attn_cache_device_status(cache) == bd.OK
    if name == "large_scores":  # scores of rms 9 carry nine times the rounding of unit ones
        ref, _ = b.reference()
        assert np.linalg.norm(gu.to_f64(out) - ref) <= 9 * 6.6e-3 * np.linalg.norm(ref)
    else:
        b.check(out, lse)
    assert torch.equal(out, again)  # with or without lse, call after call


@pytest.mark.parametrize("name", ["ragged", "hundreds", "fp32"])
def test_one_head_each_agrees_with_the_ungrouped_cache(name):
    c = dict(CASES[name])
    c["kv"] = c["heads"]
    b = Batch(**c)
    with b.cache() as cache:
        out, lse = b.score(cache)
    plain = bd.rec_attn_cache_create(bd.make_params(b.H, b.d, dtype=b.dtype), b.hoff, torch.from_numpy(b.t).cuda(),
                                     torch.from_numpy(b.ty).cuda(), to_dev(b.k, b.dtype), to_dev(b.v, b.dtype), max(b.cands))
    with plain:
        ref, ref_lse = b.score(plain)
    tol = 2 * gu.BF16_MAX_ABS if b.dtype == "bf16" else 2 * gu.FP32_MAX_ABS  # each within it of the oracle
    assert (out.float() - ref.float()).abs().max() <= tol
    assert (lse - ref_lse).abs().max() <= 2 * (5e-2 if b.dtype == "bf16" else 1e-4)


@pytest.mark.parametrize("micro", [1, 5, 64])
def test_micro_batches_give_every_candidate_its_output(micro):
    b = Batch(hist=[900, 130], cands=[70, 33], heads=8, kv=2, d=64, rt=40)
    tc, q, k, v = b.device()
    out = torch.full_like(q, float("nan"))
    with b.cache(max_cands=micro) as cache:
        for i0 in range(0, max(b.cands), micro):
            take = [np.arange(b.coff[r] + min(i0, n), b.coff[r] + min(i0 + micro, n)) for r, n in enumerate(b.cands)]
            idx = torch.from_numpy(np.concatenate(take)).cuda()
            off = np.concatenate([[0], np.cumsum([len(x) for x in take])])
            part = torch.empty((len(idx),) + q.shape[1:], dtype=q.dtype, device="cuda")
            bd.rec_attn_cache_score(cache, off, tc[idx], q[idx].contiguous(), k[idx].contiguous(), v[idx].contiguous(), part)
            out[idx] = part
        torch.cuda.synchronize()
    b.check(out, None)


def test_refusals():
    b = Batch(hist=[100], cands=[4], heads=8, kv=2, d=64)
    tc, q, k, v = b.device()
    out = torch.empty_like(q)
    with b.cache(max_cands=4) as cache:
        def code(off=(0, 4), tc=tc, q=q, k=k, v=v, out=out, lse=None):
            try:
                bd.rec_attn_cache_score(cache, np.array(off), tc, q, k, v, out, lse)
                return bd.OK
            except bd.RecAttnError as e:
                return e.code
        assert code() == bd.OK
        assert code(off=(0, 5)) == bd.ERR_INVALID_ARG  # more than max_cands
        assert code(off=(1, 4)) == bd.ERR_INVALID_ARG
        assert code(off=(0, -1)) == bd.ERR_INVALID_ARG
        for name in ("tc", "q", "k", "v", "out"):
            assert code(**{name: None}) == bd.ERR_INVALID_ARG
        assert code(out=q) == bd.ERR_INVALID_ARG and code(out=k) == bd.ERR_INVALID_ARG
        assert code(q=q.data_ptr() + 8) == bd.ERR_INVALID_ARG
        assert code(off=(0, 0), tc=None, q=None, k=None, v=None, out=None) == bd.OK  # nothing to score
        torch.cuda.synchronize()


def test_two_streams_and_a_graph_share_one_cache():
    """Calls on one bf16 cache write nothing into it: two at once, and a replayed capture whose
    inputs change between replays."""
    b = Batch(hist=[3000, 1200, 64], cands=[3, 1, 2], heads=8, kv=2, d=64, rt=40)
    with b.cache() as cache:
        ref, _ = b.score(cache)
        tc, q, k, v = b.device()
        streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(8)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            with torch.cuda.stream(streams[i % 2]):
                bd.rec_attn_cache_score(cache, b.coff, tc, q, k, v, o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
        graphs = []
        for _ in range(2):
            out = torch.empty_like(q)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                bd.rec_attn_cache_score(cache, b.coff, tc, q, k, v, out)
            graphs.append((graph, out))
        for _ in range(3):
            for graph, out in graphs:
                out.fill_(float("nan"))
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, ref) for _, out in graphs)
        q.copy_(q.flip(0))
        want = torch.empty_like(q)
        bd.rec_attn_cache_score(cache, b.coff, tc, q, k, v, want)
        graphs[0][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], want) and not torch.equal(want, ref)
        del graphs


def test_rows_behind_the_last_candidate_stay_as_they_were():
    b = Batch(hist=[300, 50], cands=[2, 1], heads=8, kv=2, d=64)
    tc, q, k, v = b.device()
    out = torch.full((8,) + q.shape[1:], 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((8, b.H), 7.0, device="cuda")
    with b.cache() as cache:
        bd.rec_attn_cache_score(cache, b.coff, tc, q, k, v, out, lse)
        torch.cuda.synchronize()
    assert (out[3:] == 7).all() and (lse[3:] == 7).all() and torch.isfinite(lse[:3]).all()


def test_bad_history_keys_are_seen_by_nobody():
    """Types outside the user side and times out of range: reported where they are device
    errors, and without weight."""
    b = Batch(hist=[200], cands=[3], heads=8, kv=2, d=64)
    with b.cache() as cache:
        out, _ = b.score(cache)
    keep = np.ones(200, dtype=bool)
    keep[[5, 77, 130]] = False
    b.ty[5], b.ty[77] = 9, W.CAND
    b.t[130] = 1 << 62
    with b.cache() as cache:
        got, lse = b.score(cache)
        assert bd.rec_attn_cache_device_status(cache) == bd.ERR_DEVICE_INPUT
    small = Batch(hist=[197], cands=[3], heads=8, kv=2, d=64)
    small.k, small.v, small.t, small.ty = b.k[keep], b.v[keep], b.t[keep], b.ty[keep]
    small.qc, small.kc, small.vc, small.tc = b.qc, b.kc, b.vc, b.tc
    small.check(got, lse)


def test_more_requests_than_one_launch_takes():
    n = 1100
    b = Batch(hist=[i % 7 for i in range(n)], cands=[i % 3 for i in range(n)], heads=4, kv=2, d=64)
    with b.cache() as cache:
        out, lse = b.score(cache)
    b.check(out, lse)
