"""How the feed-forward and scaled calls are used: streams, graphs, empty batches, places behind the last
row, tensors off 32-byte boundaries, values that are not finite, offsets past 2^31, and a run of them
with the layer norm and the attention."""
import math

import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W
from test_gpu_ffn import inputs, reference, within
from test_gpu_layernorm import reference as norm_reference
from test_gpu_layernorm import within as norm_within
from test_gpu_scaled import F8, at_values, held, quantize, quantized
from test_gpu_scaled import s as sums

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def train(t, act="silu", stream=None):
    x, dy, wi, wo = t
    o = [torch.full_like(x, 7), torch.full_like(x, 7), torch.full_like(wi, 7), torch.full_like(wo, 7)]
    bd.rec_attn_ffn_fwd(x, wi, wo, o[0], activation=act, stream=stream)
    bd.rec_attn_ffn_bwd(x, wi, wo, dy, *o[1:], activation=act, stream=stream)
    return o


def serving(seed, rows=70, width=144, hidden=256):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g).to(BF).cuda()
    wi, wis = quantize((torch.randn(2 * hidden, width, generator=g) / 12).cuda(), 128)
    wo, wos = quantize((torch.randn(width, hidden, generator=g) / 16).cuda(), 128)
    return x, wi, wis, wo, wos


def serve(t, stream=None):
    x, wi, wis, wo, wos = t
    y = torch.full_like(x, 7)
    bd.rec_attn_ffn_scaled_fwd(x, wi, wis, wo, wos, y, stream=stream)
    q, sc = torch.zeros(x.shape, device="cuda").to(F8), torch.zeros(x.shape[0], wis.shape[1], device="cuda")
    bd.rec_attn_scaled_quantize(x, q, sc, stream=stream)
    z = torch.full((x.shape[0], wi.shape[0]), 7.0, dtype=BF, device="cuda")
    bd.rec_attn_scaled_matmul(q, sc, wi, wis, z, stream=stream)
    return [y, q.view(torch.uint8), sc, z]


def same(a, b):
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    return all(torch.equal(x, y) for x, y in zip(a, b))


CASES = [lambda seed: (train, inputs(300, 136, 264, BF, seed)), lambda seed: (train, inputs(3, 512, 1024, BF, seed)),
         lambda seed: (train, inputs(150, 132, 68, F32, seed)), lambda seed: (serve, serving(seed)),
         lambda seed: (serve, serving(seed, rows=2)), lambda seed: (serve, serving(seed, rows=700))]
IDS = ["bf16", "few", "fp32", "e4m3", "e4m3_few", "e4m3_rows"]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_equal_calls_give_equal_bits(case):
    run, t = case(1)
    assert same(run(t), run(t))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_two_streams_at_once(case):
    """Calls on two streams share nothing, and see what their own stream has written just before."""
    run, a = case(1)
    _, b = case(2)
    want = run(a), run(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(3):
        for k, (st, t) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(st):
                late = list(t)
                late[0] = torch.zeros_like(t[0])
                torch.cuda._sleep(200000)
                late[0].copy_(t[0])
                got[k] = run(tuple(late))
        for st in streams:
            st.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_graphs(case):
    """Two graphs of the same call on other tensors, replayed in turn and with new inputs, beside an eager
    call."""
    run, a = case(1)
    _, b = case(2)
    _, c = case(3)
    want = [run(t) for t in (a, b, c)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(t))
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            for x in o:
                x.zero_()
        graphs[0].replay()
        eager = run(c)
        graphs[1].replay()
        assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(eager, want[2])
    a[0].copy_(c[0])  # new rows, the weights as they were
    fresh = run((c[0],) + tuple(a[1:]))
    graphs[0].replay()
    assert same(outs[0], fresh)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_rows(dtype):
    x, dy, wi, wo = (t[:0] if t.shape[0] == 1 else t for t in inputs(1, 64, 128, dtype))
    _, _, dwi, dwo = train((x, dy, wi, wo))
    torch.cuda.synchronize()
    assert (dwi == 0).all() and (dwo == 0).all()
    bd.rec_attn_ffn_bwd(x, wi, wo, dy)  # nothing wanted
    e = torch.empty(0, 128, device="cuda").to(F8)
    bd.rec_attn_scaled_quantize(torch.empty(0, 128, device="cuda"), e, torch.empty(0, 1, device="cuda"))
    w, ws = quantize(torch.ones(64, 128, device="cuda"), 128)
    bd.rec_attn_scaled_matmul(e, torch.empty(0, 1, device="cuda"), w, ws, torch.empty(0, 64, dtype=BF, device="cuda"))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_not_wanted(dtype):
    t = inputs(200, 136, 264, dtype)
    full = train(t)
    for k in range(3):
        o = [torch.full_like(f, 7) if i == k else None for i, f in enumerate(full[1:])]
        bd.rec_attn_ffn_bwd(t[0], t[2], t[3], t[1], *o)
        assert same([o[k]], [full[1 + k]])


@pytest.mark.parametrize("rows", [3, 40, 129, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_only_its_rows_are_written_and_any_16_byte_boundary_does(rows, dtype):
    x, dy, wi, wo = inputs(rows, 136, 264, dtype)
    y, dx, dwi, dwo = train((x, dy, wi, wo))
    step = 16 // x.element_size()

    def moved(t, fill=None):  # the same matrix 16 bytes past a 32-byte boundary, between guards
        buf = torch.full((t.numel() + 2 * step + 4096,), 5.0, dtype=t.dtype, device="cuda")
        off = step if (buf.data_ptr() + 16) % 32 else 2 * step
        v = buf[off:off + t.numel()].view(t.shape)
        assert v.data_ptr() % 32 == 16
        v.copy_(t) if fill is None else v.fill_(fill)
        return v, buf, off

    ins = [moved(t) for t in (x, dy, wi, wo)]
    outs = [moved(t, 7.0) for t in (y, dx, dwi, dwo)]
    bd.rec_attn_ffn_fwd(ins[0][0], ins[2][0], ins[3][0], outs[0][0])
    bd.rec_attn_ffn_bwd(ins[0][0], ins[2][0], ins[3][0], ins[1][0], *(o[0] for o in outs[1:]))
    assert same([o[0] for o in outs], [y, dx, dwi, dwo])
    for v, buf, off in outs:
        assert (buf[:off] == 5).all() and (buf[off + v.numel():] == 5).all()


@pytest.mark.parametrize("rows", [2, 50, 200])
def test_scaled_outputs_end_with_their_rows(rows):
    t = serving(5, rows=rows)
    y, q, sc, z = serve(t)
    pad = lambda like: torch.full((like.shape[0] + 9,) + like.shape[1:], 5.0, device="cuda").to(like.dtype)
    y2, q2, s2, z2 = pad(y), pad(q), pad(sc), pad(z)
    bd.rec_attn_ffn_scaled_fwd(*t, y2[:rows])
    bd.rec_attn_scaled_quantize(t[0], q2.view(F8)[:rows], s2[:rows])
    bd.rec_attn_scaled_matmul(q2.view(F8)[:rows], s2[:rows], t[1], t[2], z2[:rows])
    assert same([y2[:rows], q2[:rows], s2[:rows], z2[:rows]], [y, q, sc, z])
    assert all((p[rows:].float() == 5).all() for p in (y2, s2, z2)) and (q2[rows:] == 5).all()


@pytest.mark.parametrize("rows", [6, 60, 300])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_a_row_that_is_not_finite_stays_alone(rows, kind):
    """NaN and infinity in some rows of x reach their own rows of y (and dx), and no other bit changes."""
    if kind == "e4m3":
        t = serving(6, rows=rows)
        run = lambda x: serve((x,) + t[1:])[:1]
    else:
        t = inputs(rows, 136, 264, BF if kind == "bf16" else F32)
        run = lambda x: train((x,) + t[1:])[:2]
    good = run(t[0])
    x = t[0].clone()
    x[1, 3], x[4, 7] = float("nan"), float("inf")
    bad = run(x)
    torch.cuda.synchronize()
    rest = [r for r in range(rows) if r not in (1, 4)]
    for g, b in zip(good, bad):
        assert torch.equal(g[rest], b[rest])
        assert torch.isnan(b[1]).all() and not torch.isfinite(b[4]).all()


def test_offsets_past_2_31():
    """p of the backward has 2^31 elements and more; rows at the end and the sums over all of them."""
    R, Wd, H = 1_100_003, 64, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy, wi, wo = rnd(R, Wd).to(BF), rnd(R, Wd).to(BF), (rnd(2 * H, Wd) / 8).to(BF), (rnd(Wd, H) / 32).to(BF)
    y, dx, dwi, dwo = train((x, dy, wi, wo))
    assert bd.rec_attn_dense_device_status() == bd.OK
    ref = reference(x[-300:], dy[-300:], wi, wo, "silu", 2.0**-8)
    within(y[-300:], ref["y"], "y")
    within(dx[-300:], ref["dx"], "dx")
    total, slack = 0, 0
    for r in range(0, R, 65536):
        ref = reference(x[r:r + 65536], dy[r:r + 65536], wi, wo, "silu", 2.0**-8)
        total, slack = total + ref["dw_out"][0], slack + ref["dw_out"][1]
    # (parts' tolerances add up; each has its own rounding of the result, which covers the one of the sum, and
    # the sum's longer chain is bounded by the rows' share of s(R))
    within(dwo, (total, slack + 2.0**-8 * total.abs() + R / 8 * 2.0**-22 * slack), "dw_out")


def test_scaled_offsets_past_2_31():
    R, K, N = 2_100_003, 1024, 1032
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(R, K, generator=g, device="cuda", dtype=BF)
    q, sc = quantize(x, 1)
    ref, rs = quantized(x[-200:].double(), 1)
    assert torch.equal(q[-200:].float().double(), ref) and torch.equal(sc[-200:].double(), rs)
    w, ws = quantize(torch.randn(N, K, generator=g, device="cuda") / 32, 128)
    y = torch.empty(R, N, dtype=BF, device="cuda")
    bd.rec_attn_scaled_matmul(q, sc, w, ws, y)
    torch.cuda.synchronize()
    A, B = held(q[-200:], sc[-200:], 1), held(w, ws, 128)
    want = A @ B.T
    over = (y[-200:].double() - want).abs() - 2.0**-8 * want.abs() - sums(K) * (A.abs() @ B.abs().T)
    assert over.max() <= 0


def test_with_the_attention_and_the_layer_norm():
    """A training step's half block: attention, layer norm, feed-forward, and back through all three; then the
    same rows served with e4m3 weights.  Each step is held to its own formula on what it was given."""
    w = W.mtgr(batch=3, hist=(150, 300), rt=(20, 60), cand=(10, 30), heads=8)
    t = gu.device_inputs(w)
    T, D, H = t["q"].shape[0], 512, 1024
    _, dy, wi, wo = inputs(T, D, H, BF, seed=4)
    gain, bias = torch.full((4, D), 1.25, device="cuda"), torch.full((4, D), -0.1, device="cuda")
    o, lse = torch.empty_like(t["q"]), torch.empty(T, 8, device="cuda")
    with bd.rec_attn_plan(gu.params_for(w), t["off_h"], t["off_d"], t["t"], t["ty"]) as plan:
        bd.rec_attn_fwd(plan, t["q"], t["k"], t["v"], o, lse)
        rows = o.view(T, D)
        n = torch.empty_like(rows)
        bd.rec_attn_layernorm_fwd(rows, gain, bias, n, types=t["ty"])
        y, dn, dwi, dwo = train((n, dy, wi, wo))
        do = torch.empty_like(rows)
        dgain, dbias = torch.empty_like(gain), torch.empty_like(bias)
        bd.rec_attn_layernorm_bwd(rows, gain, dn, do, dgain, dbias, types=t["ty"])
        dq, dk, dv = (torch.empty_like(t[c]) for c in "qkv")
        bd.rec_attn_bwd(plan, t["q"], t["k"], t["v"], o, lse, do.view_as(o), dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK and bd.rec_attn_dense_device_status() == bd.OK
    norm = norm_reference(rows, dn, gain, bias, t["ty"], 1e-5)
    norm_within(n, norm["y"], 2.0**-8)
    norm_within(do, norm["dx"], 2.0**-8)
    norm_within(dgain, norm["dw"], 2.0**-24)
    ref = reference(n, dy, wi, wo, "silu", 2.0**-8)
    for name, got in (("y", y), ("dx", dn), ("dw_in", dwi), ("dw_out", dwo)):
        within(got, ref[name], name)
    assert all(torch.isfinite(x).all() and x.abs().sum() > 0 for x in (dq, dk, dv))
    # served: the same rows on quantized weights, far from the bf16 result by no more than e4m3's three mantissa bits
    ys = torch.empty_like(n)
    qi, qis = quantize(wi, 128)
    qo, qos = quantize(wo, 128)
    bd.rec_attn_ffn_scaled_fwd(n, qi, qis, qo, qos, ys)
    torch.cuda.synchronize()
    # x, both weights and h are off by at most 2^-4 each: three of them in g, u and h = act(g) u, one more in w_out
    assert (ys.double() - y.double()).norm() <= 6 * 2.0**-4 * y.double().norm()


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import test_gpu_ffn_calls as t
run, tensors = {case}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run(tensors)
g.replay()
torch.cuda.synchronize()
assert t.same(out, run(tensors))
"""


@pytest.mark.parametrize("case", [
    "t.train, t.inputs(300, 136, 264, t.BF)", "t.train, t.inputs(3, 512, 1024, t.BF)", "t.train, t.inputs(40, 512, 1024, t.BF)",
    "t.train, t.inputs(150, 132, 68, t.F32)", "t.train, t.inputs(2, 132, 68, t.F32)", "t.quantize_and_product, t.raw(300)",
    "t.quantize_and_product, t.raw(3)", "t.quantize_and_product, t.raw(40)"])
def test_first_call_of_a_process_is_captured(case):
    import os
    import subprocess
    import sys
    code = FIRST.format(root=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), case=case)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def raw(rows):
    """Rows and weights that nothing of the library has touched."""
    g = torch.Generator().manual_seed(rows)
    return [torch.randn(s, generator=g).to(BF).cuda() for s in ((rows, 256), (512, 256), (256, 256))]


def quantize_and_product(t):
    def q(m, br):
        v, sc = torch.empty(m.shape, dtype=F8, device="cuda"), torch.empty(-(-m.shape[0] // br), m.shape[1] // 128, device="cuda")
        bd.rec_attn_scaled_quantize(m, v, sc, block_rows=br)
        return v, sc

    x, wi, wo = t
    a, b, c = q(x, 1), q(wi, 128), q(wo, 128)
    y, z = torch.empty_like(x), torch.empty(x.shape[0], 512, dtype=BF, device="cuda")
    bd.rec_attn_scaled_matmul(*a, *b, z)
    bd.rec_attn_ffn_scaled_fwd(x, *b, *c, y)
    return [z, y]


def test_a_few_rows_of_many_blocks():
    """Long summed axes for few rows (a cluster's CTAs go round their stages), and more columns than SMs."""
    for rows, width, hidden in ((2, 8192, 128), (20, 8192, 128), (60, 8192, 136), (33, 128, 40000), (5, 136, 40000)):
        t = inputs(rows, width, hidden, BF, seed=rows)
        y = torch.empty_like(t[0])
        bd.rec_attn_ffn_fwd(t[0], t[2], t[3], y)
        torch.cuda.synchronize()
        assert bd.rec_attn_dense_device_status() == bd.OK
        within(y, reference(*t, "silu", 2.0**-8)["y"], "y")
    for rows, cols, depth in ((3, 128, 40000), (40, 128, 40000), (64, 40000, 272), (7, 40000, 272), (200, 40, 131072)):
        g = torch.Generator().manual_seed(rows)
        a, asc = quantize(torch.randn(rows, depth, generator=g).cuda(), 1)
        b, bsc = quantize(torch.randn(cols, depth, generator=g).cuda(), 128)
        y = torch.full((rows, cols), float("nan"), dtype=BF, device="cuda")
        bd.rec_attn_scaled_matmul(a, asc, b, bsc, y)
        torch.cuda.synchronize()
        assert bd.rec_attn_dense_device_status() == bd.OK
        A, B = held(a, asc, 1), held(b, bsc, 128)
        want = A @ B.T
        assert ((y.double() - want).abs() <= 2.0**-8 * want.abs() + sums(depth) * (A.abs() @ B.abs().T) + 1e-30).all()


def test_largest_widths():
    """65536 wide, and e4m3 131072: few rows, and past a tile."""
    for rows in (3, 70, 300):
        t = inputs(rows, 65536, 64, BF, seed=rows)
        out = train(t)
        torch.cuda.synchronize()
        ref = reference(*t, "silu", 2.0**-8)
        for n, got in zip(("y", "dx", "dw_in", "dw_out"), out):
            within(got, ref[n], n)
        t = inputs(rows, 64, 65536, BF, seed=rows)
        out = train(t)
        torch.cuda.synchronize()
        ref = reference(*t, "silu", 2.0**-8)
        for n, got in zip(("y", "dx", "dw_in", "dw_out"), out):
            within(got, ref[n], n)


def test_binding_refuses_on_the_device():
    x, dy, wi, wo = inputs(4, 64, 128, BF)
    y = torch.empty_like(x)
    for bad in ((x.float(), wi, wo, y), (x, wi.float(), wo, y), (x, wi[:128], wo, y), (x, wi, wo.T, y), (x, wi, wo, y[:2]),
                (x.T, wi, wo, y), (x, wi.cpu(), wo, y), (x, wi, wo, x), (x[:, ::2], wi, wo, y), (x, None, wo, y)):
        with pytest.raises(bd.RecAttnError) as e:
            bd.rec_attn_ffn_fwd(*bad)
        assert e.value.code == bd.ERR_INVALID_ARG
    with pytest.raises(bd.RecAttnError):
        bd.rec_attn_ffn_fwd(x, wi, wo, y, activation="relu")
    with pytest.raises(bd.RecAttnError):
        bd.rec_attn_ffn_bwd(x, wi, wo, dy, dx=dy)
    with pytest.raises(bd.RecAttnError):
        bd.rec_attn_scaled_quantize(x, torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda"))
    assert bd.rec_attn_dense_device_status() == bd.OK


@pytest.mark.parametrize("size", [64.0, 1e9, 2.0**127])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [3, 24, 150])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_closed_gates(rows, act, dtype, size):
    """Hidden columns whose gate is far below zero, down to the types' lowest power of two: they add nothing, neither
    to y nor to dx (act and its slope are below 64 e^-64 there), and their weights have no gradient; the others are
    as if they were alone."""
    closed, hidden = 40, 264
    x, dy, wi, wo = inputs(rows, 136, hidden, dtype, 11)
    x[:, 0] = 1
    wi[:closed] = 0
    wi[:closed, 0] = -size
    y, dx, dwi, dwo = train((x, dy, wi, wo), act)
    assert same([], [])
    rest = torch.arange(2 * hidden, device="cuda") % hidden >= closed
    ref = reference(x, dy, wi[rest], wo[:, closed:], act, 2.0**-8 if dtype == BF else 2.0**-24)
    for got, name in ((y, "y"), (dx, "dx"), (dwi[rest], "dw_in"), (dwo[:, closed:], "dw_out")):
        within(got, ref[name], name)
    for got in (dwi[~rest], dwo[:, :closed]):
        assert got.double().abs().max() < 1e-20


@pytest.mark.parametrize("size", [64.0, 1e9, 2.0**127])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [3, 24, 150])
def test_closed_gates_scaled(rows, act, size):
    """As if the up projections of the closed columns were zero."""
    closed, hidden, width = 128, 256, 144
    g = torch.Generator().manual_seed(12)
    x = torch.randn(rows, width, generator=g).to(BF).cuda()
    x[:, 0] = 1
    wi = (torch.randn(2 * hidden, width, generator=g) / 12).cuda()
    wi[:closed] = 0
    wi[:closed, 0] = -size
    wo = quantize((torch.randn(width, hidden, generator=g) / 16).cuda(), 128)
    out = []
    for up in (1, 0):
        wi[hidden : hidden + closed] *= up
        y = torch.full_like(x, 7)
        bd.rec_attn_ffn_scaled_fwd(x, *quantize(wi, 128), *wo, y, activation=act)
        out.append(y)
    assert same(out[:1], out[1:])
