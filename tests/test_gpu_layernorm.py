"""Layer norm by token type (rec_attn_layernorm_fwd / _bwd) vs the formulas in 64 bits.

Tolerances, from the formulas' roundings (e = 2^-24 for fp32 arithmetic, h = half a step of
the output type: 2^-8 bf16, 2^-24 fp32):
  y    n = (x - m) r carries a few e relative plus the mean's error e |m| r (sums of W terms by
       a tree of depth ~ 16 + 5 + W / 16 threads' warps: below 64 e max|x|), so
       |dy| <= h |y| + 64 e (|x|max r + 1) |w| + e (|n w| + |b|).
  dx   the same, once more through two means: |ddx| <= h |dx| + 256 e r (max|u| + max|u| n^2max).
  dw   sums over R rows in chains of at most R / blocks rows and then over the blocks; each
       term carries about 64 e: |ddw| <= (64 + chain) e sum |dy n| + 64 e sum |dy|(|x|max r + 1),
       taken with chain = 2048 (more rows than any group of threads adds up here).
  db   the same without the normalisation: |ddb| <= 2048 e sum |dy|."""
import numpy as np
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd

pytestmark = pytest.mark.gpu
E32 = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def inputs(rows, width, dtype, by_type, seed=0, runs=True, offset=0.25):
    g = torch.Generator().manual_seed(seed)
    types = 4 if by_type else 1
    x = (torch.randn(rows, width, generator=g) * 1.5 + offset).to(dtype).cuda()
    dy = torch.randn(rows, width, generator=g).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(types, width, generator=g)).cuda()
    b = (0.1 * torch.randn(types, width, generator=g)).cuda()
    ty = None
    if by_type:
        ty = torch.arange(rows) * 13 % 97 // 25 if runs else torch.randint(0, 4, (rows,), generator=g)
        ty = ty.to(torch.int8).cuda()
    return x, dy, w, b, ty


def reference(x, dy, w, b, ty, eps):
    """Outputs in 64 bits, with the sums of absolute terms the tolerances use."""
    x, dy, w, b = (a.double() for a in (x, dy, w, b))
    rows, types = x.shape[0], w.shape[0]
    ty = torch.zeros(rows, dtype=torch.long, device=x.device) if ty is None else ty.long()
    ok = (ty >= 0) & (ty < types)
    gi = torch.where(ok, ty, 0)
    m = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps)
    n = (x - m) * r
    W, B, keep = w[gi], b[gi], ok[:, None].double()
    y = (n * W + B) * keep
    u = dy * W
    dx = r * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True)) * keep
    z = torch.zeros_like(w)
    xr = x.abs().amax(1, keepdim=True) * r + 1 if x.shape[1] else r
    out = {"y": (y, 64 * E32 * xr * W.abs() + E32 * ((n * W).abs() + B.abs())),
           "dx": (dx, 256 * E32 * r * u.abs().amax(1, keepdim=True) * (1 + n.abs().amax(1, keepdim=True) ** 2 + xr))}
    add = lambda t: z.index_add(0, gi, t * keep)
    out["dw"] = (add(dy * n), (64 + 2048) * E32 * add((dy * n).abs()) + 64 * E32 * add(dy.abs() * xr) + 1e-30)
    out["db"] = (add(dy), 2048 * E32 * add(dy.abs()) + 1e-30)
    return out


def within(got, ref, half):
    r, slack = ref
    x = got.double()
    assert torch.isfinite(x).all()
    over = (x - r).abs() - (half * r.abs() + slack)
    assert over.max() <= 0, float(over.max())


def run(x, dy, w, b, ty, eps, dweight=True, dbias=True):
    y, dx = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    dw, db = torch.full_like(w, float("nan")), torch.full_like(w, float("nan"))
    bd.rec_attn_layernorm_fwd(x, w, b, y, types=ty, eps=eps)
    bd.rec_attn_layernorm_bwd(x, w, dy, dx, dw if dweight else None, db if dbias else None, types=ty, eps=eps)
    torch.cuda.synchronize()
    return y, dx, dw, db


SHAPES = [(1, 8), (1, 512), (3, 64), (301, 512), (77, 136), (1000, 352), (129, 264), (65, 1408), (33, 2048),
          (19, 4104), (7, 8192), (5, 16384), (4099, 512), (20011, 64)]


@pytest.mark.parametrize("by_type", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_against_64_bits(rows, width, dtype, by_type):
    x, dy, w, b, ty = inputs(rows, width, dtype, by_type)
    y, dx, dw, db = run(x, dy, w, b, ty, 1e-5)
    ref = reference(x, dy, w, b, ty, 1e-5)
    half = torch.finfo(dtype).eps / 2
    within(y, ref["y"], half)
    within(dx, ref["dx"], half)
    within(dw, ref["dw"], E32)
    within(db, ref["db"], E32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_types_in_any_order_absent_and_out_of_range(dtype):
    """A type per row at random (every row may change it), one type absent, some rows of none."""
    x, dy, w, b, ty = inputs(5003, 264, dtype, True, seed=3, runs=False)
    ty[ty == 2] = 1
    ty[5::97] = 4
    ty[6::97] = -1
    ty[7::97] = 127
    y, dx, dw, db = run(x, dy, w, b, ty, 1e-5)
    ref = reference(x, dy, w, b, ty, 1e-5)
    half = torch.finfo(dtype).eps / 2
    for got, n, h in ((y, "y", half), (dx, "dx", half), (dw, "dw", E32), (db, "db", E32)):
        within(got, ref[n], h)
    none = ((ty < 0) | (ty > 3))
    assert (y[none] == 0).all() and (dx[none] == 0).all()
    assert (dw[2] == 0).all() and (db[2] == 0).all()


def test_rows_far_from_zero():
    """A mean of 1000 standard deviations in fp32: the variance comes from the differences."""
    x, dy, w, b, ty = inputs(64, 512, torch.float32, False, offset=1500.0)
    y, dx, dw, db = run(x, dy, w, b, ty, 1e-5)
    ref = reference(x, dy, w, b, ty, 1e-5)
    within(y, ref["y"], E32)
    within(dx, ref["dx"], E32)


def test_constant_rows_and_zero_eps():
    """A constant row has no spread: with eps its output is the bias, exactly."""
    x = torch.full((9, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    w, b = torch.ones(1, 512, device="cuda"), torch.full((1, 512), 0.5, device="cuda")
    y = torch.empty_like(x)
    bd.rec_attn_layernorm_fwd(x, w, b, y, eps=1e-5)
    assert (y == 0.5).all()
    x, dy, w, b, ty = inputs(9, 512, torch.float32, False)
    y, dx, dw, db = run(x, dy, w, b, ty, 0.0)
    within(y, reference(x, dy, w, b, ty, 0.0)["y"], E32)


def test_nan_and_infinite_rows_stay_in_their_rows():
    x, dy, w, b, ty = inputs(40, 512, torch.bfloat16, False)
    clean = run(x, dy, w, b, ty, 1e-5)
    x[7, 100], x[21, 3] = float("nan"), float("inf")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    bd.rec_attn_layernorm_fwd(x, w, b, y)
    bd.rec_attn_layernorm_bwd(x, w, dy, dx)
    rest = torch.tensor([i for i in range(40) if i not in (7, 21)], device="cuda")
    assert torch.equal(y[rest], clean[0][rest]) and torch.equal(dx[rest], clean[1][rest])
    assert torch.isnan(y[[7, 21]].float()).all() and torch.isnan(dx[[7, 21]].float()).all()


@pytest.mark.parametrize("by_type", [False, True])
def test_in_place_no_bias_and_unwanted_gradients(by_type):
    x, dy, w, b, ty = inputs(1003, 512, torch.bfloat16, by_type)
    y, dx, dw, db = run(x, dy, w, torch.zeros_like(b), ty, 1e-5)
    z, g = x.clone(), dy.clone()
    bd.rec_attn_layernorm_fwd(z, w, None, z, types=ty)  # y over x, no bias
    assert torch.equal(z, y)
    only = torch.full_like(w, float("nan"))
    bd.rec_attn_layernorm_bwd(x, w, g, g, only, None, types=ty)  # dx over dy, no dbias
    assert torch.equal(g, dx) and torch.equal(only, dw)
    z = x.clone()
    bd.rec_attn_layernorm_bwd(z, w, dy, z, None, only, types=ty)  # dx over x, no dweight
    assert torch.equal(z, dx) and torch.equal(only, db)


def test_no_rows():
    w = torch.ones(4, 64, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ty = torch.empty(0, dtype=torch.int8, device="cuda")
    dw, db = torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    bd.rec_attn_layernorm_fwd(x, w, None, x, types=ty)
    bd.rec_attn_layernorm_bwd(x, w, x, x, dw, db, types=ty)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    x, dy, w, b, ty = inputs(9001, 512, torch.bfloat16, True, runs=False)
    first = run(x, dy, w, b, ty, 1e-5)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    torch.cuda.synchronize()
    for s in (s1, s2):
        with torch.cuda.stream(s):
            dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
            bd.rec_attn_layernorm_bwd(x, w, dy, dx, dw, db, types=ty)
            got.append((dx, dw, db))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, c) for a, c in zip(g, first[1:]))
    dx, dw, db, y = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.rec_attn_layernorm_fwd(x, w, b, y, types=ty)
        bd.rec_attn_layernorm_bwd(x, w, dy, dx, dw, db, types=ty)
    for _ in range(3):
        for a in (dx, dw, db, y):
            a.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((y, dx, dw, db), first))


def test_gradient_against_differences():
    """dx, dw and db against central differences of the 64-bit forward on a few entries."""
    x, dy, w, b, ty = inputs(6, 64, torch.float32, True)
    _, dx, dw, db = run(x, dy, w, b, ty, 1e-5)

    def loss(xx, ww, bb):
        return float((reference(xx, dy, ww, bb, ty, 1e-5)["y"][0] * dy.double()).sum())

    h = 1e-5  # error of the difference: h^2 times a third derivative below ~1e2, plus 1e-16 / h
    for i, j in ((0, 0), (3, 17), (5, 63)):
        t = int(ty[i])
        for a, got, at in ((0, dx, (i, j)), (1, dw, (t, j)), (2, db, (t, j))):
            v = [x.double(), w.double(), b.double()]
            up, dn = [z.clone() for z in v], [z.clone() for z in v]
            up[a][at] += h
            dn[a][at] -= h
            d = (loss(*up) - loss(*dn)) / (2 * h)
            assert abs(d - float(got[at])) <= 1e-5 * (1 + abs(d)), (a, at, d, float(got[at]))
