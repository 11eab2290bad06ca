"""Gated feed-forward block (rec_attn_ffn_fwd / _bwd) vs the formulas in 64 bits.

Tolerances, from the roundings (h = half a step of the type: 2^-8 bf16, 2^-24 fp32).  A sum of K
products in fp32 carries at most s(K) = (K / 8 + 16) 2^-22 of the sum of their absolute values: the
tensor cores add 16 products at a time to a sum that may lose a step of 2^-23 each time, taken four
times over.  (fp32 inputs are summed no worse.)  act and its slope carry a(g) = (|g| + 4) 2^-22
relative to |act| + |slope| g-wise (the exponential's argument is rounded in fp32).
  g, u     dg = s(W) sum |x||w|, du alike
  h        dh = |act'| dg |u| + |act| du + a(g) (1 + |g|) |u| + h |h|
  y        h |y| + sum dh |w_out| + s(H) sum |h||w_out|
  dh       e = s(W) sum |dy||w_out|
  p        each factor's error times the others, with |act''| <= 1, and h |p|
  dx, dw   h |.| + sum (dp |.|) + s(K) sum |p||.|"""
import ctypes
import math

import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def inputs(rows, width, hidden, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g).to(dtype).cuda()
    dy = torch.randn(rows, width, generator=g).to(dtype).cuda()
    w_in = (torch.randn(2 * hidden, width, generator=g) / math.sqrt(width) * 1.5).to(dtype).cuda()
    w_out = (torch.randn(width, hidden, generator=g) / math.sqrt(hidden)).to(dtype).cuda()
    return x, dy, w_in, w_out


def s(k):
    return (k / 8 + 16) * 2.0**-22


def act_both(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def reference(x, dy, w_in, w_out, act, half):
    """{name: (value, tolerance)} in 64 bits."""
    x, dy, wi, wo = (t.double() for t in (x, dy, w_in, w_out))
    R, W = x.shape
    H = wo.shape[1]
    wg, wu = wi[:H], wi[H:]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = s(W) * (x.abs() @ wg.abs().T), s(W) * (x.abs() @ wu.abs().T)
    a, sl = act_both(g, act)
    ea = (g.abs() + 4) * (1 + g.abs()) * 2.0**-22
    h = a * u
    eh = 1.13 * eg * u.abs() + a.abs() * eu + ea * u.abs() + half * h.abs()
    y = h @ wo.T
    out = {"y": (y, half * y.abs() + eh @ wo.abs().T + s(H) * (h.abs() @ wo.abs().T))}
    dh = dy @ wo
    edh = s(W) * (dy.abs() @ wo.abs())
    dg, du = dh * u * sl, dh * a
    edg = (edh * (u * sl).abs() + eu * (dh * sl).abs() + (eg + ea) * (dh * u).abs()) * 1.01 + half * dg.abs()
    edu = (edh * a.abs() + (1.13 * eg + ea) * dh.abs()) * 1.01 + half * du.abs()
    p, ep = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    dx, dwi, dwo = p @ wi, p.T @ x, dy.T @ h
    out["dx"] = (dx, half * dx.abs() + ep @ wi.abs() + s(2 * H) * (p.abs() @ wi.abs()))
    out["dw_in"] = (dwi, half * dwi.abs() + ep.T @ x.abs() + s(R) * (p.abs().T @ x.abs()))
    out["dw_out"] = (dwo, half * dwo.abs() + dy.abs().T @ eh + s(R) * (dy.abs().T @ h.abs()))
    return out


def within(got, ref, name):
    value, tol = ref
    assert torch.isfinite(got).all(), name
    over = (got.double() - value).abs() - tol - 1e-30
    assert over.max() <= 0, (name, float(over.max()), float(value.abs().max()))


def run(x, dy, w_in, w_out, act, wanted=("dx", "dw_in", "dw_out")):
    out = {"y": torch.full_like(x, float("nan")), "dx": torch.full_like(x, float("nan")),
           "dw_in": torch.full_like(w_in, float("nan")), "dw_out": torch.full_like(w_out, float("nan"))}
    bd.rec_attn_ffn_fwd(x, w_in, w_out, out["y"], activation=act)
    bd.rec_attn_ffn_bwd(x, w_in, w_out, dy, *(out[n] if n in wanted else None for n in ("dx", "dw_in", "dw_out")),
                        activation=act)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    return out


SHAPES = [(1, 8, 8), (1, 512, 1024), (5, 64, 128), (127, 72, 136), (128, 128, 128), (129, 200, 72), (300, 520, 264),
          (77, 1408, 8), (513, 256, 1000), (2000, 64, 64), (1031, 512, 1024),
          (90, 520, 2056), (260, 264, 4096)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width,hidden", SHAPES)
def test_against_64_bits(rows, width, hidden, dtype, act):
    if dtype == torch.float32 and rows % 2:  # (a row of four values is 16 bytes)
        width, hidden = width + 4, hidden + 12
    t = inputs(rows, width, hidden, dtype, seed=rows)
    out = run(*t, act)
    ref = reference(*t, act, torch.finfo(dtype).eps / 2)
    for n in ("y", "dx", "dw_in", "dw_out"):
        within(out[n], ref[n], n)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 3, 7, 8, 9, 16, 17, 24, 25, 31, 32, 33, 64, 65, 127])
def test_few_rows(rows, dtype, act):
    """Row counts about the borders of the few-row kernels, columns and summed axes off their blocks."""
    for width, hidden in ((72, 1096), (1160, 24), (200, 136)):
        t = inputs(rows, width, hidden, dtype, seed=rows)
        y = torch.full_like(t[0], float("nan"))
        bd.rec_attn_ffn_fwd(t[0], t[2], t[3], y, activation=act)
        torch.cuda.synchronize()
        assert bd.rec_attn_dense_device_status() == bd.OK
        within(y, reference(*t, act, torch.finfo(dtype).eps / 2)["y"], "y")
