"""The feed-forward block's activation and its slope over the whole range of the gate: open gates of any size,
whose slope is 1, and gelu's tail below zero.  Tolerances as in test_gpu_ffn.py, but for the gates that these
tests set: their g is exact, so that no bound grows with its size.

The activation of a set gate is off by at most 2^-11 relative (gelu's tail: its form is off by 4e-4, and by what
rounding the exponential's argument, at most 104, does: 104 2^-23 ln 2), silu's and open gates' by 2^-20 (two
roundings of the exponential and the reciprocal, 2^-22 each)."""
import math

import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import act_both, inputs, s, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def train(x, dy, wi, wo, act):
    o = [torch.full_like(x, 7), torch.full_like(x, 7), torch.full_like(wi, 7), torch.full_like(wo, 7)]
    bd.rec_attn_ffn_fwd(x, wi, wo, o[0], activation=act)
    bd.rec_attn_ffn_bwd(x, wi, wo, dy, *o[1:], activation=act)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    return dict(zip(("y", "dx", "dw_in", "dw_out"), o))


@pytest.mark.parametrize("size", [1e4, 1e6, 1e9, 2.0**100])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [3, 24, 150])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_open_gates(rows, act, dtype, size):
    """Every second hidden column has a gate of `size` exactly, its neighbour an ordinary one (the two share a
    reciprocal in bf16): act(g) = g and the slope is 1 to every bit that the result has."""
    hidden, half = 264, torch.finfo(dtype).eps / 2
    x, dy, wi, wo = inputs(rows, 136, hidden, dtype, 21)
    x[:, 0] = 1
    wi[:hidden:2] = 0
    wi[:hidden:2, 0] = size
    wi[hidden::2, 0] = 0  # (so that dx[:, 0] holds the open gates' slopes alone, times their size)
    got = train(x, dy, wi, wo, act)
    X, DY, WI, WO = (t.double() for t in (x, dy, wi, wo))
    opened = torch.arange(hidden, device="cuda") % 2 == 0
    g, u = X @ WI[:hidden].T, X @ WI[hidden:].T
    eu = s(136) * (X.abs() @ WI[hidden:].abs().T)
    eg = torch.where(opened, 0.0, s(136) * (X.abs() @ WI[:hidden].abs().T))
    a, sl = act_both(g, act)
    a, sl = torch.where(opened, g, a), torch.where(opened, torch.ones_like(sl), sl)
    ea = torch.where(opened, g.abs() * 2.0**-20, (g.abs() + 4) * (1 + g.abs()) * 2.0**-22)
    es = torch.where(opened, 2.0**-20, ea)
    h = a * u
    eh = 1.13 * eg * u.abs() + a.abs() * eu + ea * u.abs() + half * h.abs()
    within(got["y"], (h @ WO.T, half * (h @ WO.T).abs() + eh @ WO.abs().T + s(hidden) * (h.abs() @ WO.abs().T)), "y")
    dh, edh = DY @ WO, s(136) * (DY.abs() @ WO.abs())
    dg, du = dh * u * sl, dh * a
    edg = (edh * (u * sl).abs() + eu * (dh * sl).abs() + (eg + es) * (dh * u).abs()) * 1.01 + half * dg.abs()
    edu = (edh * a.abs() + (1.13 * eg + ea) * dh.abs()) * 1.01 + half * du.abs()
    for name, v, e in (("dw_in gate", dg, edg), ("dw_in up", du, edu)):
        part = slice(0, hidden) if name.endswith("gate") else slice(hidden, None)
        ref = v.T @ X
        within(got["dw_in"][part], (ref, half * ref.abs() + e.T @ X.abs() + s(rows) * (v.abs().T @ X.abs())), name)
    ref = DY.T @ h
    within(got["dw_out"], (ref, half * ref.abs() + DY.abs().T @ eh + s(rows) * (DY.abs().T @ h.abs())), "dw_out")
    p, ep = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    ref = p @ WI
    within(got["dx"], (ref, half * ref.abs() + ep @ WI.abs() + s(2 * hidden) * (p.abs() @ WI.abs())), "dx")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [3, 24, 150])
def test_tail_below_zero(rows, act):
    """Gates from -4 to -12, one a column, with u = 1, w_out and dh = 1: y is h itself, the up rows of dw_in act(g) and
    the gate rows the slope.  Each has one rounding (2^-8) and the activation's 2^-11, relative to the value itself;
    silu's cut of its weight by 2^-60 and a bit is added."""
    n = 264
    gates = torch.linspace(-4, -12, n).to(BF)
    x = torch.zeros(rows, n, dtype=BF, device="cuda")
    wi = torch.zeros(2 * n, n, dtype=BF, device="cuda")
    wi[:n, 0], wi[n:, 1] = gates.cuda(), 1
    wo = torch.eye(n, dtype=BF, device="cuda")
    dy = torch.ones(rows, n, dtype=BF, device="cuda")
    x[:, :2] = 1
    g = gates.double().cuda()
    if act == "gelu":  # (Phi by erfc: a difference from 1 would lose the tail)
        a, slope = (torch.special.erfc(-g / math.sqrt(2)) / 2,) * 2
        a, slope = g * a, slope + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        a, slope = act_both(g, act)
    cut = 2.0**-59 * 16 if act == "silu" else 0.0
    tol = 2.0**-8 + 2.0**-11
    y = train(x, dy, wi, wo, act)["y"]
    within(y, (a.expand(rows, n), tol * a.abs() + cut), "y")
    x[: rows - 1] = 0  # one row: its p is the gradient
    dw = train(x, dy, wi, wo, act)["dw_in"]
    within(dw[n:, 1], (a, tol * a.abs() + cut), "up")
    within(dw[:n, 0], (slope, tol * slope.abs() + cut), "gate")
