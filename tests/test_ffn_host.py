"""What the feed-forward and scaled calls refuse on the host, before any CUDA call (no GPU), and the
formulas of their gradients against differences in 64 bits."""
import math

import pytest
import torch

from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import build as bld

X, WI, WO, Y, DX, DWI, DWO, DY = ((1 << 40) + (i << 36) for i in range(8))
INV, UNS = bd.ERR_INVALID_ARG, bd.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    bld.build()
    return bd.lib()


def fwd(L, dtype=0, act=0, rows=4, width=64, hidden=64, x=X, wi=WI, wo=WO, y=Y):
    return L.rec_attn_ffn_fwd(dtype, act, rows, width, hidden, x, wi, wo, y, None)


def bwd(L, dtype=0, act=0, rows=4, width=64, hidden=64, x=X, wi=WI, wo=WO, dy=DY, dx=DX, dwi=DWI, dwo=DWO):
    return L.rec_attn_ffn_bwd(dtype, act, rows, width, hidden, x, wi, wo, dy, dx, dwi, dwo, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_ffn_refusals(L, call):
    for bad in (dict(dtype=2), dict(dtype=-1), dict(act=2), dict(act=-1), dict(rows=-1), dict(width=0), dict(hidden=0),
                dict(width=12), dict(hidden=60), dict(width=-8), dict(dtype=1, width=6), dict(dtype=1, hidden=2)):
        assert call(L, **bad) == INV, bad
    for big in (dict(width=65544), dict(hidden=65544), dict(rows=1 << 31), dict(rows=(1 << 31) - 65536, hidden=65536)):
        assert call(L, **big) == UNS, big
    for p in ("x", "wi", "wo"):
        assert call(L, **{p: None}) == INV, p
        assert call(L, **{p: X + 8}) == INV, p  # misaligned
    if call is fwd:
        assert call(L, y=None) == INV and call(L, y=Y + 2) == INV
        assert call(L, rows=0, x=None, y=None) == bd.OK  # nothing to do
        for y in (X, X + 4 * 64 * 2 - 16, WI, WI + 16, WO):
            assert call(L, y=y) == INV
    else:
        assert call(L, dy=None) == INV
        for o in ("dx", "dwi", "dwo"):
            assert call(L, **{o: Y + 4}) == INV, o
            for other in (X, WI, WO, DY):
                assert call(L, **{o: other}) == INV, (o, other)
        assert call(L, dx=DWI) == INV and call(L, dwi=DWO) == INV and call(L, dwo=DWI + 64) == INV


def test_scaled_refusals(L):
    q = lambda dtype=0, br=1, rows=4, width=64, x=X, q=Y, s=DX: L.rec_attn_scaled_quantize(dtype, br, rows, width, x, q, s, None)
    for bad in (dict(dtype=3), dict(br=2), dict(br=0), dict(rows=-1), dict(width=0), dict(width=8), dict(width=24),
                dict(x=None), dict(q=None), dict(s=None), dict(x=X + 8), dict(q=Y + 1), dict(s=DX + 4), dict(q=X),
                dict(s=X + 16), dict(s=Y)):
        assert q(**bad) == INV, bad
    assert q(width=131088) == UNS and q(rows=1 << 31) == UNS
    assert q(rows=0, x=None) == bd.OK
    m = lambda rows=4, cols=64, depth=64, a=X, sa=WI, b=WO, sb=DX, y=Y: L.rec_attn_scaled_matmul(rows, cols, depth, a, sa, b,
                                                                                                sb, y, None)
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=12), dict(depth=0), dict(depth=24), dict(a=None), dict(sa=None),
                dict(b=None), dict(sb=None), dict(y=None), dict(a=X + 8), dict(sa=WI + 4), dict(b=WO + 1), dict(sb=DX + 4),
                dict(y=Y + 2), dict(y=X), dict(y=WI), dict(y=WO), dict(y=DX)):
        assert m(**bad) == INV, bad
    assert m(depth=131088) == UNS and m(cols=131080) == UNS and m(rows=1 << 31) == UNS
    assert m(rows=0, a=None) == bd.OK
    f = lambda act=0, rows=4, width=64, hidden=128, x=X, wi=WI, si=DX, wo=WO, so=DY, y=Y: L.rec_attn_ffn_scaled_fwd(
        act, rows, width, hidden, x, wi, si, wo, so, y, None)
    for bad in (dict(act=2), dict(rows=-1), dict(width=8), dict(width=0), dict(hidden=64), dict(hidden=0), dict(x=None),
                dict(wi=None), dict(si=None), dict(wo=None), dict(so=None), dict(y=None), dict(x=X + 8), dict(si=DX + 4),
                dict(y=X), dict(y=WI), dict(y=DX), dict(y=WO), dict(y=DY)):
        assert f(**bad) == INV, bad
    assert f(width=65552) == UNS and f(hidden=65664) == UNS
    assert f(rows=0, x=None) == bd.OK
    assert L.rec_attn_dense_device_status(None, None) == INV


def test_binding_refusals():
    """Shapes, types and places that do not belong together, on CPU tensors: refused before the library."""
    bf, f32 = torch.bfloat16, torch.float32
    x, wi, wo = torch.zeros(3, 64, dtype=bf), torch.zeros(128, 64, dtype=bf), torch.zeros(64, 64, dtype=bf)
    for call in (lambda: bd.rec_attn_ffn_fwd(x, wi, wo, torch.zeros_like(x)),
                 lambda: bd.rec_attn_ffn_fwd(x, wi, None, torch.zeros_like(x)),
                 lambda: bd.rec_attn_ffn_bwd(x, wi, wo, torch.zeros_like(x)),
                 lambda: bd.rec_attn_scaled_quantize(x, x, x),
                 lambda: bd.rec_attn_scaled_matmul(x, x, wi, wi, x),
                 lambda: bd.rec_attn_ffn_scaled_fwd(x, wi, wi, wo, wo, x)):
        with pytest.raises(bd.RecAttnError) as e:
            call()
        assert e.value.code == INV


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_formulas_against_differences(act):
    """p, dx, dw_in and dw_out as the header has them, against central differences of sum(y c) in 64 bits."""
    torch.manual_seed(3)
    R, W, H = 5, 8, 12
    x, wi, wo, c = (torch.randn(*s, dtype=torch.float64) for s in ((R, W), (2 * H, W), (W, H), (R, W)))

    def value(g):
        return g * torch.sigmoid(g) if act == "silu" else g * torch.special.ndtr(g)

    def loss(x, wi, wo):
        pre = x @ wi.T
        return ((value(pre[:, :H]) * pre[:, H:]) @ wo.T * c).sum()

    pre = x @ wi.T
    g, u = pre[:, :H], pre[:, H:]
    if act == "silu":
        slope = torch.sigmoid(g) * (1 + g * (1 - torch.sigmoid(g)))
    else:
        slope = torch.special.ndtr(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    dh = c @ wo
    p = torch.cat((dh * u * slope, dh * value(g)), 1)
    grads = (p @ wi, p.T @ x, c.T @ (value(g) * u))
    for k, grad in enumerate(grads):
        for _ in range(4):
            d = torch.randn_like(grad)
            args, step = [x, wi, wo], 1e-5
            args[k] = args[k] + step * d
            up = loss(*args)
            args[k] = args[k] - 2 * step * d
            diff = (up - loss(*args)) / (2 * step)
            # (the differences are off by step^2 of the third derivative and 2^-53 / step of the loss)
            assert abs(diff - (grad * d).sum()) <= 1e-6 * (1 + grad.abs().sum() * d.abs().max())
