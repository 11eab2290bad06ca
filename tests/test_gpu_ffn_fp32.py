"""What the fp32 feed-forward block has to keep of its values, which go through the tensor cores as three bf16 planes:
every bit, so that results are off by a few 2^-24 in norm.

The bound is 1e-6 of each result's norm.  One product of two matrices: pairs left out (mid lo, lo mid, lo lo) 2^-25 of a
product at most; a block of 64 is summed in 24 additions of 16 products, of which the last four have the whole size (small
planes go first), each cut by half a step of 2^-23 of a sum that is half there on average: 2^-23; blocks are added up
rounded to nearest, 2^-25 of the sum for each, in either direction: 2^-25 sqrt(80).  That is 1.2e-7 and 2.7e-7 (for the
longest axis here, mostly 6e-8), 3e-7 together; y has two products in a row, the gradients three, whose errors meet as
squares: 5e-7, and the activation's 2^-22 for single values.  Two planes instead of three are off by 2^-17 a product, which
the first test shows to be eight times the bound; a whole axis in one cut sum is off by 2^-25 for 16 products."""
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import act_both, inputs

F32 = torch.float32
BOUND = 1e-6
NAMES = ("y", "dx", "dw_in", "dw_out")


def block(product, x, dy, wi, wo, act, keep=lambda v: v):
    """y, dx, dw_in, dw_out in 64 bits with `product(a, b)` for a b', and `keep` of what stands between products."""
    h_cols = wo.shape[1]
    pre = product(x, wi)
    g, u = pre[:, :h_cols], pre[:, h_cols:]
    a, slope = act_both(g, act)
    h, dh = keep(a * u), product(dy, wo.T)
    p = keep(torch.cat((dh * u * slope, dh * a), 1))
    return product(h, wo), product(p, wi.T), product(p.T, x.T), product(dy.T, h.T)


def off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def planes(v):
    hi = v.float().bfloat16().double()
    mid = (v - hi).float().bfloat16().double()
    return hi, mid, (v - hi - mid).float().bfloat16().double()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_bound_tells_three_planes_from_two(act):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g).double()  # (fp32 values)
    x, dy, wi, wo = rnd(90, 200), rnd(90, 200), rnd(272, 200).float().div(14).double(), rnd(200, 136).float().div(12).double()
    ref = block(lambda a, b: a @ b.T, x, dy, wi, wo, act)

    def pairs(a, b, which):
        a, b = planes(a), planes(b)
        return sum(a[i] @ b[j].T for i, j in which)

    six = block(lambda a, b: pairs(a, b, [(0, 2), (1, 1), (2, 0), (0, 1), (1, 0), (0, 0)]), x, dy, wi, wo, act, lambda v: v.float().double())
    three = block(lambda a, b: pairs(a, b, [(0, 1), (1, 0), (0, 0)]), x, dy, wi, wo, act, lambda v: v.float().double())
    no_mid = block(lambda a, b: pairs(a, b, [(0, 2), (2, 0), (0, 1), (1, 0), (0, 0)]), x, dy, wi, wo, act, lambda v: v.float().double())
    for k, name in enumerate(NAMES):
        assert off(six[k], ref[k]) < BOUND / 4 < BOUND < min(off(three[k], ref[k]), off(no_mid[k], ref[k])), name


@pytest.fixture(scope="module")
def built():
    gu.ensure_built()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7F800001, 0x7F80FFFF, 0x7FC00000, -0x7FFFFF])  # (the last: 0xff800001)
@pytest.mark.parametrize("rows", [3, 20, 200])
def test_nan_of_any_payload_stays_nan(built, rows, bits):
    """NaN whose payload is in the low half: its leading plane is NaN too, not the infinity of its upper half.  The
    weights' planes are all above zero, so that no product of an infinity would make up for it."""
    w = 1 + 2.0**-9 + 2.0**-18
    x = torch.full((rows, 8), 0.5, device="cuda")
    x.view(torch.int32)[1, 3] = bits
    wi, wo = torch.full((32, 8), w, device="cuda"), torch.full((8, 16), w, device="cuda")
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dwi, dwo = torch.zeros_like(wi), torch.zeros_like(wo)
    bd.rec_attn_ffn_fwd(x, wi, wo, y)
    bd.rec_attn_ffn_bwd(x, wi, wo, torch.full_like(x, w), dx, dwi, dwo)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all() and torch.isnan(dx[1]).all() and torch.isnan(dwi).any() and torch.isnan(dwo).all()
    rest = [r for r in range(rows) if r != 1]
    assert torch.isfinite(y[rest]).all() and torch.isfinite(dx[rest]).all()


SHAPES = [(9, 64, 128), (20, 132, 68), (129, 200, 72), (300, 520, 268), (2000, 64, 64), (1031, 512, 1024), (260, 264, 4096),
          (90, 1416, 264), (5003, 132, 204), (64, 4, 12), (257, 8, 4100)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,width,hidden", SHAPES)
def test_fp32_precision(built, rows, width, hidden, act):
    x, dy, wi, wo = inputs(rows, width, hidden, F32, seed=rows)
    got = [torch.full_like(t, float("nan")) for t in (x, x, wi, wo)]
    bd.rec_attn_ffn_fwd(x, wi, wo, got[0], activation=act)
    bd.rec_attn_ffn_bwd(x, wi, wo, dy, *got[1:], activation=act)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    ref = block(lambda a, b: a @ b.T, x.double(), dy.double(), wi.double(), wo.double(), act)
    for k, name in enumerate(NAMES):
        e = off(got[k], ref[k])
        print(name, e)
        assert e < BOUND, (name, e)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [1, 2, 3, 8])
def test_fp32_precision_of_few_rows(built, rows, act):
    """(CUDA cores: a lane's sums of a 1024th of the axis, joined in a tree.)"""
    for width, hidden in ((72, 1096), (4096, 136)):
        x, dy, wi, wo = inputs(rows, width, hidden, F32, seed=rows)
        y = torch.full_like(x, float("nan"))
        bd.rec_attn_ffn_fwd(x, wi, wo, y, activation=act)
        ref = block(lambda a, b: a @ b.T, x.double(), dy.double(), wi.double(), wo.double(), act)
        assert off(y, ref[0]) < BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32], ids=["bf16", "fp32"])
def test_small_gradients(built, dtype):
    """The backward is linear in dy, and powers of two move no rounding: 2^-60 dy gives 2^-60 of each gradient, bit for
    bit.  At 2^-108 fp32's last plane meets the end of bf16's range: p is of size one (times that), so 2^-133 is 2^-25 of it
    and of dy; two operands and three products give less than 2^-22."""
    x, dy, wi, wo = inputs(200, 136, 264, dtype, 3)

    def gradients(e):
        o = [torch.full_like(t, 7) for t in (x, wi, wo)]
        bd.rec_attn_ffn_bwd(x, wi, wo, (dy.double() * 2.0**e).to(dtype), *o)
        torch.cuda.synchronize()
        return [t.double() * 2.0**-e for t in o]

    full = gradients(0)
    for got, want in zip(gradients(-60), full):
        assert torch.equal(got, want)
    for got, want in zip(gradients(-108), full):
        assert off(got, want) < 2.0**-22
