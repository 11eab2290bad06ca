"""e4m3 matrices with a scale for each block of 128 (rec_attn_scaled_quantize, rec_attn_scaled_matmul,
rec_attn_ffn_scaled_fwd) vs the definitions in 64 bits.

The quantizer has no tolerance: scales are powers of two, so x / scale is exact and one rounding
remains.  Products: h |y| for y's rounding (h = 2^-8) and s(K) = (K / 8 + 16) 2^-22 of the sum of
absolute products for the sums (the tensor cores add at least 16 products at a time, each time losing
at most a step of 2^-23, taken four times over).  Feed-forward: as test_gpu_ffn.py up to h in fp32,
whose error eh moves its e4m3 value at most to that of h +- eh, or, where a block's largest value is
within eh of a power of two times 448, its scale, which moves values below 2^-6 of the scale by a step
of 2^-9."""
import math

import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import act_both, s

pytestmark = pytest.mark.gpu
F8, H2 = torch.float8_e4m3fn, 2.0**-8


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def blocks(n):
    return -(-n // 128)


def at_values(scale, br, rows, width):
    return scale.repeat_interleave(br, 0)[:rows].repeat_interleave(128, 1)[:, :width]


def tops(x, br):
    """The largest finite size of each block."""
    r, w = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), 0.0)
    p = a.new_zeros(-(-r // br) * br, blocks(w) * 128)
    p[:r, :w] = a
    return p.view(-1, br, blocks(w), 128).amax((1, 3))


def scales(top):
    m, e = torch.frexp(top)  # 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).int()).clamp_min(-126)
    return torch.where(top > 0, ((e.long() + 1023) << 52).view(torch.float64), 1.0)


def to_e4m3(v):
    e = (torch.frexp(v)[1] - 1).clamp_min(-6) - 3
    step = ((e.long() + 1023) << 52).view(torch.float64)
    return torch.round(v / step) * step


def quantized(x, br):
    """(e4m3 values, scales) in 64 bits."""
    sc = scales(tops(x, br))
    return to_e4m3(x / at_values(sc, br, *x.shape)), sc


def quantize(x, br):
    q = torch.full(x.shape, 1.0, device="cuda").to(F8)
    sc = torch.full((-(-x.shape[0] // br), blocks(x.shape[1])), float("nan"), device="cuda")
    bd.rec_attn_scaled_quantize(x, q, sc, block_rows=br)
    torch.cuda.synchronize()
    return q, sc


def held(q, sc, br):
    return q.float().double() * at_values(sc.double(), br, *q.shape)


def spread(rows, width, seed=0):
    """Rows of very unlike sizes: blocks of zeros, of subnormal numbers, of numbers near the type's largest."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-12, 1, (rows, width), generator=g).float())
    for r, f in ((0, 0.0), (2, 1e-42), (3, 2.0**125), (4, 2.0**-130)):
        if r < rows:
            x[r] = x[r].sign() * f
    if rows > 5:
        x[5] = 448.0 * 2.0**-3  # at the border of a scale exactly
    return x


QUANT = [(1, 16), (1, 512), (3, 144), (128, 128), (129, 128), (300, 1040), (1000, 48), (257, 4112), (5, 16384)]


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", QUANT)
def test_quantizer_is_exact(rows, width, dtype, br):
    x = spread(rows, width, seed=rows).to(dtype).cuda()
    q, sc = quantize(x, br)
    ref, rsc = quantized(x.double(), br)
    assert torch.equal(sc.double(), rsc)
    assert torch.equal(q.float().double(), ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("br", [1, 128])
def test_ties_and_values_that_are_not_finite(dtype, br):
    """Every tie of e4m3 rounds to even; NaN and infinities become NaN and leave the scale alone."""
    grid = torch.arange(0, 128).to(torch.uint8).view(F8).float()[:127]
    ties = ((grid[:-1].double() + grid[1:].double()) / 2).float()
    x = torch.zeros(4, 256)
    x[0, :126], x[1, :126], x[2, :126] = ties, -ties, ties * 2.0**-20
    x[0, 127], x[2, 127] = 448.0, 448.0 * 2.0**-20
    x[:, 128:] = torch.randn(4, 128, generator=torch.Generator().manual_seed(1))
    x[1, 130], x[2, 131], x[3, 132] = float("nan"), float("inf"), -float("inf")
    x = x.to(dtype).cuda()
    q, sc = quantize(x, br)
    ref, rsc = quantized(x.double(), br)
    assert torch.equal(sc.double(), rsc)
    bad = ~torch.isfinite(x)
    assert torch.isnan(q.float()[bad]).all() and int(torch.isnan(q.float()).sum()) == 3
    assert torch.equal(q.float()[~bad].double(), ref[~bad])


def within(got, value, tol, name):
    assert torch.isfinite(got).all(), name
    over = (got.double() - value).abs() - tol - 1e-30
    assert over.max() <= 0, (name, float(over.max()), float(value.abs().max()))


PRODUCTS = [(1, 8, 16), (1, 512, 512), (3, 136, 144), (7, 4096, 256), (128, 256, 128), (129, 264, 1040), (300, 72, 2064),
            (1000, 1000, 400), (2049, 128, 640), (16, 2048, 1024), (33, 520, 4096), (8, 24, 272), (9, 136, 400),
            (17, 1160, 144), (24, 520, 1040), (25, 264, 656), (31, 2056, 528), (32, 1000, 2064), (64, 264, 400),
            (65, 136, 1040), (100, 520, 4112), (300, 264, 8208)]


@pytest.mark.parametrize("any_scale", [False, True])
@pytest.mark.parametrize("rows,cols,depth", PRODUCTS)
def test_matmul(rows, cols, depth, any_scale):
    g = torch.Generator().manual_seed(rows)
    a, asc = quantize(torch.randn(rows, depth, generator=g).cuda() * 3, 1)
    b, bsc = quantize(torch.randn(cols, depth, generator=g).cuda(), 128)
    if any_scale:  # a checkpoint's own: any fp32
        asc *= torch.exp(torch.randn(asc.shape, generator=g)).cuda()
        bsc *= torch.exp(torch.randn(bsc.shape, generator=g)).cuda()
    y = torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    bd.rec_attn_scaled_matmul(a, asc, b, bsc, y)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    A, B = held(a, asc, 1), held(b, bsc, 128)
    ref = A @ B.T
    within(y, ref, H2 * ref.abs() + s(depth) * (A.abs() @ B.abs().T), "y")


FFN = [(1, 16, 128), (1, 512, 1024), (5, 144, 256), (129, 512, 128), (300, 1040, 384), (1031, 512, 1024), (20, 4096, 512), (8, 272, 128), (9, 400, 640), (25, 144, 256),
       (32, 1040, 384), (33, 272, 256), (64, 144, 640), (65, 400, 128), (100, 528, 2048), (280, 272, 4096)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,width,hidden", FFN)
def test_ffn(rows, width, hidden, act):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, width, generator=g).bfloat16().cuda()
    wi, wis = quantize((torch.randn(2 * hidden, width, generator=g) / math.sqrt(width)).cuda(), 128)
    wo, wos = quantize((torch.randn(width, hidden, generator=g) / math.sqrt(hidden)).cuda(), 128)
    y = torch.full_like(x, float("nan"))
    bd.rec_attn_ffn_scaled_fwd(x, wi, wis, wo, wos, y, activation=act)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    xq, xs = quantized(x.double(), 1)
    X, Wi, Wo = xq * at_values(xs, 1, *x.shape), held(wi, wis, 128), held(wo, wos, 128)
    gu_, e = X @ Wi.T, s(width) * (X.abs() @ Wi.abs().T)
    gt, up, eg, eu = gu_[:, :hidden], gu_[:, hidden:], e[:, :hidden], e[:, hidden:]
    a, _ = act_both(gt, act)
    h = a * up
    eh = 1.13 * eg * up.abs() + a.abs() * eu + (gt.abs() + 4) * (1 + gt.abs()) * 2.0**-22 * up.abs()
    hq, hs = quantized(h, 1)
    sv = at_values(hs, 1, *h.shape)
    near = scales(tops(h.abs() + eh, 1)) != scales(tops((h.abs() - eh).clamp_min(0), 1))
    move = torch.maximum(to_e4m3((h + eh) / sv) - hq, hq - to_e4m3((h - eh) / sv)) * sv
    move += torch.where(at_values(near.double(), 1, *h.shape) > 0, 2 * sv * 2.0**-9, 0.0)
    ref = (hq * sv) @ Wo.T
    within(y, ref, H2 * ref.abs() + move @ Wo.abs().T + s(hidden) * ((hq * sv).abs() @ Wo.abs().T), "y")
