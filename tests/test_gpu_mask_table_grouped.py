"""Pairs beyond the plan's mask table (test_gpu_mask_table) with shared heads, at head_dim 128 and in
fp32: the kernels build those pairs' visibility themselves, in the backward with the heads of a group in
one item too.  Bounds: bf16 output 2e-2 and 2e-3 on average, gradients 1e-2 relative Frobenius and 2e-2
of the largest value; fp32 1e-4, 1e-5 and 1e-4."""
import numpy as np
import pytest
import torch

import gpu_util as gu
import oracle
from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import workloads as W
from test_gpu_mask_table import TILE, _interleaved

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


# dtype, query heads, key/value heads, head_dim (39 tiles: dK/dV items of one head, and with 8 key/value heads of two)
@pytest.mark.parametrize("dtype,H,Hk,d", [
    ("bf16", 4, 1, 64), ("bf16", 16, 8, 64), ("bf16", 2, 1, 128), ("bf16", 16, 8, 128), ("fp32", 2, 1, 64),
    ("fp32", 2, 2, 32)])
def test_pairs_beyond_the_table(dtype, H, Hk, d):
    w = _interleaved(n_tokens=4901, heads=1)
    T, off, rng = w.total_tokens, w.offsets, np.random.default_rng(11)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    new = lambda h: dev(rng.standard_normal((T, h, d)).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    q, k, v, do = new(H), new(Hk), new(Hk), new(H)
    t, ty, mask = dev(w.t), dev(w.types), dict(w.mask)
    o, dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, q, k, v))
    lse = torch.empty(T, H, device="cuda")
    with bd.rec_attn_plan_grouped(bd.make_params(H, d, dtype=dtype, **mask), Hk, off, dev(off), t, ty) as plan:
        n_tiles = (T + TILE - 1) // TILE
        assert int((bd.rec_attn_tile_classes(plan) == bd.TILE_PARTIAL).sum()) > 8 * n_tiles + 1024
        bd.rec_attn_fwd(plan, q, k, v, o, lse)
        bd.rec_attn_bwd(plan, q, k, v, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        assert bd.rec_attn_device_status(plan) == bd.OK
    # against 64 bits on the device, head by head, with the oracle's mask and rotation
    seen = dev(oracle.mask_block(oracle.Params(H, d, **mask), w.t, w.types, 0, T, 0, T)[:T, :T]).bool()
    pair = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    angle = (t - t[0]).double()[:, None] * (1e-4 / (365.0 * 86400.0) * 6e5 ** (2 * pair / d))

    def turn(x, back=False):
        z = torch.view_as_complex(x.reshape(T, d // 2, 2).contiguous())
        return torch.view_as_real(z * torch.polar(torch.ones_like(angle), -angle if back else angle)).reshape(T, d)

    G, want = H // Hk, [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (o, dq, dk, dv)]
    for h in range(H):
        Q, K, V, dO = turn(q[:, h].double()), turn(k[:, h // G].double()), v[:, h // G].double(), do[:, h].double()
        P = torch.softmax((Q @ K.t() * d ** -0.5).masked_fill(~seen, -float("inf")), 1)
        P = torch.where(seen.any(1, keepdim=True), P, torch.zeros((), dtype=P.dtype, device="cuda"))
        O = P @ V
        dS = P * (dO @ V.t() - (dO * O).sum(1, keepdim=True)) * d ** -0.5
        want[0][:, h], want[1][:, h] = O, turn(dS @ K, True)
        want[2][:, h // G] += turn(dS.t() @ Q, True)
        want[3][:, h // G] += P.t() @ dO
    err = (o.double() - want[0]).abs()
    if dtype == "bf16":
        assert err.max() <= gu.BF16_MAX_ABS and err.mean() <= gu.BF16_MEAN_ABS
    else:
        assert err.max() <= gu.FP32_MAX_ABS
    rel_bound, top_bound = (1e-2, 2e-2) if dtype == "bf16" else (1e-5, 1e-4)
    for what, got, ref in zip(("dq", "dk", "dv"), (dq, dk, dv), want[1:]):
        diff = got.double() - ref
        rel, top = float(diff.norm() / ref.norm()), float(diff.abs().max() / ref.abs().max())
        assert rel <= rel_bound and top <= top_bound, (what, rel, top)
