"""What the fp32 feed-forward block has to keep of its values, which go through the tensor cores as three bf16 planes."""
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd

F32 = torch.float32


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
