"""A tensor that is not given (None) where the feed-forward, scaled and layer norm calls need one is refused like any other
wrong argument."""
import pytest
import torch

from generative_recommender_ranking_gb300 import binding as bd

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def refused(call, *args):
    with pytest.raises(bd.RecAttnError) as e:
        call(*args)
    assert e.value.code == bd.ERR_INVALID_ARG


def calls(device):
    m = lambda r, c, t=BF: torch.zeros(r, c, device=device).to(t)
    x, wi, wo = m(4, 128), m(256, 128), m(128, 128)
    qi, qo, sx, si, so = m(256, 128, F8), m(128, 128, F8), m(4, 1, torch.float32), m(2, 1, torch.float32), m(1, 1, torch.float32)
    g = m(1, 128, torch.float32)
    return [(bd.rec_attn_ffn_fwd, (x, wi, wo, m(4, 128))), (bd.rec_attn_ffn_bwd, (x, wi, wo, m(4, 128))),
            (bd.rec_attn_scaled_quantize, (x, m(4, 128, F8), sx)),
            (bd.rec_attn_scaled_matmul, (m(4, 128, F8), sx, qo, so, m(4, 128))),
            (bd.rec_attn_ffn_scaled_fwd, (x, qi, si, qo, so, m(4, 128))),
            (bd.rec_attn_layernorm_fwd, (x, g, g, m(4, 128)))]


def check(device):
    for call, args in calls(device):
        for k in range(len(args)):
            if call is bd.rec_attn_layernorm_fwd and k == 2:
                continue  # (a bias may be left out)
            refused(call, *args[:k], None, *args[k + 1:])


def test_missing_tensors():
    check("cpu")


@pytest.mark.gpu
def test_missing_tensors_on_the_device():
    import gpu_util as gu
    gu.ensure_built()
    for call, args in calls("cuda"):
        call(*args)  # (good as they are)
    check("cuda")
    torch.cuda.synchronize()
