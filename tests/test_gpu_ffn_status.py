"""The status word of the feed-forward and scaled calls: an error is reported once, and later calls by themselves."""
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import inputs


@pytest.mark.gpu
def test_an_error_is_reported_once():
    gu.ensure_built()
    assert bd.rec_attn_dense_device_status() == bd.OK
    bd.rec_attn_check_dense_wait_timeout(20)
    # a good call on another stream neither hides nor clears it
    x, _, wi, wo = inputs(70, 64, 128, torch.bfloat16)
    y = torch.empty_like(x)
    with torch.cuda.stream(torch.cuda.Stream()):
        bd.rec_attn_ffn_fwd(x, wi, wo, y)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.ERR_TIMEOUT
    assert bd.rec_attn_dense_device_status() == bd.OK
    bd.rec_attn_ffn_fwd(x, wi, wo, y)
    assert bd.rec_attn_dense_device_status() == bd.OK
    bd.rec_attn_check_dense_wait_timeout(20)  # and the next is reported again
    assert bd.rec_attn_dense_device_status() == bd.ERR_TIMEOUT
    assert bd.rec_attn_dense_device_status() == bd.OK


def test_self_check_refusals():
    from generative_recommender_ranking_gb300 import build as bld
    bld.build()
    L = bd.lib()
    for ms in (0, 10001, 20000):
        assert L.rec_attn_check_dense_wait_timeout(ms, None) == bd.ERR_INVALID_ARG
