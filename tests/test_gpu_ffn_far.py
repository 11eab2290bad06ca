"""Far rows of the feed-forward block: offsets past 2^31 elements of its workspaces and operands.

Only a few hundred rows have values, at the start, about element 2^31 of p and of h, at the seams of the rows' parts and at
the end; the others are zero, and so are their h and p (act(0) 0).  So the weights' gradients are the chosen rows' alone
and are compared with tolerances of that many rows: a lost, repeated or misplaced row shows."""
import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import reference, within

pytestmark = pytest.mark.gpu
H, WIDTH = 1024, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


def chosen(rows):
    spans = [(0, 40), (rows // 3 - 20, rows // 3 + 20), (rows - 40, rows)]
    for at in (2**31 // (2 * H), 2**31 // H, 2**32 // (2 * H)):
        if at + 20 <= rows:
            spans.append((at - 20, at + 20))
    return torch.cat([torch.arange(a, b) for a, b in spans]).unique().cuda()


@pytest.mark.parametrize("dtype,rows", [(torch.bfloat16, 1_100_003), (torch.bfloat16, 2_150_001), (torch.float32, 1_100_003)])
def test_gradients_of_far_rows(dtype, rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    at = chosen(rows)
    x, dy = torch.zeros(rows, WIDTH, dtype=dtype, device="cuda"), torch.zeros(rows, WIDTH, dtype=dtype, device="cuda")
    x[at], dy[at] = rnd(len(at), WIDTH).to(dtype), rnd(len(at), WIDTH).to(dtype)
    wi, wo = (rnd(2 * H, WIDTH) / 8).to(dtype), (rnd(WIDTH, H) / 32).to(dtype)
    y, dx = torch.full_like(x, 7), torch.full_like(x, 7)
    dwi, dwo = torch.full_like(wi, 7), torch.full_like(wo, 7)
    bd.rec_attn_ffn_fwd(x, wi, wo, y)
    bd.rec_attn_ffn_bwd(x, wi, wo, dy, dx, dwi, dwo)
    torch.cuda.synchronize()
    assert bd.rec_attn_dense_device_status() == bd.OK
    ref = reference(x[at], dy[at], wi, wo, "silu", torch.finfo(dtype).eps / 2)
    for name, got in (("y", y[at]), ("dx", dx[at]), ("dw_in", dwi), ("dw_out", dwo)):
        within(got, ref[name], name)
        value = ref[name][0]  # and in norm: bf16 2^-8 for each of the roundings of p or h and of the result
        assert (got.double() - value).norm() <= (2 * 2.0**-8 if dtype == torch.bfloat16 else 1e-6) * value.norm(), name
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not y[rest].any() and not dx[rest].any()
