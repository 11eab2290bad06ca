"""Layer norm of rows of more than 256 threads, many rows a block: the slots of the rows on their way are
used again, the two halves of the reductions between warps alternate, and a block's type changes and
comes back.  Tolerances as in test_gpu_layernorm."""
import pytest
import torch

import gpu_util as gu
from test_gpu_layernorm import E32, inputs, reference, run, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gu.ensure_built()


# widths of 288, 512, 544 and 1024 threads (the last chunks missing in some), each with more rows
# than the device holds blocks at a time
@pytest.mark.parametrize("types", ["one", "runs", "random"])
@pytest.mark.parametrize("rows,width,dtype", [
    (1500, 4104, torch.bfloat16), (1000, 8192, torch.bfloat16), (901, 8200, torch.bfloat16), (700, 16384, torch.bfloat16),
    (1500, 2056, torch.float32), (1000, 4096, torch.float32), (901, 8192, torch.float32), (700, 8196, torch.float32),
    (500, 16384, torch.float32)])
def test_many_rows_a_block(rows, width, dtype, types):
    x, dy, w, b, ty = inputs(rows, width, dtype, types != "one", seed=6, runs=types == "runs")
    if types == "random":
        ty[11::101] = 5  # rows of no type among them
    y, dx, dw, db = run(x, dy, w, b, ty, 1e-5)
    ref = reference(x, dy, w, b, ty, 1e-5)
    half = torch.finfo(dtype).eps / 2
    for got, n, h in ((y, "y", half), (dx, "dx", half), (dw, "dw", E32), (db, "db", E32)):
        within(got, ref[n], h)
    again = run(x, dy, w, b, ty, 1e-5)
    assert all(torch.equal(a, c) for a, c in zip((y, dx, dw, db), again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(dtype):
    from generative_recommender_ranking_gb300 import binding as bd
    x, dy, w, b, ty = inputs(700, 16384, dtype, True, seed=8)
    y, dx, dw, db = run(x, dy, w, b, ty, 1e-5)
    z, g = x.clone(), dy.clone()
    bd.rec_attn_layernorm_fwd(z, w, b, z, types=ty, eps=1e-5)
    bd.rec_attn_layernorm_bwd(x, w, g, g, types=ty, eps=1e-5)
    assert torch.equal(z, y) and torch.equal(g, dx)
