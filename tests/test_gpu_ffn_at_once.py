"""Feed-forward and scaled calls from several host threads, and several captured graphs of them, at the same time: each gives
the bits that it gives alone (workspaces, attributes asked for once and the status word are all that calls share)."""
import threading

import pytest
import torch

import gpu_util as gu
from generative_recommender_ranking_gb300 import binding as bd
from test_gpu_ffn import inputs
from test_gpu_ffn_calls import serve, serving, train

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def runs():
    gu.ensure_built()
    made = [(train, inputs(5, 136, 264, BF, 1)), (train, inputs(300, 136, 264, BF, 2)), (train, inputs(150, 132, 68, F32, 3)),
            (train, inputs(900, 136, 264, F32, 4)), (serve, serving(5, rows=40)), (serve, serving(6, rows=700))]
    calls = [lambda f=f, t=t: f(t) for f, t in made]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    return calls, want


def test_threads(runs):
    calls, want = runs
    wrong = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = calls[k]()
                torch.cuda.current_stream().synchronize()
                wrong.extend(k for a, b in zip(got, want[k]) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert bd.rec_attn_dense_device_status() == bd.OK


def test_graphs(runs):
    calls, want = runs
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append((g, torch.cuda.Stream()))
    for _ in range(10):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert bd.rec_attn_dense_device_status() == bd.OK
