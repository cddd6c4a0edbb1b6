"""Token quantisation and the scaled and gated calls in captured graphs: the first calls of a process,
work that forks to a second stream and joins again, two graphs on one workspace, and inputs that
change between replays."""
import os
import subprocess
import sys

import pytest
import torch

import gemv_w4a16_w8a8_b200 as qg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# few tokens, dX by the few-token kernel or by tiles in parts, whole tiles
SHAPES = [(1, 272, 528), (77, 1371, 528), (300, 640, 528), (2000, 1376, 528)]


class Calls:
    """One pass of every call on buffers of its own; fill() gives the inputs of a seed."""

    def __init__(self, M, F, K, dtype, workspace=None):
        def new(*shape, dt=dtype):
            return torch.zeros(shape, dtype=dt, device=DEV)

        self.shape, self.dtype = (M, F, K), dtype
        self.X, self.Wg, self.Wu = new(M, K), new(F, K), new(F, K)
        self.G, self.U, self.dH = new(M, F), new(M, F), new(M, F)
        self.A, self.W = new(M, K, dt=torch.int8), new(F, K, dt=torch.int8)
        self.sa, self.sw, self.b = new(M, dt=torch.float32), new(F, dt=torch.float32), new(F)
        need = qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K)
        self.ws = new(need, dt=torch.uint8) if workspace is None else workspace
        self.out = dict(Q=new(M, K, dt=torch.int8), s=new(M, dt=torch.float32), C=new(M, F), H8=new(M, F),
                        H=new(M, F), dX=new(M, K), dWg=new(F, K), dWu=new(F, K))

    def fill(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        for t in (self.X, self.Wg, self.Wu, self.G, self.U, self.dH, self.b):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV) / 4)
        for t in (self.A, self.W):
            t.copy_(torch.randint(-128, 128, t.shape, generator=g, device=DEV, dtype=torch.int8))
        for t in (self.sa, self.sw):
            t.copy_(torch.rand(t.shape, generator=g, device=DEV) / 256)
        return self

    def eight(self):
        o = self.out
        qg.quant_int8_tokens(self.X, Q=o["Q"], scales=o["s"])
        qg.qgemm_w8a8_scaled(self.A, self.W, self.sa, self.sw, bias=self.b, C=o["C"])
        qg.qgemm_w8a8_gated(self.A, self.W, self.W, self.sa, self.sw, self.sw, H=o["H8"])

    def sixteen(self):
        o = self.out
        qg.qgemm_dense_gated(self.X, self.Wg, self.Wu, H=o["H"])
        qg.qgemm_dense_gated_backward(self.dH, self.X, self.Wg, self.Wu, self.G, self.U, dX=o["dX"],
                                      dWg=o["dWg"], dWu=o["dWu"], workspace=self.ws)

    def run(self):
        self.eight()
        self.sixteen()

    def eager(self, seed):
        """What the calls give for the inputs of `seed`, each waited for."""
        self.fill(seed)
        torch.cuda.synchronize()
        self.run()
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in self.out.items()}

    def check(self, want):
        torch.cuda.synchronize()
        for k, v in self.out.items():
            assert torch.equal(v, want[k]), k


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from test_gpu_ffn_capture import SHAPES, Calls, qg
calls = [Calls(*s, dt).fill(7) for s in SHAPES for dt in (torch.float16, torch.bfloat16)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for c in calls:
        c.run()
graph.replay()
torch.cuda.synchronize()
got = [{{k: v.clone() for k, v in c.out.items()}} for c in calls]
for c, g in zip(calls, got):
    c.eager(7)
    c.check(g)
qg.qgemm_sync_check()
"""


def test_the_first_calls_of_a_process():
    """Kernels load at their first use, inside the capture here."""
    script = FIRST.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,F,K", SHAPES)
def test_fork_and_join(M, F, K, dtype):
    """8-bit calls on a second stream beside the 16-bit ones; what follows the join reads both."""
    c = Calls(M, F, K, dtype)
    tail = dict(Q=torch.zeros(M, K, dtype=torch.int8, device=DEV), s=torch.zeros(M, device=DEV),
                C=torch.zeros(M, F, dtype=dtype, device=DEV))

    def after():
        qg.quant_int8_tokens(c.out["dX"], Q=tail["Q"], scales=tail["s"])
        qg.qgemm_w8a8_scaled(c.out["Q"], c.W, c.out["s"], c.sw, C=tail["C"])

    want = {}
    for seed in (1, 2, 3):
        first = c.eager(seed)
        after()
        torch.cuda.synchronize()
        want[seed] = first, {k: v.clone() for k, v in tail.items()}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.eight()
        c.sixteen()
        torch.cuda.current_stream().wait_stream(side)
        after()
    for seed in (2, 3, 1):
        c.fill(seed)
        graph.replay()
        c.check(want[seed][0])
        assert all(torch.equal(tail[k], v) for k, v in want[seed][1].items())


def test_two_graphs_share_a_workspace():
    """Replayed one after the other, with no synchronisation between them."""
    size = max(qg.qgemm_dense_gated_backward_workspace_bytes(*s) for s in ((77, 1371, 528), (300, 640, 528)))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    a, b = (Calls(*s, torch.bfloat16, ws) for s in ((77, 1371, 528), (300, 640, 528)))
    want = [(a.eager(seed), b.eager(seed + 10)) for seed in range(3)]
    graphs = []
    for c in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.sixteen()
    for seed, (wa, wb) in enumerate(want):
        a.fill(seed)
        b.fill(seed + 10)
        for _ in range(5):
            graphs[0].replay()
            graphs[1].replay()
        torch.cuda.synchronize()
        for c, w in ((a, wa), (b, wb)):
            assert all(torch.equal(c.out[k], w[k]) for k in ("H", "dX", "dWg", "dWu"))
