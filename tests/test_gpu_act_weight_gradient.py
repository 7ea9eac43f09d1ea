"""te_act_bwd_bf16's fp32 weight gradient beside dX: calls one behind the other, each adding to what the one before it has
left, give the bits that they give one at a time; eagerly, in a graph, and on two streams at once."""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, K, F, N, seed):
        g = torch.Generator(device=G.DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, device=G.DEV, generator=g)   # noqa: E731
        self.x, self.w, self.w2, self.dy, self.z = (r(*s).bfloat16() for s in ((T, K), (F, K), (N, F), (T, N), (T, F)))
        self.start = r(F, K)
        self.dz, self.dx, self.dw, self.db = (torch.empty_like(self.z), torch.empty_like(self.x), torch.empty_like(self.start),
                                              torch.empty(F, device=G.DEV))
        self.ws = torch.empty(te.te_act_dbias_workspace_bytes(T, F) // 4, device=G.DEV)

    def call(self, what, stream=None):
        te.te_act_bwd_bf16(self.x, self.w, self.w2, self.dy, self.z, te.ACT_SILU, self.dz, self.db if "db" in what else None,
                           self.ws if "db" in what else None, self.dx if "dx" in what else None, self.dw, 1, stream)

    def outputs(self, what):
        return [self.dw] + [t for t, n in ((self.db, "db"), (self.dx, "dx")) if n in what]


SIZES = [(1001, 768, 2048, 768), (4100, 64, 272, 96), (300, 2304, 2560, 160), (2100, 1024, 1040, 48)]


@pytest.mark.parametrize("what", [("db", "dx"), ("dx",), ("db",), ()])
@pytest.mark.parametrize("size", SIZES)
def test_each_call_adds_to_the_one_before(size, what):
    c, n = Case(*size, 1), 6
    c.dw.copy_(c.start)
    for _ in range(n):
        c.call(what)
        torch.cuda.synchronize()
    want = [t.clone() for t in c.outputs(what)]
    assert bool((want[0] != c.start).any())

    def again():
        c.dw.copy_(c.start)
        for _ in range(n):
            c.call(what)
        return [t.clone() for t in c.outputs(what)]

    for _ in range(3):
        got = again()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = again()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    G.check_no_device_error()


def test_two_streams_at_once():
    a, b, what = Case(*SIZES[0], 2), Case(*SIZES[2], 3), ("db", "dx")
    want = []
    for c in (a, b):
        c.dw.copy_(c.start)
        for _ in range(4):
            c.call(what)
        torch.cuda.synchronize()
        want.append([t.clone() for t in c.outputs(what)])
    side = torch.cuda.Stream()
    for _ in range(5):
        for c in (a, b):
            c.dw.copy_(c.start)
        torch.cuda.synchronize()
        for _ in range(4):
            a.call(what)
            b.call(what, side)
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            assert all(torch.equal(p, q) for p, q in zip(c.outputs(what), w))
    G.check_no_device_error()
