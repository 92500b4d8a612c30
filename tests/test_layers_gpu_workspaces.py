"""Workspaces whose memory comes from a graph capture: their zero-fill runs when the graph does."""
import pytest
import torch

import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

CUT = dict(tile_m=256, tile_n=256)  # its 16 tiles are cut along the contraction: sums and flags in the workspace


class Products:
    """Integer products whose results are exact, and a graph pool whose free memory is full of ones."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)
        ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").bfloat16()
        self.A, self.B = ints(512, 8192), ints(8192, 2000)
        self.want = (self.A.double() @ self.B.double()).float()
        warm = gct.matmul_act(self.A, self.B, torch.empty_like(self.want), config=CUT)  # before any capture
        self.nbytes = warm.nbytes
        assert self.nbytes > 1 << 20
        torch.cuda.synchronize()
        self.filled = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.filled):
            t = torch.full((256 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        self.filled.replay()
        torch.cuda.synchronize()
        del t

    def call(self, ws, times=1, out=None, **kw):
        out = torch.full_like(self.want, 7) if out is None else out
        return gct.matmul_act(self.A * times, self.B, out, config=dict(CUT, **kw), workspace=ws), out

    def check(self, ws, times=1):
        ws, out = self.call(ws, times)
        assert torch.equal(out, self.want * times)
        return ws

    def capture(self, ws, out, **kw):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=self.filled.pool()):
            ws = self.call(ws, out=out, **kw)[0]
        return graph, ws


@pytest.mark.parametrize("given", [True, False], ids=["grown", "made"])
def test_calls_beside_a_graph_that_has_not_run(given):
    """A workspace that a capture has grown, or made and returned, serves eager calls before the graph's first replay, between
    replays, and the graph keeps its own."""
    p = Products()
    out = torch.zeros_like(p.want)
    graph, ws = p.capture(gct.Workspace(256) if given else None, out)
    assert ws.nbytes >= p.nbytes
    assert gct.query_status(ws)[0] == 0
    for times in (1, 2, 4, 1):
        assert p.check(ws, times) is ws
    for _ in range(3):
        out.zero_()
        graph.replay()
        p.check(ws, 2)
        assert torch.equal(out, p.want)
    assert gct.query_status(ws)[0] == 0


def test_two_graphs_and_a_workspace_that_one_of_them_grew():
    """The second, replayed first, does not rest on what the first one would have filled."""
    p = Products()
    outs = [torch.zeros_like(p.want) for _ in range(2)]
    ws = gct.Workspace(256)
    first, _ = p.capture(ws, outs[0])
    second, _ = p.capture(ws, outs[1])
    for graph, out in ((second, outs[1]), (second, outs[1]), (first, outs[0]), (second, outs[1])):
        out.zero_()
        graph.replay()
        assert torch.equal(out, p.want)
    p.check(ws, 2)
    assert gct.query_status(ws)[0] == 0


def test_errors_of_a_graph_with_memory_of_its_own_are_found():
    """By the caller's workspace, once the graph has run, also after eager calls have moved it to other memory."""
    p = Products()
    ws, out = gct.Workspace(256), torch.zeros_like(p.want)
    graph, _ = p.capture(ws, out, debug_skip_flag=1, wait_ns=20_000_000)
    p.check(ws)
    assert gct.query_status(ws) == (0, 0, 0, 0)
    graph.replay()
    assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
    assert gct.query_status(ws)[0] == 0
    p.check(ws, 2)


def test_layers_trained_in_a_graph_without_a_call_before():
    """Forward and backward in a capture whose workspace has to grow, then eager steps, then replays."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((300, 264), (264, 520), (300, 520)))
    x.requires_grad_(), w.requires_grad_()

    def step(ws):
        y = gct.linear_act(x, w, act="gelu", workspace=ws)
        return [y.detach(), *torch.autograd.grad(y, [x, w], dy)]

    want = step(gct.Workspace(256))
    torch.cuda.synchronize()
    ws, graph = gct.Workspace(256), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ws)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(ws), want))
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gct.query_status(ws)[0] == 0
