"""Workspaces that the ops make themselves: whose memory they are, and what the host waits for."""
import time

import numpy as np
import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import done, f64, mm_ints, mm_want, wg_ints

pytestmark = pytest.mark.gpu


def product(op, stream=None):
    if op == "matmul":
        args, out = mm_ints(70, 300, 257, False, seed=61), torch.empty(70, 257, device="cuda")
        return lambda: gct.matmul_fp8(*args, out, stream=stream)
    if op == "weight_grad":
        args, out = wg_ints(70, 300, 257, "bf16", seed=61), torch.empty(300, 257, device="cuda")
        return lambda: gct.weight_grad_fp8(*args, out, stream=stream)
    heap = gct.SymmetricHeap(2, 1 << 20)
    A, B, C = (heap.alloc((256, 256), torch.bfloat16) for _ in range(3))
    heap.buf.zero_()
    return lambda: gct.matmul_all_reduce(heap, A, B, C, stream=stream)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["matmul", "weight_grad", "all_reduce"])
def test_a_dropped_workspace_goes_back_to_its_stream(op, raw):
    """Memory of a workspace that was made for another stream is not handed to
    the current one while that stream may still use it."""
    side = torch.cuda.Stream()
    call = product(op, side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    ws = call()
    size, at = ws.buf.numel(), ws.ptr
    del ws
    held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert at not in [t.data_ptr() for t in held]
    side.synchronize()
    with torch.cuda.stream(torch.cuda.ExternalStream(side.cuda_stream) if raw else side):
        ws = call()
        assert ws.ptr == at  # its own stream has it back
    done_on(ws, side)


def done_on(ws, stream):
    assert gct.query_status(ws, stream)[0] == 0


@pytest.mark.parametrize("op", ["matmul", "weight_grad", "all_reduce"])
def test_making_a_workspace_waits_for_nothing(op):
    call = product(op)
    done(call())
    torch.cuda._sleep(1 << 30)  # half a second
    t = time.perf_counter()
    ws = call()
    t = time.perf_counter() - t
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    done(ws)
    assert busy and t < 0.2


def test_a_call_without_a_workspace_can_be_captured():
    args = mm_ints(300, 700, 500, False, seed=62)
    want = mm_want(*args)[0]
    out = torch.zeros(300, 500, device="cuda")
    gct.matmul_fp8(*args, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gct.matmul_fp8(*args, out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert np.array_equal(f64(out), want)


def layer(tokens, K, N, seed=63):
    g = torch.Generator(device="cuda").manual_seed(seed)
    weight = (torch.randn(K, N, generator=g, device="cuda") / K ** 0.5).requires_grad_()
    W, W_scale = gct.empty_fp8(K, N, "tiles")
    gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
    x = torch.randn(tokens, K, generator=g, device="cuda").bfloat16().requires_grad_()
    return x, W, W_scale, weight


def step(x, W, W_scale, weight, workspace=None, dy=None):
    x.grad = weight.grad = None
    y = gct.fp8_linear(x, W, W_scale, weight, workspace=workspace)
    y.backward(torch.ones_like(y) if dy is None else dy)
    return y.detach(), x.grad, weight.grad


def unaligned(tokens=256, K=4096, N=4095):
    """A layer whose weights are copied into the workspace for every product (rows of 4095 bytes)."""
    x, W, W_scale, weight = layer(tokens, K, N)
    packed = torch.empty(K, N, dtype=torch.uint8, device="cuda")
    packed.copy_(W.view(torch.uint8))
    return x, packed.view(W.dtype), W_scale, weight


@pytest.mark.parametrize("own", [False, True])
def test_linear_layer_waits_for_nothing(own):
    args = layer(300, 512, 384)
    ws = gct.Workspace(256) if own else None
    step(*args, workspace=ws)
    torch.cuda.synchronize()
    torch.cuda._sleep(1 << 30)
    t = time.perf_counter()
    step(*args, workspace=ws)
    t = time.perf_counter() - t
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy and t < 0.2


def test_linear_layer_keeps_no_workspace_for_its_backward_pass():
    """Between forward and backward a layer holds codes, scales and its output,
    not the 16 MB that its products copy weights into."""
    x, W, W_scale, weight = unaligned()
    gct.fp8_linear(x, W, W_scale, weight).sum().backward()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [gct.fp8_linear(x, W, W_scale, weight) for _ in range(4)]
    each = (torch.cuda.memory_allocated() - before) / 4
    assert each <= 256 * 4096 + 256 * 32 * 4 + 256 * 4095 * 2 + 4096
    del kept


def test_linear_layer_grows_the_workspace_it_is_given():
    """A small workspace grows in place, once: tail tiles hand their sums over in it."""
    args = layer(16384, 4096, 4096)
    ws = gct.Workspace(256)
    first = step(*args, workspace=ws)
    size, at = ws.nbytes, ws.ptr
    assert size > 16 * 16384
    second = step(*args, workspace=ws)
    assert (ws.nbytes, ws.ptr) == (size, at)
    done(ws)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_products_grow_the_workspace_they_are_given():
    x, W, W_scale, _ = unaligned(100)
    codes, scales = gct.empty_fp8(100, 4096)
    gct.quantize_fp8(x.detach(), codes, scales)
    out = torch.empty(100, 4095, device="cuda")
    ws = gct.Workspace(256)
    assert gct.matmul_fp8(codes, scales, W, W_scale, out, workspace=ws) is ws
    want = mm_want(codes, scales, W, W_scale)
    done(ws)
    assert (np.abs(f64(out) - want[0]) <= 170 * 2.0 ** -23 * want[1]).all()


def test_a_workspace_takes_its_error_along_when_it_grows():
    args, out = mm_ints(300, 700, 500, False, seed=64), torch.empty(300, 500, device="cuda")
    ws = gct.Workspace(256)
    gct.matmul_fp8(*args, out, workspace=ws, config=dict(debug_skip_flag=2, wait_ns=20_000_000, tile_m=256))
    step(*unaligned(), workspace=ws)
    assert ws.nbytes > 1 << 20
    assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
    assert gct.query_status(ws)[0] == 0


def test_errors_of_layers_without_a_workspace_are_found(monkeypatch):
    import ctypes

    from gemm_collective_tiles_gb300 import fp8
    args = layer(300, 512, 640)
    assert gct.query_status(gct.fp8_workspace())[0] == 0
    config = gct.make_config(debug_skip_flag=2, wait_ns=20_000_000, tile_m=256)
    with monkeypatch.context() as m:
        m.setattr(fp8, "_cfgp", lambda c: ctypes.byref(config))
        y = gct.fp8_linear(*args)
    assert gct.query_status(gct.fp8_workspace())[0] == gct._native.IRIS_ETIMEOUT
    with monkeypatch.context() as m:
        m.setattr(fp8, "_cfgp", lambda c: ctypes.byref(config))
        y.backward(torch.ones_like(y))
    assert gct.query_status(gct.fp8_workspace())[0] == gct._native.IRIS_ETIMEOUT
    step(*args)
    assert gct.query_status(gct.fp8_workspace())[0] == 0


def test_streams_have_workspaces_of_their_own():
    side = torch.cuda.Stream()
    here = gct.fp8_workspace()
    assert gct.fp8_workspace() is here and gct.fp8_workspace("cuda:0") is here
    with torch.cuda.stream(side):
        assert gct.fp8_workspace() is not here and gct.fp8_workspace() is gct.fp8_workspace()


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("make", [lambda: layer(300, 512, 384), lambda: unaligned(64, 256, 255)])
def test_linear_layer_in_a_graph(make, own):
    """Forward and backward captured once, replayed on new values, beside
    eager calls and after the workspace has grown for another layer."""
    x, W, W_scale, weight = make()
    ws = gct.Workspace(256) if own else None
    dy = torch.ones(x.shape[0], W.shape[1], dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, W, W_scale, weight, ws, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    x.grad = weight.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, W, W_scale, weight, ws, dy)
    for i in range(3):
        with torch.no_grad():
            x.mul_(-1.5)
            dy.mul_(0.5)
        graph.replay()
        got_now = [t.clone() for t in got]
        want = step(x.detach().clone().requires_grad_(), W, W_scale, weight.detach().clone().requires_grad_(), ws, dy)
        for a, b in zip(got_now, want):
            assert torch.equal(a, b)
        if i == 0:
            step(*unaligned(200, 512, 1023), workspace=ws)
    done(ws if own else gct.fp8_workspace())


def test_errors_of_a_graph_captured_before_the_workspace_grew_are_found():
    args, out = mm_ints(300, 700, 500, False, seed=65), torch.empty(300, 500, device="cuda")
    ws = gct.Workspace(256)
    config = dict(debug_skip_flag=2, wait_ns=20_000_000, tile_m=256)
    gct.matmul_fp8(*args, out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gct.matmul_fp8(*args, out, workspace=ws, config=config)
    step(*unaligned(), workspace=ws)
    assert ws.nbytes > 1 << 20
    done(ws)
    graph.replay()
    assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
    done(ws)


def test_a_workspace_elsewhere_is_refused():
    """Before anything is launched: the device would write to the host's address."""
    args, out = mm_ints(30, 256, 64, False, seed=66), torch.full((30, 64), 7.0, device="cuda")
    ws = gct.Workspace(1 << 20, "cpu")
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gct.matmul_fp8(*args, out, workspace=ws)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gct.weight_grad_fp8(*wg_ints(30, 30, 64, "bf16"), out, workspace=ws)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        gct.fp8_linear(*layer(30, 256, 64), workspace=ws)
    assert (out == 7).all() and not ws.buf.any()
