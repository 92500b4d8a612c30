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
