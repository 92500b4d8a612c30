"""Calls from a thread that has made no CUDA call of its own yet, as autograd's are."""
import threading

import numpy as np
import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import done, f64, mm_ints, mm_want, wg_ints, wg_want

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    failed = []

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001 (raised again below)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("M", [5, 70, 900])
@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
def test_products(op, M):
    args = mm_ints(M, 300, 520, False, seed=51) if op == "matmul" else wg_ints(300, M, 520, "bf16", seed=51)
    fn, want = (gct.matmul_fp8, mm_want) if op == "matmul" else (gct.weight_grad_fp8, wg_want)
    out = torch.full((M, 520), float("nan"), device="cuda")
    ws = fn(*args, out)
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    in_a_new_thread(lambda: fn(*args, out, workspace=ws))
    done(ws)
    assert np.array_equal(f64(out), want(*args)[0])


def test_quantize():
    x = torch.ones(30, 300, device="cuda")
    codes, scales = gct.empty_fp8(30, 300)
    in_a_new_thread(lambda: gct.quantize_fp8(x, codes, scales))
    assert torch.equal(codes.float() * scales.repeat_interleave(128, 1)[:, :300], x)


def test_a_backward_pass_that_starts_with_the_weight_gradient():
    x = torch.ones(64, 256, dtype=torch.bfloat16, device="cuda")  # asks for no gradient
    weight = torch.full((256, 128), 0.5, device="cuda", requires_grad=True)
    W, W_scale = gct.empty_fp8(256, 128, "tiles")
    gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
    y = gct.fp8_linear(x, W, W_scale, weight)
    in_a_new_thread(lambda: y.backward(torch.ones_like(y)))
    assert (weight.grad == 64).all()
