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


def test_threads_that_share_a_stream_and_its_workspace():
    """Layers whose weights are copied into the workspace before each product
    (rows of 255 bytes), from several threads on one stream, without one of their own."""
    def layer(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        K, N = 256 + 128 * (seed % 3), 255
        weight = torch.randn(K, N, generator=g, device="cuda").requires_grad_()
        W, W_scale = torch.empty(K, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.empty(K // 128, 2, device="cuda")
        gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
        x = torch.randn(64 + seed, K, generator=g, device="cuda").bfloat16().requires_grad_()
        return x, W, W_scale, weight

    def step(x, W, W_scale, weight):
        y = gct.fp8_linear(x, W, W_scale, weight)
        return (y, *torch.autograd.grad(y, (x, weight), torch.ones_like(y)))

    layers = [layer(s) for s in range(6)]
    wants = [step(*a) for a in layers]
    wrong = []

    def run(a, want):
        try:
            for _ in range(60):
                if not all(torch.equal(p, q) for p, q in zip(step(*a), want)):
                    wrong.append(a[0].shape)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=run, args=p) for p in zip(layers, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert gct.query_status(gct.fp8_workspace())[0] == 0
