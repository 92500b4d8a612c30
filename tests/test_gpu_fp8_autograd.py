"""fp8_linear as autograd sees it."""
import numpy as np
import pytest
import torch

import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu


def layer(tokens, K, N, seed=71, dtype=torch.bfloat16, bias=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    weight = (torch.randn(K, N, generator=g, device="cuda") / max(K, 1) ** 0.5).requires_grad_()
    W, W_scale = gct.empty_fp8(K, N, "tiles")
    gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
    x = torch.randn(tokens, K, generator=g, device="cuda").to(dtype).requires_grad_()
    b = torch.randn(N, generator=g, device="cuda").to(bias).requires_grad_()
    return x, W, W_scale, weight, b


def test_second_derivatives_are_refused():
    x, W, W_scale, weight, bias = layer(40, 256, 128)
    y = gct.fp8_linear(x, W, W_scale, weight, bias)
    loss = (y.float() ** 2).sum()
    grads = torch.autograd.grad(loss, (x, weight, bias), create_graph=True)
    for g in grads:  # a penalty on a gradient beside the loss itself
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (loss + g.float().sum()).backward(retain_graph=True)
