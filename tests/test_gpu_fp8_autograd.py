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


@pytest.mark.parametrize("what", ["codes and scales", "the scales alone"])
def test_weights_quantised_again_before_the_backward_pass_are_an_error(what):
    x, W, W_scale, weight, bias = layer(40, 256, 128)
    y = gct.fp8_linear(x, W, W_scale, weight, bias)
    other = gct.empty_fp8(256, 128, "tiles")[0]
    gct.quantize_fp8(weight.detach() * 2, other if "alone" in what else W, W_scale, block="tiles")
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(torch.ones_like(y))
    gct.fp8_linear(x, W, W_scale, weight, bias).sum().backward()  # the next forward pass has the new ones


def test_what_the_ops_write_counts_as_written():
    x, W, W_scale, _, _ = layer(40, 256, 128)
    codes, scales = gct.empty_fp8(40, 256)
    out, dw = torch.empty(40, 128, device="cuda"), torch.empty(256, 128, device="cuda")
    before = [t._version for t in (codes, scales, out, dw)]
    gct.quantize_fp8(x.detach(), codes, scales)
    gct.matmul_fp8(codes, scales, W, W_scale, out)
    gct.weight_grad_fp8(codes, scales, torch.ones(40, 128, dtype=torch.bfloat16, device="cuda"), dw)
    assert all(t._version > v for t, v in zip((codes, scales, out, dw), before))
    with torch.inference_mode():  # whose tensors have no count
        again = gct.empty_fp8(40, 256)
        gct.quantize_fp8(x.detach(), *again)
        y = torch.empty(40, 128, device="cuda")
        gct.matmul_fp8(*again, W, W_scale, y)
    assert torch.equal(y, out)


@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
def test_an_output_that_a_graph_has_kept_is_not_overwritten_unnoticed(op):
    x, W, W_scale, _, _ = layer(40, 256, 128)
    codes, scales = gct.empty_fp8(40, 256)
    gct.quantize_fp8(x.detach(), codes, scales)
    out = torch.ones((40, 128) if op == "matmul" else (256, 128), device="cuda")
    factor = torch.ones_like(out, requires_grad=True)
    loss = (factor * out).sum()  # keeps out
    if op == "matmul":
        gct.matmul_fp8(codes, scales, W, W_scale, out)
    else:
        gct.weight_grad_fp8(codes, scales, torch.ones(40, 128, dtype=torch.bfloat16, device="cuda"), out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("tokens", [1, 70, 5000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_gradient_of_a_32_bit_bias_has_32_bits(dtype, tokens):
    """Sums of `tokens` fp32 additions: at most tokens * 2^-23 of the terms' sizes off, and no 16-bit rounding."""
    x, W, W_scale, weight, bias = layer(tokens, 128, 96, dtype=dtype, bias=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(72)
    y = gct.fp8_linear(x.detach(), W, W_scale, None, bias)
    dy = torch.randn(y.shape, generator=g, device="cuda").to(dtype)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    db, = torch.autograd.grad(y, bias, dy)
    assert torch.cuda.max_memory_allocated() - held < dy.numel() * 2 + 65536  # no 32-bit copy of dy
    assert db.dtype == torch.float32
    want, S = dy.double().sum(0), dy.double().abs().sum(0)
    assert ((db.double() - want).abs() <= tokens * 2.0 ** -23 * S).all()


@pytest.mark.parametrize("bias", [torch.bfloat16, torch.float16, torch.float32])
def test_bias_gradients_have_the_biass_type(bias):
    x, W, W_scale, weight, b = layer(33, 128, 96, bias=bias)
    gct.fp8_linear(x, W, W_scale, weight, b).backward(torch.ones(33, 96, dtype=torch.bfloat16, device="cuda"))
    assert b.grad.dtype == bias and (b.grad == 33).all()


@pytest.mark.parametrize("shape,N", [((3, 0), 40), ((2, 5, 0), 40), ((0, 256), 40), ((2, 0, 256), 40), ((0, 0), 40), ((7, 256), 0),
                                     ((256,), 40), ((0,), 40)])
def test_layers_of_no_size(shape, N):
    """No tokens, no inputs, no outputs: bias or nothing forward, zeros or nothing backward."""
    K = shape[-1]
    _, W, W_scale, weight, bias = layer(1, K, N)
    x = torch.ones(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = gct.fp8_linear(x, W, W_scale, weight, bias)
    assert y.shape == (*shape[:-1], N)
    if K == 0:
        assert torch.equal(y, bias.expand(y.shape))
    y.backward(torch.ones_like(y))
    assert x.grad.shape == x.shape and weight.grad.shape == weight.shape and bias.grad.shape == bias.shape
    tokens = y.numel() // N if N else 7
    assert (bias.grad == tokens).all()
    if N == 0:
        assert (x.grad == 0).all()
    if tokens == 0:
        assert (weight.grad == 0).all()
