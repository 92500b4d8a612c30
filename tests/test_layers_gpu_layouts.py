"""block_norm of tensors (..., D) whose gradients, or who themselves, are no matrix as they lie."""
import pytest
import torch

import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def tensors(B, S, D, dtype, x_dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ins = dict(y=rand(B, S, D).to(dtype), x=rand(B, S, D).to(x_dtype), gate=(0.5 + 0.3 * rand(B, D)).to(dtype),
               post_weight=(1 + 0.2 * rand(D)).to(dtype), weight=(1 + 0.2 * rand(D)).to(dtype))
    return ins, rand(B, S, D).to(x_dtype), rand(B, S, D).to(dtype)


def swapped(t):
    """The same values with the first two dimensions the other way round in memory."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def grads(ins, dh, dn, workspace, **kw):
    leaves = {k: v.detach().requires_grad_() for k, v in ins.items()}
    h, n = gct.block_norm(**leaves, post="rms", workspace=workspace, **kw)
    outs, d = ([h, n], [dh, dn]) if n is not None else ([h], [dh])
    return torch.autograd.grad(outs, list(leaves.values()), d)


# 264: whole pieces; 131: single elements.  A workspace of 256 bytes has to grow, and may take what was released.
@pytest.mark.parametrize("own", [False, True], ids=["stream's", "grows"])
@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("B,S,D", [(3, 5, 264), (4, 70, 131), (8, 300, 1024)])
def test_gradients_in_another_order(B, S, D, x_dtype, own):
    ins, dh, dn = tensors(B, S, D, BF, x_dtype)
    want = grads(ins, dh, dn, None, pre="layer")
    for a, b in ((swapped(dh), swapped(dn)), (swapped(dh), dn), (dh, swapped(dn))):
        got = grads(ins, a, b, gct.Workspace(256) if own else None, pre="layer")
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_gradients_of_outputs_that_are_used_transposed():
    """As a model has it: h goes on with its dimensions swapped, n is averaged over a sequence."""
    ins, _, _ = tensors(3, 5, 264, F32, F32)
    w = torch.randn(5, 3, 264, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")

    def run(h_of, n_of):
        leaves = {k: v.detach().requires_grad_() for k, v in ins.items()}
        h, n = gct.block_norm(**leaves, post="rms", pre="rms")
        return torch.autograd.grad((h_of(h) * w).sum() + n_of(n).square().sum(), list(leaves.values()))

    got = run(lambda h: h.transpose(0, 1), lambda n: n.mean(1))
    dn = []
    want = run(lambda h: h.transpose(0, 1), lambda n: (n.register_hook(lambda g: dn.append(g.contiguous()) or dn[0]), n.mean(1))[1])
    assert dn and all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("own", [False, True], ids=["stream's", "grows"])
@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("B,S,D", [(3, 5, 264), (4, 70, 131), (8, 300, 1024)])
def test_inputs_in_another_order(B, S, D, x_dtype, own):
    ins, dh, dn = tensors(B, S, D, BF, x_dtype)
    want = grads(ins, dh, dn, None, pre="layer")
    for names in ("y", "x", "yx"):
        moved = {k: swapped(v) if k in names else v for k, v in ins.items()}
        for a, b in ((dh, dn), (swapped(dh), swapped(dn))):
            for _ in range(3):  # memory of the forward pass's copies is there for the backward pass's, and others'
                got = grads(moved, a, b, gct.Workspace(256) if own else None, pre="layer")
                assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_inputs_in_another_order_without_a_pre_norm():
    ins, dh, _ = tensors(3, 5, 264, BF, F32)
    del ins["weight"]
    want = grads(ins, dh, None, None)
    got = grads({k: swapped(v) if k in "yx" else v for k, v in ins.items()}, swapped(dh), None, None)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("act", [None, "gelu"])
def test_layers_and_dropout_in_another_order(act):
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    rng = torch.tensor([5, 6], device="cuda")
    x, w, b, r, dy, do = rand(3, 50, 264), rand(264, 136), rand(136), rand(3, 50, 136), rand(3, 50, 136), rand(3, 50, 264)

    def run(lay):
        leaves = [lay(x).requires_grad_(), w.detach().requires_grad_(), b.detach().requires_grad_(), lay(r).requires_grad_()]
        y = gct.linear_act(leaves[0], leaves[1], leaves[2], act=act, residual=leaves[3], p=0.25, rng=rng, workspace=gct.Workspace(256))
        one = torch.autograd.grad(y, leaves, lay(dy))
        o = gct.dropout(leaves[0], 0.25, rng, residual=lay(do))
        return [y.detach(), *one, o.detach(), *torch.autograd.grad(o, leaves[:1], lay(do))]

    for p, q in zip(run(lambda t: swapped(t).detach()), run(lambda t: t.detach().clone())):
        assert torch.equal(p, q)
