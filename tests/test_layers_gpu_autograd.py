"""The differentiable forms around linear layers: derivatives that they do not have, rows that are not there."""
import pytest
import torch

import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fw
    x, w, r = (torch.randn(s, device="cuda").bfloat16() for s in ((6, 64), (64, 40), (6, 40)))
    v, rng = torch.ones(64, device="cuda"), torch.tensor([1, 2], device="cuda")
    dual = lambda t: fw.make_dual(t, torch.ones_like(t))
    with fw.dual_level():
        for call in (lambda: gct.linear_act(dual(x), w), lambda: gct.linear_act(x, dual(w), act="gelu"),
                     lambda: gct.linear_act(x, w, bias=dual(r[0])), lambda: gct.linear_act(x, w, residual=dual(r)),
                     lambda: gct.dropout(dual(x), 0.5, rng), lambda: gct.dropout(x, 0.5, rng, residual=dual(x)),
                     lambda: gct.block_norm(dual(x), pre="rms"), lambda: gct.block_norm(x, x=dual(x), pre="rms"),
                     lambda: gct.block_norm(x, gate=dual(x)), lambda: gct.block_norm(x, pre="rms", weight=dual(v)),
                     lambda: gct.block_norm(x, pre="layer", bias=dual(v)), lambda: gct.block_norm(x, post="rms", post_weight=dual(v))):
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(NotImplementedError):
                    call()
        inside = gct.linear_act(x, w), gct.dropout(x, 0.5, rng), gct.block_norm(x, pre="rms", weight=v)[1]
    outside = gct.linear_act(x, w), gct.dropout(x, 0.5, rng), gct.block_norm(x, pre="rms", weight=v)[1]
    assert all(torch.equal(a, b) for a, b in zip(inside, outside))


@pytest.mark.parametrize("dtype", [F32, HF, BF])
@pytest.mark.parametrize("D", [64, 131, 20000, 70000])
def test_no_rows_give_a_gate_no_gradient(D, dtype):
    """Zeros, whatever lay there, and beside other sums or alone."""
    y, gate = torch.empty(0, D, dtype=dtype, device="cuda"), torch.ones(1, D, dtype=dtype, device="cuda")
    stats, w = torch.empty(0, 4, device="cuda"), torch.ones(D, dtype=dtype, device="cuda")
    for post, grads in ((None, False), ("rms", False), ("layer", True)):
        dgate = torch.full_like(gate, 9)
        of = dict(dweight=torch.full_like(w, 9), dpost_weight=torch.full_like(w, 9)) if grads else {}
        ws = gct.norm_join_grad(y, stats, y, y, x=y, gate=gate, post=post, post_weight=w if post else None, pre="rms", weight=w, dy=y,
                                dgate=dgate, **of)
        assert (dgate == 0).all() and all((t == 0).all() for t in of.values())
        assert gct.query_status(ws)[0] == 0
    for x in (None, torch.empty(0, D, dtype=dtype, device="cuda")):
        g = gate.detach().requires_grad_()
        torch.full_like(g, 9)  # memory that is given out again
        h, n = gct.block_norm(y.detach().requires_grad_(), x=x, gate=g, pre="layer")
        (h.sum() + n.sum()).backward()
        assert (g.grad == 0).all()


@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 131)])
def test_a_gate_row_per_token_of_none(shape):
    """Rows of y, gate and all that is made of them: none; the vectors' gradients are sums of nothing."""
    D = shape[-1]
    leaves = [torch.empty(s, device="cuda", dtype=BF).requires_grad_() for s in (shape, shape, (0, D))] + [
        torch.ones(D, device="cuda", dtype=BF).requires_grad_() for _ in range(2)]
    y, x, gate, w, v = leaves
    with torch.no_grad():
        assert gct.block_norm(y, x=x, gate=gate, pre="rms", weight=w)[1].shape == shape
    h, n = gct.block_norm(y, x=x, gate=gate, post="layer", post_weight=v, pre="rms", weight=w)
    (h.sum() + n.sum()).backward()
    assert all(t.grad.shape == t.shape for t in leaves) and (w.grad == 0).all() and (v.grad == 0).all()
    rows = torch.zeros(6, D, device="cuda", dtype=BF)
    with pytest.raises(ValueError):
        gct.block_norm(rows, gate=gate.detach(), pre="rms")
