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
