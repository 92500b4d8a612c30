"""Ways through the operators around linear layers that their users have and a layer does not take: rows of more than 65536
elements, a layer's gradients with any strides, outputs that are inputs, chains of gradients."""
import pytest
import torch

import block_reference as ref
import gemm_collective_tiles_gb300 as gct
from test_gpu_matmul_act import LAYOUTS, RNG, generator, laid, rng_tensor, small_ints
from test_gpu_norm_dropout import check_norm, norm_case

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ rows that a cluster does not hold

@pytest.mark.parametrize("M,D,gate_rows,dtype,x_dtype,post,pre,layout", [
    (1, 65537, 1, F32, F32, "rms", "rms", "rows"), (3, 65544, 1, BF, F32, "layer", "rms", "rows"),
    (5, 70001, 5, HF, HF, "rms", "layer", "odd rows"), (4, 66000, 2, HF, F32, None, "layer", "every other"),
    (160, 65600, 0, BF, BF, "layer", None, "rows"), (310, 65600, 31, BF, BF, "rms", "rms", "rows"),
    (620, 65544, 310, BF, F32, None, "rms", "rows")])
def test_longest_rows(M, D, gate_rows, dtype, x_dtype, post, pre, layout):
    """Gate rows of one row, within a CTA and across several; with and without each norm."""
    check_norm(norm_case(M, D, dtype, x_dtype, gate_rows, M != 4, post, pre, layout=layout), dtype, x_dtype, layout)


def test_longest_rows_without_vectors_or_gradients_of_them():
    check_norm(norm_case(3, 65550, BF, BF, 0, True, "rms", "layer", affine=False), BF, BF)
    c = norm_case(4, 65550, BF, BF, 1, True, "rms", "rms")
    h, n, stats = torch.empty_like(c["y"]), torch.empty_like(c["y"]), torch.empty(4, 4, device="cuda")
    gct.norm_join(h=h, n=n, stats=stats, **c)
    both, dy, dx = [torch.empty_like(c["y"]) for _ in range(2)], torch.empty_like(c["y"]), torch.empty_like(c["y"])
    dw = torch.empty_like(c["weight"])
    gct.norm_join_grad(stats=stats, dh=h, dn=n, dy=both[0], dx=both[1], dweight=dw, **c)
    gct.norm_join_grad(stats=stats, dh=h, dn=n, dy=dy, **c)
    gct.norm_join_grad(stats=stats, dh=h, dn=n, dx=dx, **c)
    assert torch.equal(dy, both[0]) and torch.equal(dx, both[1])


# ------------------------------------------------------------------ a layer's gradients in one call

def layer_case(M, N, K, dtype, layouts, act, p, seed=0):
    """Integers: every step is exact until the one rounding of each output."""
    g = generator(seed)
    ints = dict(dy=small_ints(g, M, N), x=small_ints(g, M, K), weight=small_ints(g, K, N), z=small_ints(g, M, N))
    dz = ref.drop(ints["dy"].double(), p, RNG) * ref.act_grad(ints["z"].double(), act)
    want = dict(dx=dz @ ints["weight"].double().t(), dweight=ints["x"].double().t() @ dz, dbias=dz.sum(0))
    outs = dict(dx=torch.full((M, K), 9.0, device="cuda"), dweight=torch.full((K, N), 9.0, device="cuda"))
    return ({k: laid(v.to(dtype), lay) for (k, v), lay in zip(ints.items(), layouts)}, want,
            {k: laid(v.to(dtype), lay) for (k, v), lay in zip(outs.items(), layouts[4:])})


def check_layer(ins, want, outs, bias_dtype, act, p, workspace=None):
    if bias_dtype is not None:
        outs = dict(outs, dbias=torch.full((ins["dy"].shape[1],), 9.0, dtype=bias_dtype, device="cuda"))
    ws = gct.linear_act_grad(act=act, p=p, rng=rng_tensor() if p else None, workspace=workspace, **ins, **outs)
    assert gct.query_status(ws)[0] == 0
    for k, t in outs.items():
        assert torch.equal(t, want[k].to(t.dtype)), k
    return ws


@pytest.mark.parametrize("act,p", [(None, 0.0), ("relu", 0.0), (None, 0.5), ("relu", 0.5)])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 264, 72), (40, 131, 67), (130, 136, 200), (300, 328, 513)])
def test_layer_gradients_by_size(M, N, K, act, p):
    for dtype, bias_dtype in ((BF, F32), (HF, HF), (BF, BF)):
        check_layer(*layer_case(M, N, K, dtype, ["rows"] * 6, act, p), bias_dtype, act, p)


@pytest.mark.parametrize("lay", LAYOUTS)
@pytest.mark.parametrize("which", range(6), ids=["dy", "x", "weight", "z", "dx", "dweight"])
def test_layer_gradients_by_layout(which, lay):
    for N, act, p in ((136, "relu", 0.5), (131, None, 0.0)):
        layouts = ["rows"] * 6
        layouts[which] = lay
        check_layer(*layer_case(70, N, 200, BF, layouts, act, p), F32, act, p)
        check_layer(*layer_case(70, N, 200, HF, [lay] * 6, act, p), F32, act, p)


@pytest.mark.parametrize("act,p", [(None, 0.0), ("relu", 0.5)])
def test_layer_gradients_of_less(act, p):
    """Each of the three alone, and none: what only the others read need not be there."""
    ins, want, outs = layer_case(70, 136, 200, BF, ["rows"] * 6, act, p)
    no = dict(x=None, weight=None)
    ws = gct.Workspace(256)  # grows
    if act is None:
        ins["z"] = None
    check_layer({**ins, **no}, want, {}, F32, act, p, ws)
    check_layer({**ins, "x": None}, want, {"dx": outs["dx"]}, None, act, p, ws)
    check_layer({**ins, "weight": None}, want, {"dweight": outs["dweight"]}, None, act, p, ws)
    assert gct.linear_act_grad(act=act, p=p, rng=rng_tensor(), workspace=ws, **{**ins, **no}) is ws
    with pytest.raises((ValueError, TypeError)):
        gct.linear_act_grad(dx=outs["dx"], act=act, p=p, rng=rng_tensor(), **{**ins, "weight": None})
    with pytest.raises((ValueError, TypeError)):
        gct.linear_act_grad(dweight=outs["dweight"], act=act, p=p, rng=rng_tensor(), **{**ins, "x": None})


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(9, 264, 200), (300, 131, 520), (2000, 328, 264)])
def test_layer_gradients_are_those_of_its_steps(M, N, K, act):
    """One call against act_grad and two products."""
    g = generator(M)
    dy, z, x, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((M, N), (M, N), (M, K), (K, N)))
    dz, db = torch.empty_like(dy), torch.empty(N, device="cuda")
    gct.act_grad(dy, z, dz, db, act=act, p=0.25, rng=rng_tensor())
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    gct.matmul_act(dz, w.t(), dx)
    gct.matmul_act(x.t(), dz, dw)
    outs = dict(dx=torch.empty_like(x), dweight=torch.empty_like(w), dbias=torch.empty_like(db))
    gct.linear_act_grad(dy, x, w, z, act=act, p=0.25, rng=rng_tensor(), **outs)
    for a, b in zip(outs.values(), (dx, dw, db)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ outputs that are inputs

@pytest.mark.parametrize("layout", ["rows", "odd rows", "every other"])
@pytest.mark.parametrize("M,D", [(1, 264), (33, 520), (3000, 136), (5, 10000), (400, 9001), (9, 16400), (3, 70000)])
def test_norms_in_place(M, D, layout):
    """h is x or y, n is y; dx is dh, dy is dn or y."""
    c = norm_case(M, D, BF, BF, 1, True, "layer", "rms", layout=layout)
    new = lambda: laid(torch.empty(M, D, dtype=BF, device="cuda"), layout)
    keep = lambda t: laid(t.clone(), layout)
    h, n, stats = new(), new(), torch.empty(M, 4, device="cuda")
    gct.norm_join(h=h, n=n, stats=stats, **c)
    for at in (("x", "y"), ("y", None), (None, "y"), ("x", None)):
        d = dict(c, x=keep(c["x"]), y=keep(c["y"]))
        h2, n2 = (d[at[0]] if at[0] else new()), (d[at[1]] if at[1] else new())
        gct.norm_join(h=h2, n=n2, **d)
        assert torch.equal(h2, h) and torch.equal(n2, n)
    alone = keep(c["y"])
    gct.norm_join(**{**c, "y": alone, "pre": None, "weight": None, "bias": None}, h=alone, n=None)
    assert torch.equal(alone, h)
    g = generator(7)
    dh, dn = (laid(torch.randn(M, D, generator=g, device="cuda").bfloat16(), layout) for _ in range(2))
    vectors = lambda: {"d" + k: torch.empty_like(c[k]) for k in ("gate", "post_weight", "post_bias", "weight")}
    want = dict(dy=new(), dx=new(), **vectors())
    gct.norm_join_grad(stats=stats, dh=dh, dn=dn, **c, **want)
    for at in (("dn", "dh"), ("y", "dh"), ("dn", None), (None, "dh"), ("y", None)):
        d = dict(c, y=keep(c["y"]), dh=keep(dh), dn=keep(dn))
        got = dict(dy=d[at[0]] if at[0] else new(), dx=d[at[1]] if at[1] else new(), **vectors())
        gct.norm_join_grad(stats=stats, **d, **got)
        for k, t in got.items():
            assert torch.equal(t, want[k]), (at, k)


@pytest.mark.parametrize("layout", ["rows", "odd rows", "every other"])
@pytest.mark.parametrize("M,N", [(3, 264), (700, 136), (33, 1003)])
def test_act_grad_in_place(M, N, layout):
    g = generator(M)
    dy, z = (laid(torch.randn(M, N, generator=g, device="cuda").half(), layout) for _ in range(2))
    dz, db = torch.empty_like(dy), torch.empty(N, device="cuda")
    gct.act_grad(dy, z, dz, db, act="silu", p=0.25, rng=rng_tensor())
    for which in range(2):
        ins, got = [laid(dy.clone(), layout), laid(z.clone(), layout)], torch.empty_like(db)
        gct.act_grad(*ins, ins[which], got, act="silu", p=0.25, rng=rng_tensor())
        assert torch.equal(ins[which], dz) and torch.equal(got, db)


# ------------------------------------------------------------------ chains

@pytest.mark.parametrize("M,D", [(1, 512), (50, 520), (300, 512), (2000, 512), (333, 517)])
def test_gradients_that_depend_on_each_other(M, D):
    """Kernels start while the one before them ends: a chain through every gradient equals its calls one at a time."""
    g = generator(M + D)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    y0, x0, w, vec, gate = rand(M, D), rand(M, D), (rand(D, D).float() / D ** 0.5).bfloat16(), rand(D), rand(1, D)
    rng, ws = torch.tensor([1, 2], device="cuda"), gct.Workspace(1 << 20)

    def chain(wait):
        y, x, w2 = y0.clone(), x0.clone(), w.clone()
        v2, g2, db = vec.clone(), gate.clone(), vec.clone()
        for _ in range(5):
            n, z, u, dn, out = (torch.empty_like(y) for _ in range(5))
            stats, dw = torch.empty(M, 4, device="cuda"), torch.empty_like(w2)
            kw = dict(x=x, gate=g2, post="rms", post_weight=vec, pre="layer", weight=v2)
            gct.norm_join(y, None, n, stats=stats, **kw)
            wait()
            gct.matmul_act(n, w2, u, bias=db, act="silu", z=z, workspace=ws)
            wait()
            gct.linear_act_grad(u, n, w2, z, dx=dn, dweight=dw, dbias=db, act="silu", p=0.1, rng=rng, workspace=ws)
            wait()
            dg, dv = torch.empty_like(gate), torch.empty_like(vec)
            gct.norm_join_grad(y, stats, u, dn, dy=dn, dx=u, dgate=dg, dweight=dv, workspace=ws, **kw)
            wait()
            gct.norm_join(dn, y, out, x=u, pre="rms", weight=dv)
            wait()
            gct.act_grad(out, n, x, db, act="gelu", workspace=ws)
            wait()
            gct.norm_join(dw, None, w2, pre="rms")
            wait()
            w2.mul_(D ** -0.5)
            gct.norm_join(dg, None, g2, pre="rms")
            wait()
            gct.norm_join(dv.view(1, D), None, v2.view(1, D), pre="rms")
            wait()
            gct.norm_join(db.view(1, D), None, db.view(1, D), pre="rms")
            wait()
        return y, x, w2, v2, g2, db

    want = chain(torch.cuda.synchronize)
    assert all(t.isfinite().all() for t in want)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
    assert gct.query_status(ws)[0] == 0
