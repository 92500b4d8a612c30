"""norm_join, norm_join_grad, block_norm, dropout_add and dropout against 64-bit references."""
import itertools

import pytest
import torch

import block_reference as ref
import gemm_collective_tiles_gb300 as gct
from test_gpu_matmul_act import RNG, generator, laid, rng_tensor

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (5, 8), (33, 256), (20, 257), (300, 264), (7, 5003)])
def test_dropout(M, N, dtype):
    g = generator(M * N)
    x, r = (torch.randn(M, N, generator=g, device="cuda").to(dtype) for _ in range(2))
    for layout, p, residual in itertools.product(("rows", "odd rows", "cols", "every other"), (0.0, 0.1, 0.5, 1.0), (False, True)):
        out = laid(torch.full_like(x, 9), layout)
        gct.dropout_add(laid(x, layout), out, p, rng_tensor(), residual=laid(r, layout) if residual else None)
        want = ref.drop(x.double(), p, RNG)
        # v * scale is rounded to fp32, twice with the scale's own rounding, and once more where the residual is added
        tol = want.abs() * 2 * ref.U32
        if residual:
            want = want + r.double()
            tol = tol + want.abs() * ref.U32
        assert ((out.double() - want).abs() <= tol + ref.rounding(want, dtype)).all()
        if not residual:
            assert torch.equal(out == 0, want == 0)


def test_dropout_words_and_rates():
    """The generator's published vectors (key and counter of zeros), and the share that is kept."""
    bits = ref.random_bits(0, 0, 1, 8)[0].tolist()
    assert [bits[2 * i + 1] << 16 | bits[2 * i] for i in range(4)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    x = torch.ones(1000, 1000, device="cuda")
    for p in (0.1, 0.5, 0.9):
        out = torch.empty_like(x)
        gct.dropout_add(x, out, p, rng_tensor())
        kept = (out != 0).double().mean().item()
        assert abs(kept - (1 - p)) < 6 * (p * (1 - p) / 1e6) ** 0.5 + 2.0 ** -16
    other = torch.empty_like(x)
    gct.dropout_add(x, other, 0.9, rng_tensor((RNG[0], RNG[1] + 1)))
    assert not torch.equal(other, out)


def test_dropout_leaves_and_values():
    x = torch.full((40, 72), float("nan"), device="cuda")
    out = torch.empty_like(x)
    gct.dropout_add(x, out, 0.5, rng_tensor())
    kept = ref.random_bits(*RNG, 40, 72).cuda() >= 32768
    assert torch.equal(out.isnan(), kept) and (out[~kept] == 0).all()
    y = torch.randn(6, 5, 33, device="cuda").bfloat16().requires_grad_()
    r = torch.randn(6, 5, 33, device="cuda").bfloat16().requires_grad_()
    rng = rng_tensor()
    o = gct.dropout(y, 0.25, rng, residual=r)
    dy = torch.randn_like(o)
    gy, gr = torch.autograd.grad(o, [y, r], dy)
    want = ref.drop(dy.double().view(30, 33), 0.25, RNG).view_as(dy)
    assert ((gy.double() - want).abs() <= want.abs() * (2.0 ** -8 + 3 * ref.U32)).all() and torch.equal(gr, dy)
    o = gct.dropout(y, 0.25, rng)
    rng += 1
    with pytest.raises(RuntimeError):
        o.sum().backward()
    x = torch.randn(50, 64, device="cuda")
    out = x.clone()
    gct.dropout_add(out, out, 0.5, rng_tensor())  # in place
    assert torch.equal(out, ref.drop(x.double(), 0.5, RNG).float())
    for shape in ((0, 8), (8, 0)):
        assert gct.dropout(torch.empty(shape, device="cuda", requires_grad=True), 0.5, rng_tensor()).shape == shape
    for bad in (dict(p=1.1), dict(p=-1), dict(rng=None), dict(rng=rng[:1]), dict(out=out.half()), dict(residual=x[:10]), dict(x=x.double())):
        with pytest.raises((ValueError, TypeError)):
            gct.dropout_add(**{**dict(x=x, out=out, p=0.5, rng=rng), **bad})


def test_one_mask_in_every_op():
    """The product's epilogue, its gradient and dropout_add drop the same elements."""
    M, N = 300, 264
    ones = torch.ones(M, N, device="cuda").bfloat16()
    want = ref.drop(ones.double(), 0.3, RNG) != 0
    out = torch.empty_like(ones)
    gct.dropout_add(ones, out, 0.3, rng_tensor())
    assert torch.equal(out != 0, want)
    gct.act_grad(ones, None, out, p=0.3, rng=rng_tensor())
    assert torch.equal(out != 0, want)
    for config in (dict(tile_m=256, tile_n=256), dict(tile_m=256, tile_n=128), dict(tile_m=128), dict(tile_m=128, k_split=2)):
        gct.matmul_act(torch.ones(M, 128, device="cuda").bfloat16(), torch.ones(128, N, device="cuda").bfloat16(), out, p=0.3,
                       rng=rng_tensor(), config=config)
        assert torch.equal(out != 0, want)
    gct.matmul_act(torch.ones(16, 128, device="cuda").bfloat16(), torch.ones(128, N, device="cuda").bfloat16(), out[:16], p=0.3,
                   rng=rng_tensor())
    assert torch.equal(out[:16] != 0, want[:16])


# ------------------------------------------------------------------ norms

def norm_case(M, D, dtype, x_dtype, gate_rows=0, x=True, post=None, pre="rms", affine=True, seed=0, layout="rows", scale=0.75,
              vec_dtype=None, shift=0.0):
    g = generator(seed + M + D)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    c = dict(y=laid((rand(M, D) * torch.exp(rand(M, 1)) + shift).to(dtype), layout),
             x=laid((2 * rand(M, D) + 0.3).to(x_dtype), layout) if x else None,
             gate=laid((0.5 + 0.3 * rand(gate_rows, D)).to(vec_dtype or dtype), layout) if gate_rows else None, scale=scale, post=post, pre=pre)
    for name, kind, at in (("post_weight", post, 1.0), ("post_bias", post, 0.0), ("weight", pre, 1.0), ("bias", pre, 0.0)):
        c[name] = (at + 0.2 * rand(D)).to(vec_dtype or dtype) if kind and affine else None
    return c


def stat_error(D):
    """Relative error of a row's mean square: at most ceil(D / 512) + 64 additions one after another (512 threads, or fewer
    with at most 32 elements each), a handful of roundings."""
    return (D / 512 + 64 + 16) * ref.U32


def check_norm(c, dtype, x_dtype, layout="rows", grad=True):
    M, D = c["y"].shape
    f = ref.norm_join(**c)
    h = laid(torch.full((M, D), 9.0, device="cuda").to(x_dtype), layout)
    n = laid(torch.full((M, D), 9.0, device="cuda").to(dtype), layout) if c["pre"] else None
    stats = torch.empty(M, 4, device="cuda")
    gct.norm_join(h=h, n=n, stats=stats, **c)
    e = stat_error(D)
    # errors of u, of h, of n: the post-norm's is relative to each of its terms; a mean is off by e of the mean magnitude
    y = c["y"].double()
    ub, pw = 0.0, 1.0 if c["post_weight"] is None else c["post_weight"].double().abs()
    if c["post"]:
        ub = e * ((f["yhat"].abs() + f["yr"] * y.abs().mean(1, keepdim=True) * (c["post"] == "layer")) * pw) + 4 * ref.U32 * f["u"].abs()
    hb = c["scale"] * f["gate"].abs() * (ub + 3 * ref.U32 * f["u"].abs()) + 2 * ref.U32 * f["h"].abs()
    assert ((h.double() - f["h"]).abs() <= hb + ref.rounding(f["h"], x_dtype) + 1e-30).all()
    if c["pre"]:
        w = 1.0 if c["weight"] is None else c["weight"].double().abs()
        hhb = f["hr"] * (hb + hb.mean(1, keepdim=True) + e * f["h"].abs().mean(1, keepdim=True)) + f["hhat"].abs() * (
            e + f["hr"] ** 2 * (hb * f["h"].abs()).mean(1, keepdim=True) * 2)
        nb = hhb * w + 4 * ref.U32 * (f["n"].abs() + f["hhat"].abs() * w)
        assert ((n.double() - f["n"]).abs() <= nb + ref.rounding(f["n"], dtype) + 1e-30).all()
    if not grad:
        return
    g = generator(M)
    dh = laid(torch.randn(M, D, generator=g, device="cuda").to(x_dtype), layout)
    dn = laid(torch.randn(M, D, generator=g, device="cuda").to(dtype), layout) if c["pre"] else None
    gate_rows = 0 if c["gate"] is None else c["gate"].shape[0]
    want = ref.norm_join_grad(f, dh, dn, gate_rows, c["scale"], c["post"], c["post_weight"], c["pre"], c["weight"])
    got = dict(dy=laid(torch.full((M, D), 9.0, device="cuda").to(dtype), layout), dx=laid(torch.full((M, D), 9.0, device="cuda").to(x_dtype), layout))
    if gate_rows:
        got["dgate"] = laid(torch.full_like(c["gate"], 9.0), layout)
    for v in ("post_weight", "post_bias", "weight", "bias"):
        if c[v] is not None:
            got["d" + v] = torch.full_like(c[v], 9.0)
    gct.norm_join_grad(stats=stats, dh=dh, dn=dn, **c, **got)
    # The first failures here (rows of one element, whose gradient is a difference of equal terms) showed bounds that were
    # relative to the result; errors are relative to the terms: each carries the errors of two norms' values and factors,
    # some 4 e each, and a sum over rows adds a rounding a row.
    for name, t in got.items():
        exact, size = want[name], want["|" + name + "|"]
        rows = 0 if name in ("dx", "dy") else M / gate_rows if name == "dgate" else M
        assert ((t.double() - exact).abs() <= (rows * ref.U32 + 16 * e) * size + ref.rounding(exact, t.dtype)).all(), name


KINDS = [(None, "rms"), (None, "layer"), ("rms", None), ("layer", None), ("rms", "rms"), ("layer", "layer"), ("rms", "layer"), (None, None)]


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 12])
@pytest.mark.parametrize("x", [True, False])
def test_norm_combinations(x, gate_rows, post, pre):
    for affine, layout in ((True, "rows"), (False, "odd rows")):
        check_norm(norm_case(12, 264, BF, BF, gate_rows, x, post, pre, affine, layout=layout), BF, BF, layout)


@pytest.mark.parametrize("dtype,x_dtype", [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (HF, F32)])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 64, 255, 256, 264, 1000, 4096, 4104, 5003, 8192, 16384, 16400])
def test_norm_widths_and_types(D, dtype, x_dtype):
    check_norm(norm_case(5, D, dtype, x_dtype, 1, True, "rms", "layer"), dtype, x_dtype)


@pytest.mark.parametrize("layout", ["odd rows", "cols", "every other"])
@pytest.mark.parametrize("D", [9, 256, 1030, 17000])
def test_norm_layouts(D, layout):
    check_norm(norm_case(6, D, BF, F32, 2, True, "layer", "rms", layout=layout), BF, F32, layout)
    check_norm(norm_case(6, D, HF, HF, 6, True, "rms", "layer", layout=layout, vec_dtype=F32), HF, HF, layout)


@pytest.mark.parametrize("M,gate_rows", [(1, 1), (2, 2), (700, 1), (700, 7), (700, 350), (5000, 5), (5000, 1000), (3000, 3000), (4999, 1)])
def test_norm_sums_over_rows(M, gate_rows):
    """Gate rows that are part of a CTA's rows, all of them, and shared by many CTAs."""
    check_norm(norm_case(M, 136, BF, BF, gate_rows, True, "rms", "rms"), BF, BF)
    check_norm(norm_case(M, 40, HF, F32, gate_rows, False, "layer", "layer", vec_dtype=F32), HF, F32)


@pytest.mark.parametrize("D", [264, 1032, 4096])
@pytest.mark.parametrize("gate_rows", [1, 4, 100, 700])
def test_norm_gates_of_another_type(D, gate_rows):
    """32-bit gates and vectors beside 16-bit rows, and 16-bit ones beside a 32-bit stream, several rows a CTA."""
    check_norm(norm_case(700, D, BF, BF, gate_rows, True, "rms", "layer", vec_dtype=F32), BF, BF)
    check_norm(norm_case(700, D, HF, F32, gate_rows, True, None, "rms", vec_dtype=HF), HF, F32)
    check_norm(norm_case(1400, D, HF, HF, gate_rows, False, "layer", "rms", layout="odd rows", vec_dtype=F32), HF, HF, "odd rows")


@pytest.mark.parametrize("M,D,gate_rows", [(40, 17000, 1), (40, 17000, 8), (300, 16500, 3)])
def test_long_rows(M, D, gate_rows):
    check_norm(norm_case(M, D, BF, F32, gate_rows, True, "layer", "rms"), BF, F32)


def test_norm_of_values_far_from_zero():
    """A mean of 100 deviations: the variance is taken from the centred values."""
    check_norm(norm_case(8, 4096, F32, F32, 0, False, "layer", None, shift=100.0, scale=1.0), F32, F32, grad=False)


def test_norm_zero_and_non_finite_rows():
    y = torch.zeros(4, 256, device="cuda").bfloat16()
    y[1], y[2, 3], y[3] = 1.0, float("nan"), 5.0
    n = torch.empty_like(y)
    gct.norm_join(y, None, n, pre="rms")
    assert (n[0] == 0).all() and (n[1] == 1).all() and n[2].isnan().all() and (n[3] == 1).all()
    gct.norm_join(y, None, n, pre="layer")
    assert (n[0] == 0).all() and (n[1] == 0).all() and n[2].isnan().all() and (n[3] == 0).all()


def test_norm_in_place():
    c = norm_case(33, 520, BF, BF, 1, True, "rms", "rms")
    h, n = torch.empty_like(c["x"]), torch.empty_like(c["y"])
    gct.norm_join(h=h, n=n, **c)
    d = dict(c, x=c["x"].clone(), y=c["y"].clone())
    gct.norm_join(h=d["x"], n=d["y"], **d)
    assert torch.equal(d["x"], h) and torch.equal(d["y"], n)


def test_norm_sizes_of_zero():
    for M, D in ((0, 64), (4, 0), (0, 0)):
        y = torch.empty(M, D, device="cuda", requires_grad=True)
        w = torch.ones(D, device="cuda", requires_grad=True)
        g = torch.ones(1, D, device="cuda", requires_grad=True)
        if M == 0:
            g = None
        h, n = gct.block_norm(y, x=torch.empty(M, D, device="cuda"), gate=g, pre="layer", weight=w)
        (h.sum() + n.sum()).backward()
        assert (w.grad == 0).all() and y.grad.shape == y.shape


@pytest.mark.parametrize("dtype", [BF, F32])
def test_block_norm_gradients(dtype):
    for shape, gate_rows, post, pre in (((3, 5, 264), 3, "rms", "rms"), ((30, 100), 30, None, "layer"), ((7, 65), 1, "layer", None), ((9, 72), 0, None, "rms")):
        M, D = int(torch.tensor(shape[:-1]).prod()), shape[-1]
        c = norm_case(M, D, dtype, dtype, gate_rows, gate_rows > 0, post, pre, scale=0.75 if gate_rows else 1.0)
        leaves = {k: v.detach().clone().requires_grad_() for k, v in c.items() if torch.is_tensor(v)}
        for k in ("y", "x"):
            if k in leaves:
                leaves[k] = leaves[k].detach().view(shape).requires_grad_()
        h, n = gct.block_norm(**{**c, **leaves})
        wide = {k: v.detach().double().requires_grad_() for k, v in leaves.items()}
        flat = {k: (v.view(M, D) if k in ("y", "x") else v) for k, v in wide.items()}
        u = ref.norm(flat["y"], post, flat.get("post_weight"), flat.get("post_bias"), 1e-6)[0]
        if gate_rows:
            u = u * flat["gate"].repeat_interleave(M // gate_rows, 0)
        hh = c["scale"] * u + (flat["x"] if "x" in flat else 0)
        nn = ref.norm(hh, pre, flat.get("weight"), flat.get("bias"), 1e-6)[0]
        g = generator(1)
        dh, dn = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
        outs, douts, wouts = [h], [dh], [hh]
        if pre:
            outs, douts, wouts = outs + [n], douts + [dn], wouts + [nn]
        if h.requires_grad and h.is_leaf:  # nothing joined: h is y itself
            outs, douts, wouts = outs[1:], douts[1:], wouts[1:]
        got = torch.autograd.grad(outs, list(leaves.values()), douts)
        want = torch.autograd.grad(wouts, list(wide.values()), [d.double().view(M, D) for d in douts])
        for k, a, b in zip(leaves, got, want):
            b = b.view(a.shape)
            assert ((a.double() - b).abs() <= ref.rounding(b, dtype) + 2e-4 * b.abs().max()).all(), k


def test_block_norm_uses_of_less():
    y = torch.randn(6, 64, device="cuda", requires_grad=True)
    x = torch.randn(6, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    h, n = gct.block_norm(y, x=x, pre="rms", weight=w)
    h.sum().backward()  # n has no part in it
    assert (y.grad == 1).all() and (x.grad == 1).all() and w.grad is None
    h, n = gct.block_norm(y, pre="rms", weight=w)
    assert h is y
    h, n = gct.block_norm(y, x=x, pre="rms", weight=w)
    y.data.add_(0)
    with torch.no_grad():
        y.add_(1)
    with pytest.raises(RuntimeError):
        n.sum().backward()
    h, n = gct.block_norm(y, x=x, pre="rms", weight=w)
    d, = torch.autograd.grad(n.square().sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_block_norm_saved_tensors_that_are_moved():
    """A hook on saved tensors may bring one back with other strides, in the same place among others."""
    M, D = 40, 264
    g = generator(5)
    base = torch.randn(M, 2 * D, generator=g, device="cuda").bfloat16()
    w = torch.rand(D, generator=g, device="cuda").requires_grad_()
    dh, dn = (torch.randn(M, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    for moved in (0, 1):
        y, x = torch.randn(2, M, D, generator=g, device="cuda").bfloat16().unbind()
        plain = [y.clone().requires_grad_(), x.clone().requires_grad_()]
        want = torch.autograd.grad(gct.block_norm(*plain, post="rms", pre="rms", weight=w), [*plain, w], (dh, dn))
        ins = [y.clone(), x.clone()]
        base[:, :D].copy_(ins[moved])
        ins[moved] = base[:, :D]
        ins = [t.detach().requires_grad_() for t in ins]
        at = base.data_ptr()

        def pack(t):
            there = t.data_ptr() == at
            return there, t.clone(memory_format=torch.contiguous_format) if there else t.detach()

        def unpack(kept):
            there, t = kept
            return base.view(-1)[:M * D].copy_(t.view(-1)).view(M, D) if there else t

        with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
            outs = gct.block_norm(*ins, post="rms", pre="rms", weight=w)
        got = torch.autograd.grad(outs, [*ins, w], (dh, dn))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_norm_refusals():
    y, x, w = torch.zeros(6, 64, device="cuda").bfloat16(), torch.zeros(6, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda")
    n = torch.empty_like(y)
    for bad in (dict(pre=None), dict(n=None), dict(pre="batch"), dict(post_weight=w), dict(weight=w[:63]), dict(gate=w.view(1, 64)[:, :63]),
                dict(gate=torch.ones(4, 64, device="cuda")), dict(gate=torch.ones(12, 64, device="cuda")), dict(x=x.half()), dict(x=x[:5]),
                dict(n=n.float()), dict(stats=torch.empty(6, 3, device="cuda")), dict(y=y.cpu()), dict(weight=w.cpu()),
                dict(h=torch.empty(6, 64, device="cuda", dtype=HF)), dict(gate=torch.ones(0, 64, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            gct.norm_join(**{**dict(y=y, h=None, n=n, x=x, pre="rms", weight=w), **bad})
    with pytest.raises(gct.IrisError):
        gct.norm_join(y, None, n, pre="rms", eps=-1.0)
    stats = torch.zeros(6, 4, device="cuda")
    for bad in (dict(dh=None, dn=None), dict(stats=None), dict(dx=y.float()), dict(dgate=w.view(1, 64)), dict(dweight=w), dict(pre=None),
                dict(dh=x.half())):
        with pytest.raises((ValueError, TypeError)):
            gct.norm_join_grad(**{**dict(y=y, stats=stats, dh=x, dn=n, x=x, pre="rms"), **bad})
    with pytest.raises(ValueError):
        gct.block_norm(y)
