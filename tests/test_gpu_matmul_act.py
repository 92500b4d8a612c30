"""matmul_act, act_grad and linear_act against 64-bit references."""
import math

import pytest
import torch

import block_reference as ref
import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
PAIR, HALF, CTA = dict(tile_m=256, tile_n=256), dict(tile_m=256, tile_n=128), dict(tile_m=128)
RNG = (0x1234567890ABCDEF, 0x0FEDCBA987654321)


def rng_tensor(rng=RNG):
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in rng], dtype=torch.int64, device="cuda")


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def laid(t, layout):
    """The matrix with other strides: rows or columns contiguous, rows that start anywhere, neither contiguous."""
    R, C = t.shape
    if layout == "rows":
        return t.contiguous()
    if layout == "cols":
        return t.t().contiguous().t()
    if layout == "odd rows":
        buf = torch.full((R, C + 3), 7, dtype=t.dtype, device=t.device)
        buf[:, 1:C + 1] = t
        return buf[:, 1:C + 1]
    if layout == "odd cols":
        return laid(t.t(), "odd rows").t()
    buf = torch.full((R, 2 * C), 7, dtype=t.dtype, device=t.device)
    buf[:, ::2] = t
    return buf[:, ::2]


def small_ints(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").float()


def check_ints(M, N, K, dtype=BF, out_dtype=F32, config=None, layouts=("rows", "rows", "rows"), bias=True, act=None,
               residual=True, z=False, p=0.0, seed=0, in_place=False):
    """Integers small enough for every step to be exact: outputs have to be equal."""
    g = generator(seed)
    A, B = small_ints(g, M, K).to(dtype), small_ints(g, K, N).to(dtype)
    b = small_ints(g, N).to(dtype) if bias else None
    r = small_ints(g, M, N).to(out_dtype) if residual else None
    want_z = A.double() @ B.double() + (0 if b is None else b.double())
    want = ref.drop(ref.act(want_z, act), p, RNG) + (0 if r is None else r.double())
    out = laid(torch.full((M, N), 77.0, device="cuda").to(out_dtype), layouts[2])
    if residual:
        r = laid(r, layouts[2])
    if in_place:
        out.copy_(r)
        r = out
    zt = laid(torch.full((M, N), 77.0, device="cuda").to(out_dtype), layouts[2]) if z else None
    ws = gct.matmul_act(laid(A, layouts[0]), laid(B, layouts[1]), out, bias=b, act=act, residual=r, z=zt, p=p,
                        rng=rng_tensor() if p else None, config=config)
    assert gct.query_status(ws)[0] == 0
    assert torch.equal(out, want.to(out_dtype))
    if z:
        assert torch.equal(zt, want_z.to(out_dtype))


@pytest.mark.parametrize("config", [None, PAIR, HALF, CTA], ids=["auto", "pair", "half", "cta"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 8, 64), (3, 130, 70), (65, 129, 63), (128, 128, 64), (129, 257, 200), (300, 520, 328),
                                   (513, 264, 1000)])
def test_integers_by_size(M, N, K, config):
    check_ints(M, N, K, config=config)
    check_ints(M, N, K, config=config, dtype=HF, out_dtype=HF, act="relu", p=0.5, z=True)


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_few_rows(M, split):
    for tile_m in (16, 32, 64, 128):
        if M <= tile_m:
            config = dict(tile_m=tile_m, k_split=split)
            check_ints(M, 392, 1024, config=config, z=True, p=0.5, seed=M)
            check_ints(M, 136, 520, out_dtype=BF, config=config, layouts=("cols", "cols", "rows"), act="relu")
            check_ints(M, 129, 300, dtype=HF, out_dtype=HF, config=config, layouts=("every other", "odd rows", "odd rows"))


def test_few_rows_many_tiles():
    """More tiles than CTAs run at once, whole and in parts."""
    for tile_m, split in ((16, 1), (32, 2), (64, 1), (64, 4), (16, 8)):
        check_ints(tile_m - 3, 42000, 256, config=dict(tile_m=tile_m, k_split=split), act="relu", z=True)


@pytest.mark.parametrize("split", [2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(65, 129, 1000), (300, 520, 512), (1500, 1600, 1024)])
def test_split_contraction(M, N, K, split):
    # 1500 x 1600: 156 tiles, so that clusters take several each
    check_ints(M, N, K, config=dict(tile_m=128, k_split=split), z=True, act="relu", p=0.5)


LAYOUTS = ["rows", "cols", "odd rows", "odd cols", "every other"]


@pytest.mark.parametrize("config", [PAIR, HALF, CTA], ids=["pair", "half", "cta"])
@pytest.mark.parametrize("la", LAYOUTS)
@pytest.mark.parametrize("lb", LAYOUTS)
def test_operand_layouts(la, lb, config):
    check_ints(200, 328, 200, layouts=(la, lb, "rows"), config=config)


@pytest.mark.parametrize("config", [PAIR, HALF, CTA, dict(tile_m=128, k_split=4)], ids=["pair", "half", "cta", "split"])
def test_operands_of_whole_groups(config):
    """Rows and columns in multiples of 64: other boxes, which may lie partly past the end."""
    for M, N in ((64, 64), (320, 448), (576, 704)):
        for layouts in (("cols", "rows", "rows"), ("cols", "cols", "rows"), ("rows", "rows", "rows")):
            check_ints(M, N, 264, layouts=layouts, config=config)


@pytest.mark.parametrize("config", [PAIR, HALF], ids=["pair", "half"])
@pytest.mark.parametrize("M,N,K", [(512, 2000, 8192), (250, 250, 4096), (2100, 4300, 4096), (1000, 1300, 6200)])
def test_tail_tiles(M, N, K, config):
    """Last rounds that are cut along the contraction: their sums take memory, and meet in the order of the parts."""
    A, out = torch.ones(M, K, device="cuda").bfloat16(), torch.empty(M, N, device="cuda")
    ws = gct.matmul_act(A, torch.ones(K, N, device="cuda").bfloat16(), out, config=config)
    assert (out == K).all() and ws.nbytes > 256 + 16 * 32 * 64 * 4
    check_ints(M, N, K, layouts=("cols", "rows", "rows"), config=config, z=True, act="relu", p=0.5)
    g = generator(2)
    A, B = torch.randn(M, K, generator=g, device="cuda").half(), torch.randn(K, N, generator=g, device="cuda").half()
    gct.matmul_act(A, B, out, config=config, workspace=ws)
    for _ in range(3):
        again = torch.empty_like(out)
        gct.matmul_act(A, B, again, config=config, workspace=ws)
        assert torch.equal(again, out)
    gct.matmul_act(A, B, again, config=dict(config, debug_skip_flag=1, wait_ns=20_000_000), workspace=ws)
    assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
    gct.matmul_act(A, B, again, config=config, workspace=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("config", [PAIR, HALF, CTA, dict(tile_m=128, k_split=2)], ids=["pair", "half", "cta", "split"])
@pytest.mark.parametrize("lo", LAYOUTS)
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_output_layouts(lo, out_dtype, config):
    for N in (328, 321):
        check_ints(200, N, 128, layouts=("rows", "rows", lo), out_dtype=out_dtype, config=config, z=True, p=0.5, act="relu")
        check_ints(200, N, 128, layouts=("rows", "rows", lo), out_dtype=out_dtype, config=config)
        check_ints(200, N, 128, layouts=("rows", "rows", lo), out_dtype=out_dtype, config=config, residual=False)


@pytest.mark.parametrize("config", [None, PAIR, HALF, CTA, dict(tile_m=128, k_split=4)])
@pytest.mark.parametrize("lo", ["rows", "odd rows"])
def test_adds_to_its_output(lo, config):
    for dtype in (F32, BF):
        check_ints(300, 400, 256, in_place=True, out_dtype=dtype, bias=False, config=config, layouts=("cols", "rows", lo))
        check_ints(9, 400, 256, in_place=True, out_dtype=dtype, bias=False, layouts=("cols", "rows", lo))


def test_what_lies_around_the_output_stays():
    for config in (PAIR, HALF, CTA, dict(tile_m=128, k_split=2), None):
        for M, N in ((200, 264), (200, 261), (3, 261)):
            buf = torch.full((M + 4, N + 24), 5.0, device="cuda").bfloat16()
            out = buf[2:M + 2, 8:N + 8]
            gct.matmul_act(torch.ones(M, 64, device="cuda").bfloat16(), torch.ones(64, N, device="cuda").bfloat16(), out,
                           config=config if M > 64 else None)
            assert (out == 64).all()
            out.fill_(5)
            assert (buf == 5).all()


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1024), (2500, 9000, 256)])
def test_many_tiles_per_cta(M, N, K):
    for config in (PAIR, HALF, CTA):
        check_ints(M, N, K, dtype=HF, out_dtype=F32, config=config, p=0.5, act="relu", z=True)
        check_ints(M, N, K, dtype=HF, out_dtype=HF, config=config, residual=True, layouts=("cols", "cols", "rows"))


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_dtype", [BF, HF, F32])
def test_activations(act, out_dtype):
    """z is set by the bias alone (a product of zeros), over the activations' whole range.

    The activations are correct to 4e-6 of their value: two approximate instructions of 2^-22 each, a polynomial of
    7e-7, and exponents of up to 126 with their own half step, 126 * ln 2 * 2^-24 = 5e-6, in the far tail; below
    2^-126 / 100 results are flushed."""
    z = torch.cat([torch.linspace(-20, 20, 4001), torch.linspace(-0.01, 0.01, 401), torch.tensor([0.0, 1e-30, -1e-30, 100, -100, 6e4,
                                                                                             -6e4])]).cuda()
    if act == "gelu_tanh":
        # its argument grows with the cube, and with it the rounding of the exponent: past -5 that loses the tail
        z = z[(z > -5)]
    N = z.numel()
    out = torch.empty(5, N, dtype=out_dtype, device="cuda")
    zs = torch.empty_like(out)
    gct.matmul_act(torch.zeros(5, 64, device="cuda").bfloat16(), torch.zeros(64, N, device="cuda").bfloat16(), out, bias=z, act=act,
                   z=zs)
    want = ref.act(z.double(), act)
    small = torch.finfo(out_dtype).smallest_normal
    tol = want.abs() * (ref.half_step(out_dtype) + 1.2e-5) + small
    assert ((out.double() - want).abs() <= tol).all()
    assert torch.equal(zs[0], z.to(out_dtype))


def test_nan_and_infinity():
    A = torch.ones(70, 64, device="cuda").bfloat16()
    B = torch.ones(64, 72, device="cuda").bfloat16()
    A[3, 5], B[7, 9] = math.nan, math.inf
    for config in (PAIR, HALF, CTA, dict(tile_m=128, k_split=1)):
        for act in (None, "relu", "gelu", "gelu_tanh", "silu"):
            out = torch.empty(70, 72, device="cuda")
            gct.matmul_act(A, B, out, act=act, config=config)
            want = ref.act(A.double() @ B.double(), act)
            assert torch.equal(out.isnan(), want.isnan())
            assert torch.equal(out.isinf(), want.isinf())
            # dropped elements are 0 whatever they were
            gct.matmul_act(A, B, out, act=act, p=1.0, rng=rng_tensor(), config=config)
            assert (out == 0).all()


@pytest.mark.parametrize("shape", [(0, 5, 3), (4, 0, 3), (4, 5, 0), (0, 0, 0)])
def test_sizes_of_zero(shape):
    M, N, K = shape
    check_ints(M, N, K, z=True, p=0.5, act="relu")


def test_random_values_and_types():
    """Sums of K products in fp32: K + 1 roundings (the tensor cores add in blocks and cut off, counted twice), then bias and
    rounding."""
    for M, N, K, dtype in ((300, 500, 700, BF), (1000, 300, 5000, HF), (20, 1000, 4096, BF), (2000, 2000, 512, HF)):
        g = generator(M)
        A, B = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((M, K), (K, N)))
        bias = torch.randn(N, generator=g, device="cuda")
        for out_dtype in (dtype, F32):
            out = torch.empty(M, N, dtype=out_dtype, device="cuda")
            gct.matmul_act(A, B, out, bias=bias)
            want = A.double() @ B.double() + bias.double()
            size = A.double().abs() @ B.double().abs() + bias.double().abs()
            tol = size * 2 * (K / 16 + 16) * ref.U32 + ref.rounding(want, out_dtype)
            assert ((out.double() - want).abs() <= tol).all()


def test_repeats_bit_for_bit_and_from_a_graph():
    g = generator(5)
    A, B = torch.randn(700, 2048, generator=g, device="cuda").bfloat16(), torch.randn(2048, 900, generator=g, device="cuda").bfloat16()
    for config in (PAIR, HALF, CTA, dict(tile_m=128, k_split=8)):
        first = torch.empty(700, 900, device="cuda")
        ws = gct.matmul_act(A, B, first, act="gelu", config=config)
        out = torch.empty_like(first)
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            gct.matmul_act(A, B, out, act="gelu", config=config, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(5):
            out.zero_()
            graph.replay()
            assert torch.equal(out, first)
        assert gct.query_status(ws)[0] == 0


# ------------------------------------------------------------------ the epilogue's gradient

@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,dz_dtype", [(BF, BF), (HF, HF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,N", [(1, 1), (7, 9), (33, 256), (300, 264), (5, 5003), (2000, 130)])
def test_act_grad(M, N, dtype, dz_dtype, act):
    """Derivatives are correct to 1e-5 of the largest size that they take on, 1.13; columns are summed in any order: M
    roundings of the sum of magnitudes."""
    for layout in ("rows", "odd rows"):
        g = generator(M + N)
        dy = torch.randn(M, N, generator=g, device="cuda").to(dtype)
        z = (3 * torch.randn(M, N, generator=g, device="cuda")).to(dtype)
        dz, db = laid(torch.empty(M, N, dtype=dz_dtype, device="cuda"), layout), torch.empty(N, device="cuda")
        gct.act_grad(laid(dy, layout), laid(z, layout), dz, db, act=act, p=0.25, rng=rng_tensor())
        size = ref.drop(dy.double().abs(), 0.25, RNG)
        want = ref.drop(dy.double(), 0.25, RNG) * ref.act_grad(z.double(), act)
        err = 1.2e-5 * size
        small = torch.finfo(dz_dtype).smallest_normal
        assert ((dz.double() - want).abs() <= err + ref.rounding(want, dz_dtype) + small).all()
        tol = err.sum(0) + want.abs().sum(0) * M * ref.U32 + 1e-30
        assert ((db.double() - want.sum(0)).abs() <= tol).all()


def test_act_grad_of_less():
    g = generator(1)
    dy = torch.randn(100, 72, generator=g, device="cuda").bfloat16()
    db = torch.empty(72, dtype=BF, device="cuda")
    gct.act_grad(dy, None, None, db)
    assert ((db.double() - dy.double().sum(0)).abs() <= dy.double().sum(0).abs() * 2.0 ** -8 + 1e-4).all()
    dz = torch.empty_like(dy)
    gct.act_grad(dy, None, dz, p=0.5, rng=rng_tensor())
    assert torch.equal(dz, ref.drop(dy.double(), 0.5, RNG).bfloat16())
    gct.act_grad(dy, None, dy, p=0.5, rng=rng_tensor())  # in place
    assert torch.equal(dy, dz)
    db.fill_(3)
    gct.act_grad(dy[:0], None, dz[:0], db)  # no rows: no sums
    assert (db == 0).all()


# ------------------------------------------------------------------ the layer

def layer_reference(x, w, b, act, r, p, dy):
    x, w, b, r = (None if t is None else t.detach().double().requires_grad_() for t in (x, w, b, r))
    z = x @ w + (0 if b is None else b)
    y = ref.drop(ref.act(z, act), p, RNG) + (0 if r is None else r)
    leaves = [t for t in (x, w, b, r) if t is not None]
    return y.detach(), torch.autograd.grad(y, leaves, dy.double())


@pytest.mark.parametrize("act", [None, "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N,bias,residual,p", [(130, 200, 264, True, True, 0.25), (40, 333, 111, True, False, 0.0),
                                                   (1, 64, 64, False, True, 0.5), (600, 128, 96, False, False, 0.0)])
def test_layer_gradients(M, K, N, bias, residual, p, dtype, act):
    """Against the formulas.  z and the gradient between the products are rounded to 16 bits: a relative half step of
    each, times the derivative's own size (below 1.13) and slope (below 1.1, times |z|)."""
    g = generator(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    w = (torch.randn(K, N, generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (0.1 * torch.randn(N, generator=g, device="cuda")).to(dtype) if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(dtype) if residual else None
    dy = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    leaves = [t.requires_grad_() for t in (x, w, b, r) if t is not None]
    y = gct.linear_act(x, w, bias=b, act=act, residual=r, p=p, rng=rng_tensor() if p else None)
    grads = torch.autograd.grad(y, leaves, dy)
    want_y, want = layer_reference(x, w, b, act, r, p, dy)
    h = ref.half_step(dtype)
    assert ((y.double() - want_y).abs() <= want_y.abs() * h + 3e-5 * (1 + want_y.abs())).all()
    xd, wd = x.detach().double(), w.detach().double()
    z = xd @ wd + (0 if b is None else b.detach().double())
    ddz = ref.drop(dy.double().abs(), p, RNG) * ((1.13 + (1.1 * z.abs() if act else 0)) * h * 1.02 + 3e-5)
    sizes = [ddz @ wd.abs().t(), xd.abs().t() @ ddz] + ([ddz.sum(0)] if bias else []) + ([0 * dy.double()] if residual else [])
    for got, exact, size in zip(grads, want, sizes):
        assert got.dtype == dtype
        assert ((got.double() - exact).abs() <= size + exact.abs() * h + 1e-4 * size.abs().max() + 1e-6).all()


def test_layer_gradients_against_differences():
    """(f(w + e) - f(w - e)) / 2e of the 64-bit form is what the formulas' gradient says; here the layer's own forward pass,
    with f32-sized steps held up by a sum in 64 bits: bf16 outputs step by 2^-8 of y, so the step e has to move y by many
    steps and the comparison is as coarse as y's rounding over all elements."""
    g = generator(3)
    M, K, N = 64, 64, 64
    x = torch.randn(M, K, generator=g, device="cuda").half()
    w = (torch.randn(K, N, generator=g, device="cuda") / 8).half()
    dy = torch.randn(M, N, generator=g, device="cuda").half()
    rng = rng_tensor()
    x.requires_grad_(), w.requires_grad_()
    f = lambda x, w: (gct.linear_act(x, w, act="gelu", p=0.25, rng=rng).double() * dy.double()).sum()
    dx, dw = torch.autograd.grad(gct.linear_act(x, w, act="gelu", p=0.25, rng=rng), [x, w], dy)
    for t, d, other in ((x, dx, w), (w, dw, x)):
        # an exact step: powers of two, large enough to stay within the type at every element
        e = 2.0 ** -6 * torch.randint(0, 2, t.shape, generator=g, device="cuda").mul(2).sub(1).half()
        up, down = (t.detach() + e), (t.detach() - e)
        step = (up.double() - down.double())
        got = (f(up, w) - f(down, w) if t is x else f(x, up) - f(x, down)).item()
        want = (d.double() * step).sum().item()
        # rounding of y: 2^-11 |y| |dy| an element, as a random walk of M N elements, six deviations; the third derivative
        # (below 2) of steps of 2^-6 through K products of size one at most adds (K^0.5 2^-6)^3 / 3 |dy| an element
        noise = 6 * 2.0 ** -11 * math.sqrt(2 * M * N) + M * N * (math.sqrt(K) / 8 * 2.0 ** -6 * 3) ** 3 / 3
        assert abs(got - want) <= noise + 0.01 * abs(want)


def test_layer_shapes_leaves_and_refusals():
    x = torch.randn(2, 3, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(64, 40, device="cuda").bfloat16().requires_grad_()
    y = gct.linear_act(x, w, act="silu")
    assert y.shape == (2, 3, 40)
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
    for shape in ((0, 64), (2, 0, 64)):
        e = torch.empty(shape, device="cuda", dtype=BF, requires_grad=True)
        b = torch.zeros(40, device="cuda", dtype=BF, requires_grad=True)
        w.grad = None
        gct.linear_act(e, w, bias=b, act="gelu", residual=torch.empty(*shape[:-1], 40, device="cuda", dtype=BF)).sum().backward()
        assert (w.grad == 0).all() and (b.grad == 0).all() and e.grad.shape == e.shape
    # second derivatives
    y = gct.linear_act(x, w, act="silu")
    d, = torch.autograd.grad(y.float().square().sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        d.float().sum().backward()
    # a weight or random state that changed between forward and backward
    rng = rng_tensor()
    y = gct.linear_act(x, w, p=0.5, rng=rng)
    rng += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()
    for bad in (dict(x=x.float()), dict(weight=w.half()), dict(weight=w[:10]), dict(residual=torch.zeros(2, 3, 41, device="cuda").bfloat16()),
                dict(residual=torch.zeros(2, 3, 40, device="cuda")), dict(act="tanh"), dict(p=0.5), dict(p=1.5, rng=rng), dict(p=-0.1),
                dict(p=math.nan), dict(bias=torch.zeros(41, device="cuda")), dict(p=0.5, rng=rng.int()), dict(p=0.5, rng=rng.cpu())):
        with pytest.raises((ValueError, TypeError)):
            gct.linear_act(**{**dict(x=x, weight=w), **bad})


def test_waits_are_bounded():
    """A tile that never reports its accumulator: the call ends with an error that the host reads, and the next one runs."""
    A, B = torch.ones(300, 256, device="cuda").bfloat16(), torch.ones(256, 520, device="cuda").bfloat16()
    for M, config in ((300, PAIR), (300, HALF), (300, CTA), (300, dict(tile_m=128, k_split=2)), (16, dict(tile_m=16)),
                      (16, dict(tile_m=32, k_split=2))):
        out, res = torch.empty(M, 520, device="cuda"), torch.ones(M, 520, device="cuda")
        ws = gct.matmul_act(A[:M], B, out, residual=res, config=config)
        assert gct.query_status(ws)[0] == 0
        gct.matmul_act(A[:M], B, out, residual=res, config=dict(config, debug_skip_flag=1, wait_ns=20_000_000), workspace=ws)
        assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
        ws2 = gct.matmul_act(A[:M], B, out, residual=res, config=config, workspace=ws)
        torch.cuda.synchronize()
        assert (out == 257).all()
