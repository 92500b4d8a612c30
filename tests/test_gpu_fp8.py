"""Block-scaled 8-bit floats on the GPU against 64-bit references.

Exact where the arithmetic is: quantisation follows fp32 definitions bit for
bit, and products of small integers with power-of-two scales are exact in fp32
in any order.  Elsewhere the bounds follow from the arithmetic, with
S = sum |a| |b| over the contraction (scales included) and u = 2^-23, the
largest relative error of one fp32 addition or multiplication, truncated or
rounded:
  matmul       a block's 128 exact products are added in at most 128 steps, the
               scales are multiplied (1), the scaled block is added in one step
               per block, the bias in one:  (128 + 3 + blocks) u S
  weight_grad  chunks of 512 exact products in at most 512 steps, one step per
               chunk:  (512 + 1 + chunks) u S; scales that are not powers of
               two round X to dY's type first:  + h S, h = 2^-8 for bf16 (8
               significant bits, half a step is 2^-9 of the value, taken twice)
               and 2^-11 for f16
and rounding to a 16-bit output adds h |y|, h = 2^-8 (bf16) or 2^-11 (f16); for
f16 at least half its finest step, 2^-25."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}
STEP = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
U = 2.0 ** -23


def rounded(y, t):
    """The most that rounding y to type t can change it by."""
    return np.maximum(HALF[t] * np.abs(y), STEP[t])


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def done(ws):
    rc = gct.query_status(ws)
    assert rc[0] == 0, f"device status {rc}"


def values(g, M, K, src, spread=1.5):
    x = g.standard_normal((M, K)) * np.exp(spread * g.standard_normal((M, 1))) * np.exp(0.5 * g.standard_normal((1, K)))
    return torch.from_numpy(x.astype(np.float32)).to(T[src]).cuda()


# ------------------------------------------------------------------ quantize

def check_quantize(x, src, fp8, block, pow2, codes, scales):
    gct.quantize_fp8(x, codes, scales, block=block, pow2=pow2)
    want_c, want_s = R.quantize(f64(x), src, fp8, block == "rows", pow2)
    assert np.array_equal(f64(scales), want_s)
    assert np.array_equal(f64(codes), want_c, equal_nan=True)


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 1000), (64, 256), (65, 129), (130, 640), (257, 1111)])
def test_quantize(shape, src, fp8, block, pow2):
    g = np.random.default_rng(1)
    x = values(g, *shape, src)
    check_quantize(x, src, fp8, block, pow2, *gct.empty_fp8(*shape, block, T[fp8]))


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["transposed", "pitch", "offset", "spaced", "packed_codes", "codes_t"])
def test_quantize_layouts(layout, src, block):
    g = np.random.default_rng(2)
    M, K = 150, 333
    big = values(g, 400, 700, src)
    codes, scales = gct.empty_fp8(M, K, block)
    if layout == "transposed":
        x = big.t()[:M, :K]
    elif layout == "pitch":
        x = big.flatten()[:M * 335].view(M, 335)[:, :K]
    elif layout == "offset":
        x = big[3:3 + M, 1:1 + K]
    elif layout == "spaced":
        x = big[::2, ::2][:M, :K]
    else:
        x = big[:M, :K]
    if layout == "packed_codes":
        codes = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    elif layout == "codes_t":
        codes = torch.empty(K, M, dtype=torch.float8_e4m3fn, device="cuda").t()
        scales = torch.empty(scales.shape[1], scales.shape[0] + 5, device="cuda").t()[:scales.shape[0]]
    check_quantize(x, src, "e4m3", block, True, codes, scales)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_quantize_extremes(src, fp8, block, aligned):
    g = np.random.default_rng(3)
    M, K = 300, 384 if aligned else 383
    x = values(g, M, K, src)
    top = torch.finfo(T[src]).max
    x[0] = 0.0
    x[1] = float("nan")
    x[2, 5], x[2, 200], x[3, 7] = float("inf"), float("-inf"), float("nan")
    x[4], x[5, 1] = torch.finfo(T[src]).tiny, top
    x[6] = -0.0
    x[7] = x[7] * 0 + top
    x[8] = torch.finfo(T[src]).smallest_normal / 4
    x[140:, 128:256] = 0.0            # a whole tile of zeros and one of infinities
    x[140:, :128] = float("inf")
    for pow2 in (True, False):
        check_quantize(x, src, fp8, block, pow2, *gct.empty_fp8(M, K, block, T[fp8]))


def test_quantize_writes_nothing_else():
    x = values(np.random.default_rng(4), 70, 200, "bf16")
    codes = torch.full((72, 256), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((74, 4), 9.0, device="cuda")
    gct.quantize_fp8(x, codes.view(torch.float8_e4m3fn)[1:71, 16:216], scales[2:72, 1:3])
    codes[1:71, 16:216] = 7
    scales[2:72, 1:3] = 9.0
    assert (codes == 7).all() and (scales == 9.0).all()


def test_quantize_past_2_31_elements():
    M, K = (1 << 31) // 8192 + 100, 8192
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).random_(-17000, 17000)
    codes, scales = gct.empty_fp8(M, K)
    gct.quantize_fp8(x, codes, scales)
    for rows in (slice(0, 3), slice(M - 40, M)):
        want_c, want_s = R.quantize(f64(x[rows]), "bf16", "e4m3", True, True)
        assert np.array_equal(f64(codes[rows]), want_c, equal_nan=True) and np.array_equal(f64(scales[rows]), want_s)


# ------------------------------------------------------------------ products

def int_codes(g, M, K, fp8, top=4):
    """Codes that are small integers."""
    c = torch.from_numpy(g.integers(-top, top + 1, (M, K)).astype(np.float32)).to(T[fp8]).cuda()
    buf = torch.zeros(M, -(-K // 16) * 16, dtype=torch.uint8, device="cuda").view(T[fp8])
    buf.view(torch.uint8)[:, :K] = c.view(torch.uint8)
    return buf[:, :K]


def pow2_scales(g, M, K):
    return torch.from_numpy(np.ldexp(1.0, g.integers(-2, 3, (M, K))).astype(np.float32)).cuda()


def mm_want(a, sa, b, sb, bias=None):
    (M, K), N = a.shape, b.shape[1]
    A = f64(a) * R.spread(f64(sa), M, K, True)
    B = f64(b) * R.spread(f64(sb), K, N, False)
    y = A @ B
    return (y if bias is None else y + f64(bias)), np.abs(A) @ np.abs(B) + (0 if bias is None else np.abs(f64(bias)))


def mm_ints(M, K, N, trans, a8="e4m3", b8="e4m3", seed=5):
    g = np.random.default_rng(seed)
    a, sa = int_codes(g, M, K, a8), pow2_scales(g, R.blocks(K), M).t()
    sb = pow2_scales(g, R.blocks(K), R.blocks(N))
    if trans:
        return a, sa, int_codes(g, N, K, b8).t(), sb.t().contiguous().t()
    return a, sa, int_codes(g, K, N, b8), sb


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 129, 8), (8, 1024, 256), (63, 300, 127), (64, 640, 129), (65, 127, 260),
          (127, 256, 513), (128, 128, 128), (129, 1000, 300), (256, 512, 256), (333, 2500, 700), (1000, 384, 1111)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matmul_integers(shape, trans):
    M, K, N = shape
    a, sa, b, sb = mm_ints(M, K, N, trans)
    want, _ = mm_want(a, sa, b, sb)
    out = torch.full((M, N), float("nan"), device="cuda")
    done(gct.matmul_fp8(a, sa, b, sb, out))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(k_split=2), dict(k_split=4), dict(k_split=8),
                                    dict(tile_m=256), dict(tile_m=128, grid=1), dict(tile_m=256, grid=2), dict(grid=12, k_split=4),
                                    dict(group_m=256)])
@pytest.mark.parametrize("shape", [(5, 700, 300), (70, 640, 260), (300, 1500, 600), (1100, 2000, 900)])
def test_matmul_integers_every_variant(shape, config, trans):
    M, K, N = shape
    a, sa, b, sb = mm_ints(M, K, N, trans, seed=6)
    bias = torch.arange(N, device="cuda").float() % 7
    want, _ = mm_want(a, sa, b, sb, bias)
    out = torch.full((M, N), float("nan"), device="cuda")
    done(gct.matmul_fp8(a, sa, b, sb, out, bias=bias, config=config))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("out_t,bias_t", [("bf16", "bf16"), ("f16", None), ("f32", "f32"), ("f16", "f32"), ("bf16", None)])
@pytest.mark.parametrize("a8,b8", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("shape", [(1, 4096, 700), (17, 1000, 333), (200, 700, 1000), (600, 5000, 520)])
def test_matmul_random(shape, a8, b8, out_t, bias_t, trans):
    M, K, N = shape
    g = np.random.default_rng(7)
    a, sa = gct.empty_fp8(M, K, "rows", T[a8])
    gct.quantize_fp8(values(g, M, K, "bf16"), a, sa, pow2=False)
    w = values(g, *((N, K) if trans else (K, N)), "bf16", 0.2) * 0.02
    b, sb = gct.empty_fp8(*w.shape, "tiles", T[b8])
    gct.quantize_fp8(w, b, sb, block="tiles", pow2=False)
    if trans:
        b, sb = b.t(), sb.t()
    bias = torch.from_numpy(g.standard_normal(N).astype(np.float32)).to(T[bias_t]).cuda() if bias_t else None
    want, S = mm_want(a, sa, b, sb, bias)
    out = torch.full((M, N), float("nan"), dtype=T[out_t], device="cuda")
    done(gct.matmul_fp8(a, sa, b, sb, out, bias=bias))
    bound = (131 + R.blocks(K)) * U * S + rounded(want, out_t)
    assert (np.abs(f64(out) - want) <= bound).all()


@pytest.mark.parametrize("case", ["a_pitch", "a_offset", "a_t", "a_spaced", "b_pitch", "b_offset", "b_spaced", "bt_pitch",
                                  "scales_rows", "scales_one", "out_pitch", "out_t", "out_offset", "out_spaced"])
@pytest.mark.parametrize("shape", [(70, 300, 200), (300, 640, 600)])
def test_matmul_layouts(case, shape):
    M, K, N = shape
    a, sa, b, sb = mm_ints(M, K, N, False, seed=8)

    def relaid(t, rows, cols, r0=0, c0=0, step=1, transpose=False):
        """t inside a larger buffer"""
        buf = torch.zeros(rows, cols, dtype=t.dtype, device="cuda")
        view = (buf.t() if transpose else buf)[r0:, c0:][::step, ::step][:t.shape[0], :t.shape[1]]
        view.view(torch.uint8 if t.element_size() == 1 else t.dtype).copy_(t.view(torch.uint8) if t.element_size() == 1 else t)
        return view

    if case == "a_pitch":
        a = relaid(a, M, K + 1)
    elif case == "a_offset":
        a = relaid(a, M + 2, 1024, 1, 3)
    elif case == "a_t":
        a = relaid(a, K, M, transpose=True)
    elif case == "a_spaced":
        a = relaid(a, 2 * M, 2 * K, step=2)
    elif case == "b_pitch":
        b = relaid(b, K, N + 3)
    elif case == "b_offset":
        b = relaid(b, K + 1, 1024, 1, 5)
    elif case == "b_spaced":
        b = relaid(b, 2 * K, 2 * N, step=2)
    elif case == "bt_pitch":
        b = relaid(b, N, K + 7, transpose=True)
    elif case == "scales_rows":
        sa, sb = sa.contiguous(), sb.t().contiguous().t()
    elif case == "scales_one":
        sa, sb = torch.full((1, 1), 0.5, device="cuda").expand(sa.shape), torch.full((1, 1), 4.0, device="cuda").expand(sb.shape)
    want, _ = mm_want(a, sa, b, sb)
    for out_t in ("f32", "bf16"):
        whole = torch.full((2 * M + 4, 2 * N + 40), -77.0, dtype=T[out_t], device="cuda")
        out = whole[:M, :N]
        if case == "out_pitch":
            whole = torch.full((M, N + 1), -77.0, dtype=T[out_t], device="cuda")
            out = whole[:, :N]
        elif case == "out_t":
            whole = torch.full((N + 1, M + 3), -77.0, dtype=T[out_t], device="cuda")
            out = whole.t()[:M, :N]
        elif case == "out_offset":
            out = whole[1:1 + M, 3:3 + N]
        elif case == "out_spaced":
            out = whole[::2, ::2][:M, :N]
        for config in (None, dict(k_split=2)):
            whole.fill_(-77.0)
            done(gct.matmul_fp8(a, sa, b, sb, out, config=config))
            got = f64(out)
            assert np.array_equal(got, f64(torch.from_numpy(want).to(T[out_t])))
            out.fill_(-77.0)
            assert (whole == -77.0).all(), "written outside the output"


def test_matmul_nan_and_infinity_stay_in_their_rows():
    for M, K, N in ((40, 512, 300), (300, 512, 300)):
        a, sa, b, sb = mm_ints(M, K, N, False, seed=9)
        a[3, 100] = float("nan")
        b[200, 7] = float("nan")
        sa = sa.clone()
        sa[5, 1], sa[6, 0] = float("inf"), float("nan")
        for config in (None, dict(k_split=2)):
            out = torch.empty(M, N, device="cuda")
            done(gct.matmul_fp8(a, sa, b, sb, out, config=config))
            bad = ~np.isfinite(f64(out))
            want = np.zeros_like(bad)
            want[[3, 5, 6]] = True
            want[:, 7] = True
            assert np.array_equal(bad, want)


def test_matmul_empty_contraction():
    for bias in (None, torch.arange(40, device="cuda").float()):
        out = torch.full((5, 40), -1.0, device="cuda")
        a, sa = gct.empty_fp8(5, 0)
        b, sb = gct.empty_fp8(0, 40, "tiles")
        gct.matmul_fp8(a, sa, b, sb, out, bias=bias)
        assert torch.equal(out, torch.zeros_like(out) if bias is None else bias.expand(5, 40))


def test_matmul_operands_past_2_32_bytes():
    K, N = 4200, 200
    whole = torch.zeros(K, 1 << 20, dtype=torch.uint8, device="cuda")  # 4.4 GB
    a, sa, b, sb = mm_ints(9, K, N, False, seed=10)
    far = whole[:, (1 << 20) - 256:][:, :N]
    far.copy_(b.view(torch.uint8))
    want, _ = mm_want(a, sa, b, sb)
    out = torch.empty(9, N, device="cuda")
    done(gct.matmul_fp8(a, sa, far.view(T["e4m3"]), sb, out))
    assert np.array_equal(f64(out), want)


# ------------------------------------------------------------------ weight gradient

def wg_want(x, sx, dy):
    M, K = x.shape
    X = f64(x) * R.spread(f64(sx), M, K, True)
    return X.T @ f64(dy), np.abs(X).T @ np.abs(f64(dy))


def wg_ints(M, K, N, src, fp8="e4m3", seed=11):
    g = np.random.default_rng(seed)
    dy = torch.from_numpy(g.integers(-3, 4, (M, N)).astype(np.float32)).to(T[src]).cuda()
    return int_codes(g, M, K, fp8), pow2_scales(g, R.blocks(K), M).t(), dy


@pytest.mark.parametrize("src,fp8", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2"), ("f16", "e5m2")])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 128, 128), (2, 300, 8), (63, 127, 64), (64, 256, 128), (65, 129, 200),
                                   (512, 128, 256), (513, 200, 192), (1500, 260, 520), (3000, 600, 1111)])
def test_weight_grad_integers(shape, src, fp8):
    M, K, N = shape
    x, sx, dy = wg_ints(M, K, N, src, fp8)
    want, _ = wg_want(x, sx, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(k_split=2), dict(k_split=4), dict(k_split=8),
                                    dict(tile_m=256), dict(tile_m=128, grid=1), dict(tile_m=256, grid=2)])
@pytest.mark.parametrize("shape", [(70, 300, 260), (1000, 300, 600), (700, 1100, 900)])
def test_weight_grad_integers_every_variant(shape, config):
    M, K, N = shape
    x, sx, dy = wg_ints(M, K, N, "bf16", seed=12)
    want, _ = wg_want(x, sx, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out, config=config))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("out_t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("src,fp8", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("shape", [(1, 200, 300), (777, 1000, 333), (2100, 384, 640)])
def test_weight_grad_random(shape, src, fp8, out_t, pow2):
    M, K, N = shape
    g = np.random.default_rng(13)
    x, sx = gct.empty_fp8(M, K, "rows", T[fp8])
    gct.quantize_fp8(values(g, M, K, src, 0.7), x, sx, pow2=pow2)
    dy = (values(g, M, N, "f32") * 1e-2).to(T[src])
    want, S = wg_want(x, sx, dy)
    out = torch.full((K, N), float("nan"), dtype=T[out_t], device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out))
    h = 0.0 if pow2 else HALF[src]
    bound = ((513 + R.blocks(4 * M)) * U + h) * S + rounded(want, out_t)
    if src == "f16":
        # values below f16's normal range round by half its finest step, 2^-25
        bound = bound + 2.0 ** -25 * np.abs(f64(dy)).sum(0)
    assert (np.abs(f64(out) - want) <= bound).all()


@pytest.mark.parametrize("case", ["x_pitch", "x_t", "x_spaced", "dy_pitch", "dy_t", "dy_offset", "scales_rows", "out_pitch", "out_t"])
def test_weight_grad_layouts(case):
    M, K, N = 200, 300, 259
    x, sx, dy = wg_ints(M, K, N, "bf16", seed=14)
    if case == "x_pitch":
        x = x.contiguous().view(torch.uint8).flatten()[:(M - 1) * 299 + 299].view(-1, 299)[:M].view(T["e4m3"])
        sx, K = sx, 299
    elif case == "x_t":
        x = x.view(torch.uint8).t().contiguous().t().view(T["e4m3"])
    elif case == "x_spaced":
        buf = torch.zeros(M, 2 * K, dtype=torch.uint8, device="cuda")
        buf[:, ::2] = x.view(torch.uint8)
        x = buf[:, ::2].view(T["e4m3"])
    elif case == "dy_pitch":
        assert dy.stride(0) % 8
    elif case == "dy_t":
        dy = dy.t().contiguous().t()
    elif case == "dy_offset":
        buf = torch.zeros(M + 1, N + 30, dtype=dy.dtype, device="cuda")
        buf[1:, 3:3 + N] = dy
        dy = buf[1:, 3:3 + N]
    elif case == "scales_rows":
        sx = sx.contiguous()
    want, _ = wg_want(x, sx, dy)
    whole = torch.full((2 * K, 2 * N), -77.0, device="cuda")
    out = whole[:K, :N]
    if case == "out_pitch":
        whole = torch.full((K, N + 2), -77.0, device="cuda")
        out = whole[:, 1:1 + N]
    elif case == "out_t":
        whole = torch.full((N, K + 1), -77.0, device="cuda")
        out = whole.t()[:K]
    done(gct.weight_grad_fp8(x, sx, dy, out))
    assert np.array_equal(f64(out), want)
    out.fill_(-77.0)
    assert (whole == -77.0).all(), "written outside the output"


def test_weight_grad_nan_stays_in_its_row_and_column():
    x, sx, dy = wg_ints(700, 300, 260, "bf16", seed=15)
    x[300, 9] = float("nan")
    dy[600, 11] = float("inf")
    dy[20, 30] = float("nan")
    out = torch.empty(300, 260, device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out))
    bad = ~np.isfinite(f64(out))
    want = np.zeros_like(bad)
    want[9] = True
    want[:, [11, 30]] = True
    assert np.array_equal(bad, want)


def test_weight_grad_without_tokens_is_zero():
    x, sx = gct.empty_fp8(0, 300)
    out = torch.full((300, 40), -1.0, device="cuda")
    gct.weight_grad_fp8(x, sx, torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), out)
    assert (out == 0).all()


# ------------------------------------------------------------------ in use

def test_other_stream_graph_and_shared_workspace():
    cases = [mm_ints(*s, tr, seed=16) for s, tr in (((3, 700, 500), True), ((500, 300, 300), False), ((200, 2000, 130), True))]
    outs = [torch.empty(a.shape[0], b.shape[1], device="cuda") for a, _, b, _ in cases]
    wants = [mm_want(*c)[0] for c in cases]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = None
    with torch.cuda.stream(st):
        for c, o in zip(cases, outs):
            ws = gct.matmul_fp8(*c, o, workspace=ws)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for c, o in zip(cases, outs):
                gct.matmul_fp8(*c, o, workspace=ws)
        for _ in range(3):
            for o in outs:
                o.fill_(-1.0)
            graph.replay()
            st.synchronize()
            for o, w in zip(outs, wants):
                assert np.array_equal(f64(o), w)
    done(ws)
    # a stream given by the caller, while another is current
    for o in outs:
        o.fill_(-1.0)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        ws = gct.matmul_fp8(*c, o, workspace=ws, stream=st)
    st.synchronize()
    for o, w in zip(outs, wants):
        assert np.array_equal(f64(o), w)


def test_results_do_not_depend_on_the_run():
    g = np.random.default_rng(17)
    a, sa = gct.empty_fp8(40, 6000)
    gct.quantize_fp8(values(g, 40, 6000, "bf16"), a, sa, pow2=False)
    b, sb = gct.empty_fp8(6000, 700, "tiles")
    gct.quantize_fp8(values(g, 6000, 700, "bf16"), b, sb, block="tiles")
    dy = values(g, 40, 700, "bf16")
    outs = []
    for _ in range(5):
        y, dw = torch.empty(40, 700, device="cuda"), torch.empty(6000, 700, device="cuda")
        done(gct.matmul_fp8(a, sa, b, sb, y, config=dict(k_split=8)))
        done(gct.weight_grad_fp8(a, sa, dy, dw))
        outs.append((y, dw))
    for y, dw in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(dw, outs[0][1])


@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(k_split=4), dict(tile_m=256)])
@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
def test_a_wait_that_runs_out_is_reported(op, config):
    if op == "matmul":
        args = mm_ints(300, 700, 500, False, seed=18)
        want, fn = mm_want(*args)[0], gct.matmul_fp8
        out = torch.empty(300, 500, device="cuda")
    else:
        args = wg_ints(600, 300, 500, "bf16", seed=18)
        want, fn = wg_want(*args)[0], gct.weight_grad_fp8
        out = torch.empty(300, 500, device="cuda")
    ws = fn(*args, out, config=dict(debug_skip_flag=2, wait_ns=20_000_000, **config))
    rc = gct.query_status(ws)
    assert rc[0] == gct._native.IRIS_ETIMEOUT and rc[2] > 100
    fn(*args, out, config=config, workspace=ws)  # the workspace serves on
    done(ws)
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
@pytest.mark.parametrize("grid,rows,cols", [(152, 300, 700), (6, 500, 500), (10, 900, 700), (4, 250, 1030)])
def test_halved_tail_tiles(op, grid, rows, cols):
    """Pairs cut the tiles of a half empty last round in two along a long
    contraction: one round and several, edges inside the tail tiles, twice on
    one workspace, and with an odd number of stages."""
    config = dict(tile_m=256, grid=grid)
    if op == "matmul":
        args = mm_ints(rows, 4300, cols, True, seed=23)
        want, fn, out = mm_want(*args)[0], gct.matmul_fp8, torch.empty(rows, cols, device="cuda")
    else:
        args = wg_ints(2150, rows, cols, "bf16", seed=23)
        want, fn, out = wg_want(*args)[0], gct.weight_grad_fp8, torch.empty(rows, cols, device="cuda")
    ws = None
    for _ in range(3):
        out.fill_(float("nan"))
        ws = fn(*args, out, config=config, workspace=ws)
        done(ws)
        assert np.array_equal(f64(out), want)
    assert ws.nbytes > 4096, "no tail tile was cut"


def test_refusals_on_the_device():
    a, sa, b, sb = mm_ints(4, 256, 64, False)
    out = torch.empty(4, 64, device="cuda")
    with pytest.raises(ValueError, match="A has 256 columns"):
        gct.matmul_fp8(a, sa, b[:128], sb[:1], out)
    with pytest.raises(ValueError, match="A_scale has shape"):
        gct.matmul_fp8(a, sa[:3], b, sb, out)
    with pytest.raises(ValueError, match="B_scale has shape"):
        gct.matmul_fp8(a, sa, b, sb[:1], out)
    with pytest.raises(ValueError, match="out has shape"):
        gct.matmul_fp8(a, sa, b, sb, out.t())
    with pytest.raises(ValueError, match="bias"):
        gct.matmul_fp8(a, sa, b, sb, out, bias=out[0, :32])
    with pytest.raises(TypeError, match="bias has type"):
        gct.matmul_fp8(a, sa, b, sb, out, bias=torch.zeros(64, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="not on a CUDA device"):
        gct.matmul_fp8(a, sa, b.cpu(), sb, out)
    for bad in (dict(tile_m=64), dict(k_split=3), dict(tile_m=256, k_split=2), dict(grid=10000), dict(grid=2, k_split=4)):
        with pytest.raises(gct.IrisError):
            gct.matmul_fp8(a, sa, b, sb, out, config=bad)
    with pytest.raises(gct.IrisError):  # rows of the output on top of each other
        gct.matmul_fp8(a, sa, b, sb, out[:1].expand(4, 64))
    with pytest.raises(ValueError, match="X has 4 rows"):
        gct.weight_grad_fp8(a, sa, torch.zeros(5, 8, dtype=torch.bfloat16, device="cuda"), out)
    with pytest.raises(TypeError, match="dY has type"):
        gct.weight_grad_fp8(a, sa, out, out)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_linear_layer_gradients(dt):
    """fp8_linear: forward, dx, dweight and dbias against the formulas in 64
    bits on the quantised values, and dweight against differences of the loss
    (which is linear in the weights, so they are exact but for rounding)."""
    g = np.random.default_rng(19)
    K, N = 300, 260
    x = values(g, 70, K, dt, 0.3).view(2, 35, K).requires_grad_()
    weight = (values(g, K, N, "f32", 0.1) * 0.05).requires_grad_()
    bias = values(g, 1, N, dt, 0.1)[0].clone().requires_grad_()
    W, W_scale = gct.empty_fp8(K, N, "tiles")
    gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
    y = gct.fp8_linear(x, W, W_scale, weight, bias)
    dy = values(g, 70, N, dt, 0.3).view(2, 35, N)
    y.backward(dy)

    x2, dy2 = f64(x).reshape(70, K), f64(dy).reshape(70, N)
    Wv = f64(W) * R.spread(f64(W_scale), K, N, False)
    xc, xs = R.quantize(x2, dt, "e4m3", True, True)
    xq = xc * R.spread(xs, 70, K, True)
    dc, ds = R.quantize(dy2, dt, "e5m2", True, True)
    dq = dc * R.spread(ds, 70, N, True)
    h = HALF[dt]

    def near(got, want, S, steps, half):
        assert (np.abs(got - want) <= steps * U * S + half * np.abs(want)).all()

    near(f64(y).reshape(70, N), xq @ Wv + f64(bias), np.abs(xq) @ np.abs(Wv) + np.abs(f64(bias)), 140, h)
    near(f64(x.grad).reshape(70, K), dq @ Wv.T, np.abs(dq) @ np.abs(Wv).T, 140, h)
    near(f64(weight.grad), xq.T @ dy2, np.abs(xq).T @ np.abs(dy2), 520, 0.0)
    near(f64(bias.grad), dy2.sum(0), np.abs(dy2).sum(0), 80, h)

    def loss(w):
        return float((dy2 * (xq @ w)).sum())

    w = f64(weight)
    for k, n in ((0, 0), (5, 250), (299, 17)):
        up, down = w.copy(), w.copy()
        up[k, n] += 0.5
        down[k, n] -= 0.5
        S = np.abs(xq[:, k]) @ np.abs(dy2[:, n])
        # the losses are sums of 70 * 260 terms of 300 products in 64 bits
        slack = 2.0 ** -50 * (np.abs(dy2) * (np.abs(xq) @ np.maximum(np.abs(up), np.abs(down)))).sum()
        assert abs(f64(weight.grad)[k, n] - (loss(up) - loss(down))) <= 520 * U * S + slack


def test_linear_layer_keeps_eight_bits_of_its_input():
    """What autograd holds of x is the codes and scales."""
    x = values(np.random.default_rng(20), 512, 1024, "bf16").requires_grad_()
    W, W_scale = gct.empty_fp8(1024, 256, "tiles")
    gct.quantize_fp8(values(np.random.default_rng(21), 1024, 256, "bf16"), W, W_scale, block="tiles")
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        gct.fp8_linear(x, W, W_scale)
    ours = [t for t in kept if t.data_ptr() not in (W.data_ptr(), W_scale.data_ptr())]
    assert sum(t.numel() * t.element_size() for t in ours) == 512 * 1024 + 512 * 8 * 4


def test_example_trains_and_decodes():
    """The example's perceptron learns (its loss falls to under half in 20 steps;
    the same steps in fp32 end at 0.35 of the first), and its decode form gives what the 64-bit formula gives for the
    quantised layers."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import fp8_mlp_step as ex
    losses, layers = ex.train(steps=20, tokens=300, width=256, hidden=520, rate=3e-3)
    assert losses[-1] < losses[0] / 2
    x = values(np.random.default_rng(22), 1, 256, "bf16", 0.1)
    got = f64(ex.one_token(layers, x))
    v = f64(x)
    for i, layer in enumerate(layers):
        codes, scale = R.quantize(v, "bf16", "e4m3", True, True)
        v = (codes * R.spread(scale, *v.shape, True)) @ (f64(layer.codes) * R.spread(f64(layer.scales), *layer.codes.shape, False))
        v = f64(torch.from_numpy(v + f64(layer.bias)).to(torch.bfloat16))
        v = np.maximum(v, 0) if i == 0 else v
    # the first layer's outputs may round to the neighbouring bf16 value, which
    # moves a code by one step (2^-3 of it) at most
    assert np.abs(got - v).max() <= 2.0 ** -3 * np.abs(v).max()
