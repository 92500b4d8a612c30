"""8-bit float ops at the ends of what they accept: sizes, values, settings.

Comparisons are for equality: every expected value here is a single product or
a sum of small integers times a power of two, exact in fp32."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import T, done, f64, int_codes, mm_ints, mm_want, wg_ints, wg_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("config", [dict(tile_m=256), dict(tile_m=128, k_split=1)])
@pytest.mark.parametrize("dtype,N", [(torch.float32, (1 << 29) + 1), (torch.bfloat16, (1 << 30) + 1)])
def test_rows_of_2_31_bytes_off_the_16_byte_grid(dtype, N, config):
    """One token's weight gradient into rows whose bytes pass 2^31 and whose
    second row starts off 16 bytes, so that the warps store it themselves."""
    dy = (torch.arange(N, dtype=torch.int32, device="cuda") % 251 - 125).to(torch.bfloat16)[None]
    x, sx = gct.empty_fp8(1, 2)
    x.copy_(torch.tensor([[2.0, -4.0]], device="cuda"))
    sx.fill_(0.5)
    whole = torch.full((2 * N + 64,), 333.0, dtype=dtype, device="cuda")
    out = whole[:2 * N].view(2, N)
    done(gct.weight_grad_fp8(x, sx, dy, out, config=config))
    for row, factor in ((0, 1.0), (1, -2.0)):
        for c in range(0, N, 1 << 26):
            assert torch.equal(out[row, c:c + (1 << 26)], (dy[0, c:c + (1 << 26)] * factor).to(dtype))
    assert (whole[2 * N:] == 333.0).all()


@pytest.mark.parametrize("group_m", [1, 3, 1 << 29, 1 << 30, (1 << 30) + 1, (1 << 31) - 1])
@pytest.mark.parametrize("tile_m", [128, 256])
@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
def test_groups_larger_than_the_matrix(op, tile_m, group_m):
    config = dict(tile_m=tile_m, group_m=group_m, **(dict(k_split=1) if tile_m == 128 else {}))
    if op == "matmul":
        args, fn = mm_ints(700, 300, 1100, False, seed=31), gct.matmul_fp8
        want = mm_want(*args)[0]
    else:
        args, fn = wg_ints(150, 700, 1100, "bf16", seed=31), gct.weight_grad_fp8
        want = wg_want(*args)[0]
    out = torch.full((700, 1100), float("nan"), device="cuda")
    done(fn(*args, out, config=config))
    assert np.array_equal(f64(out), want)


# f16 weight gradients of values that f16 cannot hold, or not with all their bits

def scaled_ints(M, K, exponents, fp8="e4m3", seed=41):
    """Codes that are small integers, and scales of 2^exponents[m], the same in every column block."""
    g = np.random.default_rng(seed)
    x = int_codes(g, M, K, fp8)
    s = torch.from_numpy(np.ldexp(1.0, np.asarray(exponents)).astype(np.float32)).cuda()
    return x, s[:, None].expand(M, R.blocks(K)).t().contiguous().t()


def spread(scales, M, K):
    return torch.from_numpy(R.spread(f64(scales), M, K, True)).float().cuda()


CONFIGS = [None, dict(tile_m=128, k_split=1), dict(k_split=2), dict(k_split=8), dict(tile_m=256), dict(tile_m=256, grid=4)]


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
def test_weight_grad_of_the_largest_f16_inputs(fp8, config):
    """Codes take f16 inputs near 65504 to 65536, which f16 has not; every
    product here is a multiple of 4096 below 2^18, so sums are exact."""
    M, K, N = 700, 300, 264
    g = np.random.default_rng(42)
    top = np.array([65504, -65504, 63488, 61440, -61440, 49152, 0, 32768], np.float32)
    x = torch.from_numpy(g.choice(top, (M, K))).half().cuda()
    codes, scales = gct.empty_fp8(M, K, dtype=T[fp8])
    gct.quantize_fp8(x, codes, scales)
    assert (codes.float() * spread(scales, M, K)).abs().max() == 65536
    dy = torch.from_numpy(g.integers(-3, 4, (M, N)).astype(np.float32)).half().cuda()
    want, _ = wg_want(codes, scales, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(codes, scales, dy, out, config=config))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("exponent", [-126, -100, -30, -16, -9, 0, 8, 16, 40, 100])
def test_weight_grad_f16_of_any_scale(exponent, fp8, config):
    M, K, N = 600, 140, 136
    x, sx = scaled_ints(M, K, np.full(M, exponent), fp8)
    dy = torch.from_numpy(np.random.default_rng(43).integers(-3, 4, (M, N)).astype(np.float32)).half().cuda()
    want, _ = wg_want(x, sx, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out, config=config))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(tile_m=256), dict(tile_m=256, grid=2)])
def test_weight_grad_f16_of_scales_far_apart(config):
    """Runs of 512 tokens with scales of their own, and scales 2^21 apart within
    a run: a column of dY that leaves the large ones out shows what the small
    ones give."""
    M, K, N = 1900, 300, 136
    e = np.zeros(M, int)
    e[:512], e[512:1024], e[1024:] = -60, 40, 9
    e[1025::2] = -12
    x, sx = scaled_ints(M, K, e)
    dy = np.random.default_rng(44).integers(-3, 4, (M, N)).astype(np.float32)
    for k, (lo, step, hi) in enumerate([(0, 1, 512), (512, 1, 1024), (1024, 2, M), (1025, 2, M)]):
        keep = np.zeros(M, bool)
        keep[lo:hi:step] = True
        dy[~keep, k::4] = 0
    dy = torch.from_numpy(dy).half().cuda()
    want, _ = wg_want(x, sx, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out, config=config))
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
def test_weight_grad_keeps_f16s_last_bits(fp8):
    """Inputs of one or a few of f16's finest steps, exactly, as their codes have them."""
    M, K, N = 300, 260, 72
    g = np.random.default_rng(45)
    x = torch.from_numpy(np.ldexp(g.integers(-7, 8, (M, K)), -24).astype(np.float32)).half().cuda()
    codes, scales = gct.empty_fp8(M, K, dtype=T[fp8])
    gct.quantize_fp8(x, codes, scales)
    dy = torch.from_numpy(g.integers(-3, 4, (M, N)).astype(np.float32)).half().cuda()
    want, _ = wg_want(codes, scales, dy)
    out = torch.full((K, N), float("nan"), device="cuda")
    done(gct.weight_grad_fp8(codes, scales, dy, out))
    assert np.array_equal(f64(out), want)


def test_weight_grad_f16_infinite_scales_stay_in_their_block():
    M, K, N = 700, 300, 72
    x, sx = scaled_ints(M, K, np.full(M, 3))
    sx[600, 1], sx[20, 2] = float("inf"), float("nan")
    dy = torch.ones(M, N, dtype=torch.float16, device="cuda")
    out = torch.empty(K, N, device="cuda")
    done(gct.weight_grad_fp8(x, sx, dy, out))
    bad = ~np.isfinite(f64(out))
    assert not bad[:128].any() and bad[128:].all()
    sx[600, 1], sx[20, 2] = 8.0, 8.0
    want, _ = wg_want(x, sx, dy)
    done(gct.weight_grad_fp8(x, sx, dy, out))
    assert np.array_equal(f64(out), want)


def test_linear_layer_of_the_largest_f16_inputs():
    x = torch.full((300, 256), 65504.0, dtype=torch.float16, device="cuda")
    x[::3] = 1.0
    x.requires_grad_()
    weight = torch.full((256, 128), 2.0 ** -9, device="cuda", requires_grad=True)
    W, W_scale = gct.empty_fp8(256, 128, "tiles")
    gct.quantize_fp8(weight.detach(), W, W_scale, block="tiles")
    y = gct.fp8_linear(x, W, W_scale, weight)
    assert torch.equal(y[0], torch.full_like(y[0], 0.5)) and torch.equal(y[1], torch.full_like(y[1], 32768.0))
    y.backward(torch.ones_like(y))
    assert (weight.grad == 200 * 65536.0 + 100).all()


def test_weight_grad_f16_waits_that_run_out():
    """A tile that is never handed over while factors are still being made, and the workspace after it."""
    args = wg_ints(6000, 300, 500, "f16", seed=46)
    want = wg_want(*args)[0]
    out = torch.empty(300, 500, device="cuda")
    for config in (dict(tile_m=128, k_split=1, grid=1), dict(tile_m=256, grid=2), dict(k_split=4)):
        ws = gct.weight_grad_fp8(*args, out, config=dict(debug_skip_flag=2, wait_ns=20_000_000, **config))
        assert gct.query_status(ws)[0] == gct._native.IRIS_ETIMEOUT
        gct.weight_grad_fp8(*args, out, config=config, workspace=ws)
        done(ws)
        assert np.array_equal(f64(out), want)
