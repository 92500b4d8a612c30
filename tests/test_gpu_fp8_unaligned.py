"""8-bit float ops on rows that start anywhere: 16 bytes at a time, shifted.

Quantisation follows its reference bit for bit, and products of small integers
with power-of-two scales are exact in fp32 in any order and rounded once, so
every comparison here is for equality; what lies around an output stays."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import T, check_quantize, done, f64, mm_ints, mm_want, values, wg_ints, wg_want

pytestmark = pytest.mark.gpu


def placed(t, pitch, at):
    """The values of t in rows `pitch` apart, the first `at` elements into its memory; no byte more than they need."""
    M, K = t.shape
    buf = torch.zeros(at + (M - 1) * pitch + K, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=t.device)
    v = torch.as_strided(buf.view(t.dtype) if t.element_size() == 1 else buf, (M, K), (pitch, 1), at)
    if t.element_size() == 1:
        torch.as_strided(buf, (M, K), (pitch, 1), at).copy_(t.view(torch.uint8))
    else:
        v.copy_(t)
    return v


def surrounded(M, N, dtype, pitch, at):
    """A matrix to write within a buffer of a value that no result has; the buffer, and where the matrix lies."""
    buf = torch.full((at + M * pitch + 64,), -77.0, dtype=dtype, device="cuda")
    mine = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(mine, (M, N), (pitch, 1), at).fill_(True)
    return torch.as_strided(buf, (M, N), (pitch, 1), at), buf, mine


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape,pitch", [((1, 17), 17), ((1, 4096), 4096), ((2, 16), 19), ((37, 15), 15), ((70, 129), 129),
                                         ((130, 500), 503), ((200, 1111), 1111), ((129, 256), 261)])
def test_quantize_from_any_element(shape, pitch, src, block):
    g = np.random.default_rng(3)
    x = values(g, *shape, src)
    for at in range(1, 16 // x.element_size() + 1):
        codes, scales = gct.empty_fp8(*shape, block)
        check_quantize(placed(x, pitch, at), src, "e4m3", block, at % 2 == 0, codes, scales)


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_quantize_extremes_from_any_element(src, block):
    g = np.random.default_rng(4)
    x = values(g, 150, 401, src)
    top = torch.finfo(T[src]).max
    for i, v in enumerate([float("nan"), float("inf"), -float("inf"), top, -top, 0.0, torch.finfo(T[src]).smallest_normal]):
        x[7 * i, 13 * i] = v
        x[149 - i, 400 - i] = v
    x[60:64] = 0
    x[70] = float("nan")
    for at in (1, 3):
        codes, scales = gct.empty_fp8(*x.shape, block, torch.float8_e5m2)
        check_quantize(placed(x, 401, at), src, "e5m2", block, False, codes, scales)


@pytest.mark.parametrize("out_t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(tile_m=256)])
@pytest.mark.parametrize("M,N,pitch", [(70, 300, 300), (33, 1, 1), (257, 260, 263), (300, 647, 647), (128, 77, 90), (31, 65, 65)])
def test_matmul_into_rows_that_start_anywhere(M, N, pitch, config, out_t):
    a, sa, b, sb = mm_ints(M, 200, N, False, seed=21)
    want, _ = mm_want(a, sa, b, sb)
    want = torch.from_numpy(want).float().to(T[out_t])
    for at in (0, 1, 2, 3, 5, 7, 8):
        out, buf, mine = surrounded(M, N, T[out_t], pitch, at)
        done(gct.matmul_fp8(a, sa, b, sb, out, config=config))
        assert torch.equal(out.cpu(), want)
        assert (buf[~mine] == -77).all()


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("config", [dict(tile_m=128, k_split=1), dict(tile_m=128, k_split=4), dict(tile_m=256)])
@pytest.mark.parametrize("K,N,pitch", [(70, 300, 301), (257, 333, 333), (300, 15, 15)])
def test_weight_grad_into_rows_that_start_anywhere(K, N, pitch, config, out_t):
    x, sx, dy = wg_ints(300, K, N, "bf16")
    want, _ = wg_want(x, sx, dy)
    want = torch.from_numpy(want).float().to(T[out_t])
    for at in (0, 1, 2, 3, 7):
        out, buf, mine = surrounded(K, N, T[out_t], pitch, at)
        done(gct.weight_grad_fp8(x, sx, dy, out, config=config))
        assert torch.equal(out.cpu(), want)
        assert (buf[~mine] == -77).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 17, 3), (5, 700, 33), (70, 129, 260), (300, 1111, 333), (130, 15, 600), (3, 1, 40)])
def test_matmul_of_codes_that_start_anywhere(M, K, N, trans):
    a, sa, b, sb = mm_ints(M, K, N, trans, seed=22)
    want, _ = mm_want(a, sa, b, sb)
    for at, more in ((0, 0), (1, 0), (3, 2), (6, 1), (9, 0), (13, 5), (16, 3)):
        A = placed(a, K + more, at)
        B = placed(b.t(), K + more, at).t() if trans else placed(b, N + more, at)
        out = torch.full((M, N), float("nan"), device="cuda")
        done(gct.matmul_fp8(A, sa, B, sb, out))
        assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", [(1, 9, 5), (70, 129, 260), (300, 333, 77), (1000, 40, 1111)])
def test_weight_grad_of_operands_that_start_anywhere(M, K, N, src):
    x, sx, dy = wg_ints(M, K, N, src)
    want, _ = wg_want(x, sx, dy)
    for at, more in ((0, 0), (1, 0), (3, 2), (5, 1), (8, 3)):
        out = torch.full((K, N), float("nan"), device="cuda")
        done(gct.weight_grad_fp8(placed(x, K + more, at), sx, placed(dy, N + more, at), out))
        assert np.array_equal(f64(out), want)


def test_broadcast_operands():
    """Rows or columns that are the same one, a stride of zero apart."""
    a, sa, b, sb = mm_ints(40, 300, 70, False, seed=23)
    same = a[3:4].expand(40, 300)
    want, _ = mm_want(same, sa, b, sb)
    out = torch.empty(40, 70, device="cuda")
    done(gct.matmul_fp8(same, sa, b, sb, out))
    assert np.array_equal(f64(out), want)
    column = b[:, 2:3].expand(300, 70)
    want, _ = mm_want(a, sa, column, sb)
    done(gct.matmul_fp8(a, sa, column, sb, out))
    assert np.array_equal(f64(out), want)
    x, sx, dy = wg_ints(90, 40, 70, "bf16")
    row = dy[1:2].expand(90, 70)
    want, _ = wg_want(x, sx, row)
    out = torch.empty(40, 70, device="cuda")
    done(gct.weight_grad_fp8(x, sx, row, out))
    assert np.array_equal(f64(out), want)
    v = values(np.random.default_rng(5), 1, 333, "bf16").expand(50, 333)
    codes, scales = gct.empty_fp8(50, 333)
    check_quantize(v, "bf16", "e4m3", "rows", True, codes, scales)
