"""8-bit float ops at the ends of what they accept: sizes, values, settings.

Comparisons are for equality: every expected value here is a single product or
a sum of small integers times a power of two, exact in fp32."""
import numpy as np
import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import done, f64, mm_ints, mm_want, wg_ints, wg_want

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
