"""Waits that run out in the kernels of few rows, and tail tiles that were cut: what the workspace shows of them."""
import numpy as np
import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from test_gpu_fp8 import done, f64, mm_ints, mm_want, wg_ints, wg_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("config", [dict(k_split=1), dict(k_split=4), dict(k_split=1, grid=2), dict(k_split=2, grid=4), dict()])
@pytest.mark.parametrize("M", [1, 16, 17, 20, 32])
def test_few_rows_report_and_recover(M, config, trans):
    args = mm_ints(M, 4200, 900, trans, seed=81)
    want = mm_want(*args)[0]
    out = torch.empty(M, 900, device="cuda")
    for tile in (1, 2, 8):  # the first, one in between, the last of eight column tiles
        ws = gct.matmul_fp8(*args, out, config=dict(debug_skip_flag=tile, wait_ns=20_000_000, **config))
        rc = gct.query_status(ws)
        assert rc[0] == gct._native.IRIS_ETIMEOUT and rc[2] > 100
        for _ in range(2):
            out.fill_(float("nan"))
            gct.matmul_fp8(*args, out, config=config, workspace=ws)
            done(ws)
            assert np.array_equal(f64(out), want)


def padded(t):
    """t in rows of whole 16 bytes, so that nothing has to be copied."""
    per = 16 // t.element_size()
    buf = torch.zeros(t.shape[0], -(-t.shape[1] // per) * per, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("op", ["matmul", "weight_grad"])
@pytest.mark.parametrize("grid,rows,cols", [(152, 300, 700), (6, 500, 500), (10, 900, 700), (4, 250, 1030)])
def test_tail_tiles_are_cut_where_nothing_is_copied(op, grid, rows, cols):
    """The only thing that can make the workspace this large is the sums that
    the halves of cut tiles hand over; a short contraction cuts none."""
    config = dict(tile_m=256, grid=grid)
    if op == "matmul":
        args, fn = mm_ints(rows, 4300, cols, True, seed=82), gct.matmul_fp8
        short = mm_ints(rows, 1000, cols, True, seed=82)
        want = mm_want(*args)[0]
    else:
        x, sx, dy = wg_ints(2150, rows, cols, "bf16", seed=82)
        args, fn = (x, sx, padded(dy)), gct.weight_grad_fp8
        x, sx, dy = wg_ints(500, rows, cols, "bf16", seed=82)
        short = (x, sx, padded(dy))
        want = wg_want(*args)[0]
    out = torch.full((rows, cols), float("nan"), device="cuda")
    ws = fn(*args, out, config=config)
    done(ws)
    assert np.array_equal(f64(out), want)
    assert ws.nbytes > 16 * 16384, "no tail tile was cut"
    assert fn(*short, out, config=config).nbytes == 256
