"""The 8-bit float entry points reject bad arguments before any GPU work, and
the binding packs the argument structs as the header lays them out.  CPU only."""
import ctypes
import os
import struct
import subprocess

import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from gemm_collective_tiles_gb300 import _native as N

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned address that is never touched


def quant(x=(P, 256, 1), codes=(P, 256, 1), scales=(P, 1, 8), M=8, K=256, xt=N.IRIS_BF16, ct=N.IRIS_E4M3, rows=1, pow2=1):
    return N.load().iris_b200_quantize_fp8(N.pack_quantize_fp8(*x, *codes, *scales, M, K, xt, ct, rows, pow2), None)


def mm(A=(P, 256, 1), sa=(P, 1, 8), B=(P, 64, 1), sb=(P, 1, 1), out=(P, 64, 1), bias=0, M=8, Nn=64, K=256, at=0, bt=0,
       bd=N.IRIS_BF16, od=N.IRIS_BF16, ws=None, nbytes=0, cfg=None):
    a = N.pack_matmul_fp8(*A, *sa, *B, *sb, *out, bias, M, Nn, K, at, bt, bd, od)
    return N.load().iris_b200_matmul_fp8(a, cfg, ws, nbytes, None)


def wg(X=(P, 256, 1), sx=(P, 1, 8), dY=(P, 64, 1), out=(P, 64, 1), M=8, Nn=64, K=256, xt=0, dt=N.IRIS_BF16, od=N.IRIS_F32,
       last=0):
    a = N.pack_weight_grad_fp8(*X, *sx, *dY, *out, M, Nn, K, xt, dt, od, last)
    return N.load().iris_b200_weight_grad_fp8(a, None, None, 0, None)


def test_struct_layout_matches_the_header(tmp_path):
    src = tmp_path / "size.c"
    src.write_text('#include <stdio.h>\n#include "gemm_collective_tiles.h"\n'
                   'int main(void){printf("%zu %zu %zu", sizeof(iris_b200_quantize_fp8_args),'
                   ' sizeof(iris_b200_matmul_fp8_args), sizeof(iris_b200_weight_grad_fp8_args));return 0;}\n')
    exe = tmp_path / "size"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [struct.calcsize(f) for f in ("@11q4i", "@19q4i", "@15q4i")]


def test_null_arguments():
    lib = N.load()
    assert lib.iris_b200_quantize_fp8(None, None) == N.IRIS_EINVAL
    assert lib.iris_b200_matmul_fp8(None, None, None, 0, None) == N.IRIS_EINVAL
    assert lib.iris_b200_weight_grad_fp8(None, None, None, 0, None) == N.IRIS_EINVAL
    assert lib.iris_b200_matmul_fp8_workspace_size(None, None, None) == N.IRIS_EINVAL
    assert lib.iris_b200_weight_grad_fp8_workspace_size(None, None, None) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(K=-1), dict(M=1 << 31), dict(xt=3), dict(xt=-1), dict(ct=2), dict(rows=64), dict(x=(0, 256, 1)),
    dict(codes=(0, 256, 1)), dict(scales=(0, 1, 8)), dict(x=(P, -256, 1)), dict(x=(P, 256, -1)),
    dict(codes=(P, 0, 1)),            # rows on top of each other
    dict(codes=(P, 256, 0)), dict(codes=(P, 100, 1)), dict(scales=(P, 0, 0)),
])
def test_quantize_refusals(change):
    assert quant(**change) == N.IRIS_EINVAL


def test_quantize_alignment_refusals():
    assert quant(x=(P + 1, 256, 1)) == N.IRIS_EALIGN
    assert quant(x=(P + 2, 256, 1), xt=N.IRIS_F32) == N.IRIS_EALIGN
    assert quant(scales=(P + 2, 1, 8)) == N.IRIS_EALIGN


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(Nn=-1), dict(K=-1), dict(K=1 << 31), dict(at=2), dict(bt=-1), dict(od=3), dict(bias=P, bd=5),
    dict(A=(0, 256, 1)), dict(B=(0, 64, 1)), dict(out=(0, 64, 1)), dict(sa=(0, 1, 8)), dict(sb=(0, 1, 1)),
    dict(A=(P, -1, 1)), dict(sb=(P, -1, 1)), dict(out=(P, 0, 1)), dict(out=(P, 63, 1)), dict(out=(P, 64, 0)),
])
def test_matmul_refusals(change):
    assert mm(**change) == N.IRIS_EINVAL


def test_matmul_alignment_refusals():
    assert mm(out=(P + 1, 64, 1)) == N.IRIS_EALIGN
    assert mm(sa=(P + 2, 1, 8)) == N.IRIS_EALIGN
    assert mm(bias=P + 1) == N.IRIS_EALIGN


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(Nn=1 << 31), dict(xt=7), dict(dt=N.IRIS_F32), dict(od=-1), dict(last=1), dict(X=(0, 256, 1)),
    dict(dY=(0, 64, 1)), dict(sx=(0, 1, 8)), dict(out=(0, 64, 1)), dict(dY=(P, -64, 1)), dict(out=(P, 1, 1)),
])
def test_weight_grad_refusals(change):
    assert wg(**change) == N.IRIS_EINVAL


def test_weight_grad_alignment_refusals():
    assert wg(dY=(P + 1, 64, 1)) == N.IRIS_EALIGN
    assert wg(out=(P + 2, 64, 1)) == N.IRIS_EALIGN


def test_empty_outputs_are_no_ops():
    assert quant(M=0) == N.IRIS_OK and quant(K=0) == N.IRIS_OK
    assert mm(M=0) == N.IRIS_OK and mm(Nn=0) == N.IRIS_OK
    assert wg(Nn=0) == N.IRIS_OK and wg(K=0) == N.IRIS_OK
    assert quant(M=0, x=(0, 256, 1), codes=(0, 256, 1), scales=(0, 1, 1)) == N.IRIS_OK


def test_python_refusals():
    codes, scales = gct.empty_fp8(4, 256, device="cpu")
    assert codes.stride() == (256, 1) and scales.shape == (4, 2) and scales.stride(0) == 1
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        gct.quantize_fp8(x, codes, scales)
    with pytest.raises(TypeError, match="x has type"):
        gct.quantize_fp8(x.int(), codes, scales)
    with pytest.raises(TypeError, match="not a tensor"):
        gct.quantize_fp8([1.0], codes, scales)
    with pytest.raises(ValueError, match="unknown block"):
        gct.quantize_fp8(x, codes, scales, block="columns")
    with pytest.raises(ValueError, match="3 dimensions"):
        gct.quantize_fp8(x[None], codes, scales)
    with pytest.raises(TypeError, match="A has type"):
        gct.matmul_fp8(x, scales, codes.t(), scales.t(), x)
    with pytest.raises(TypeError, match="X has type"):
        gct.weight_grad_fp8(x, scales, x, x)
    with pytest.raises(TypeError):
        gct.empty_fp8(4, 4, dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError):
        gct.empty_fp8(4, 4, block="rowwise", device="cpu")
    with pytest.raises(TypeError, match="x is a f16 or bf16"):
        gct.fp8_linear(x, codes.t(), scales.t())


def test_empty_fp8_rows_start_on_16_bytes():
    for K in (1, 15, 16, 17, 127, 1000):
        codes, scales = gct.empty_fp8(3, K, block="tiles", dtype=torch.float8_e5m2, device="cpu")
        assert codes.shape == (3, K) and codes.stride(0) % 16 == 0
        assert scales.shape == (1, -(-K // 128))
