"""The entry points around linear layers reject bad arguments before any GPU work, and the binding packs the argument
structs as the header lays them out.  CPU only."""
import ctypes
import glob
import os
import re
import struct
import subprocess

import pytest
import torch

import gemm_collective_tiles_gb300 as gct
from gemm_collective_tiles_gb300 import _native as N

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned address that is never touched
NO = (0, 0, 0)


def mm(A=(P, 64, 1), B=(P, 48, 1), out=(P, 48, 1), residual=NO, z=NO, bias=0, rng=0, M=8, Nn=48, K=64, p=0.0, ab=N.IRIS_BF16,
       ot=N.IRIS_BF16, bt=0, act=0):
    a = N.pack_matmul_act(*A, *B, *out, *residual, *z, bias, rng, M, Nn, K, p, ab, ot, bt, act)
    return N.load().iris_b200_matmul_act(a, None, None, 0, None)


def ag(dy=(P, 48, 1), z=(P, 48, 1), dz=(P, 48, 1), dbias=0, rng=0, M=8, Nn=48, p=0.0, t=N.IRIS_BF16, dt=N.IRIS_BF16, bt=0, act=2):
    return N.load().iris_b200_act_grad(N.pack_act_grad(*dy, *z, *dz, dbias, rng, M, Nn, p, t, dt, bt, act), None, None, 0, None)


def lg(dy=(P, 48, 1), x=(P, 64, 1), w=(P, 48, 1), z=(P, 48, 1), dx=(P, 64, 1), dw=(P, 48, 1), dbias=0, rng=0, M=8, Nn=48, K=64, p=0.0,
       t=N.IRIS_BF16, bt=0, act=2, last=0):
    a = N.pack_linear_act_grad(*dy, *x, *w, *z, *dx, *dw, dbias, rng, M, Nn, K, p, t, bt, act, last)
    return N.load().iris_b200_linear_act_grad(a, None, None, 0, None)


def do(x=(P, 48, 1), residual=NO, out=(P, 48, 1), rng=P, M=8, Nn=48, p=0.5, t=N.IRIS_BF16, last=0):
    return N.load().iris_b200_dropout(N.pack_dropout(*x, *residual, *out, rng, M, Nn, p, t, last), None)


NORM = dict(y=(P, 64, 1), x=NO, gate=NO, h=NO, n=(P, 64, 1), vectors=(0, 0, 0, 0), stats=0, M=8, D=64, gate_rows=0, scale=1.0, eps=1e-6,
            types=(1, 1, 1, 1, 1, 1, 1), post=0, pre=1, last=0)


def packed(**kw):
    c = {**NORM, **kw}
    return (*c["y"], *c["x"], *c["gate"], *c["h"], *c["n"], *c["vectors"], c["stats"], c["M"], c["D"], c["gate_rows"], c["scale"],
            c["eps"], *c["types"], c["post"], c["pre"], c["last"])


def nj(**kw):
    return N.load().iris_b200_norm_join(N.pack_norm_join(*packed(**kw)), None)


def ng(dh=(P, 64, 1), dn=(P, 64, 1), dy=(P, 64, 1), dx=NO, dgate=NO, grads=(0, 0, 0, 0), **kw):
    a = N.pack_norm_join_grad(*packed(**{"stats": P, **kw}), *dh, *dn, *dy, *dx, *dgate, *grads)
    return N.load().iris_b200_norm_join_grad(a, None, None, 0, None)


def test_struct_layout_matches_the_header(tmp_path):
    names = ["matmul_act", "act_grad", "linear_act_grad", "dropout", "norm_join", "norm_join_grad"]
    src = tmp_path / "size.c"
    src.write_text('#include <stdio.h>\n#include "gemm_collective_tiles.h"\nint main(void){printf("' + "%zu " * len(names) + '"' +
                   "".join(f", sizeof(iris_b200_{n}_args)" for n in names) + ");return 0;}\n")
    exe = tmp_path / "size"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [struct.calcsize(f) for f in ("@20qd4i", "@13qd4i", "@23qd4i", "@12qd2i", "@23q2d10i", "@23q2d10i19q")]


def test_null_arguments():
    lib = N.load()
    n = ctypes.c_size_t(0)
    for name in ("matmul_act", "act_grad", "linear_act_grad", "norm_join_grad"):
        assert getattr(lib, "iris_b200_" + name)(None, None, None, 0, None) == N.IRIS_EINVAL
        assert getattr(lib, "iris_b200_" + name + "_workspace_size")(None, None, ctypes.byref(n)) == N.IRIS_EINVAL
        assert getattr(lib, "iris_b200_" + name + "_workspace_size")(None, None, None) == N.IRIS_EINVAL
    for name in ("dropout", "norm_join"):
        assert getattr(lib, "iris_b200_" + name)(None, None) == N.IRIS_EINVAL


NAN = float("nan")


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(Nn=-1), dict(K=-1), dict(K=1 << 31), dict(ab=2), dict(ot=3), dict(act=5), dict(act=-1), dict(p=-0.1), dict(p=1.1),
    dict(p=NAN), dict(p=0.5), dict(bias=P, bt=3), dict(A=NO), dict(B=NO), dict(out=NO), dict(A=(P, -1, 1)), dict(B=(P, 48, -1)),
    dict(out=(P, 0, 1)), dict(out=(P, 47, 1)), dict(z=(P, 0, 1)), dict(residual=(P, -1, 1)),
])
def test_matmul_act_refusals(change):
    assert mm(**change) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(t=3), dict(dt=3), dict(act=7), dict(p=2.0), dict(p=0.5), dict(dy=NO), dict(z=NO), dict(dz=(P, 0, 1)), dict(dbias=P, bt=9)])
def test_act_grad_refusals(change):
    assert ag(**change) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(K=-1), dict(t=2), dict(act=7), dict(p=2.0), dict(p=0.5), dict(dy=NO), dict(x=NO), dict(w=NO), dict(dx=(P, 0, 1)),
    dict(dw=(P, 47, 1)), dict(last=1)])
def test_linear_act_grad_refusals(change):
    assert lg(**change) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(Nn=1 << 31), dict(t=3), dict(last=1), dict(rng=0), dict(p=-1.0), dict(p=NAN), dict(x=NO), dict(out=NO),
    dict(out=(P, 47, 1)), dict(residual=(P, -48, 1))])
def test_dropout_refusals(change):
    assert do(**change) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(D=1 << 31), dict(post=3), dict(pre=-1), dict(last=1), dict(eps=-1.0), dict(eps=NAN), dict(types=(1, 0, 1, 1, 1, 1, 1)),
    dict(types=(2, 1, 1, 1, 1, 1, 1)), dict(types=(3, 3, 1, 1, 1, 1, 1)), dict(y=NO), dict(n=NO), dict(pre=0), dict(n=(P, 63, 1)),
    dict(gate=(P, 64, 1), gate_rows=0), dict(gate=(P, 64, 1), gate_rows=3), dict(gate=(P, 64, 1), gate_rows=16),
    dict(vectors=(P, 0, 0, 0)), dict(vectors=(0, P, 0, 0)), dict(vectors=(0, 0, P, 0), types=(1, 1, 1, 1, 1, 5, 1)),
    dict(gate=(P, 64, 1), gate_rows=1, types=(1, 1, 7, 1, 1, 1, 1))])
def test_norm_join_refusals(change):
    assert nj(**change) == N.IRIS_EINVAL


@pytest.mark.parametrize("change", [
    dict(stats=0), dict(dh=NO, dn=NO), dict(pre=0), dict(dgate=(P, 64, 1)), dict(dy=(P, 1, 1)), dict(grads=(P, 0, 0, 0)),
    dict(dx=(P, 0, 1)), dict(y=NO)])
def test_norm_join_grad_refusals(change):
    assert ng(**change) == N.IRIS_EINVAL


def test_alignment_refusals():
    E = N.IRIS_EALIGN
    assert mm(A=(P + 1, 64, 1)) == E and mm(out=(P + 2, 48, 1), ot=N.IRIS_F32) == E and mm(bias=P + 1, bt=N.IRIS_BF16) == E
    assert mm(p=0.5, rng=P + 4) == E and mm(residual=(P + 1, 48, 1)) == E
    assert ag(dy=(P + 1, 48, 1)) == E and ag(dbias=P + 2, bt=N.IRIS_F32) == E
    assert do(x=(P + 1, 48, 1)) == E and do(rng=P + 1) == E
    assert nj(y=(P + 1, 64, 1)) == E and nj(stats=P + 8) == E and nj(vectors=(0, 0, P + 1, 0)) == E
    assert ng(dn=(P + 1, 64, 1)) == E


def test_sizes_of_zero_are_accepted():
    none = (0, 1, 1)  # no memory
    assert mm(M=0, A=none, out=none) == N.IRIS_OK and mm(Nn=0, B=none, out=none) == N.IRIS_OK
    assert do(M=0, x=none, out=none) == N.IRIS_OK and do(Nn=0, x=none, out=none) == N.IRIS_OK
    assert nj(M=0, y=none, n=none) == N.IRIS_OK and nj(D=0, y=none, n=none) == N.IRIS_OK


def test_python_refuses_without_a_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: gct.matmul_act(x, x.t(), x), lambda: gct.dropout_add(x, x, 0.0, None), lambda: gct.norm_join(x, None, x, pre="rms"),
                 lambda: gct.act_grad(x, x, x, act="gelu"), lambda: gct.linear_act_grad(x, None, None, None),
                 lambda: gct.block_norm(x, pre="rms"), lambda: gct.dropout(x, 0.0, None), lambda: gct.linear_act(x, x.t())):
        with pytest.raises((ValueError, TypeError)):
            call()


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(os.path.dirname(gct.__file__), "csrc_block", "*.cu*"))), ids=os.path.basename)
def test_no_read_only_path(path):
    """These kernels start while the one before them still writes what they will read: no loads by the read-only path."""
    with open(path) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg\b|\b__restrict(__)?\b|\bld\.global\S*\.nc\b", code)


def test_reference_generator():
    """The published vectors of Philox4x32-10 for a key and counter of zeros, and of ones."""
    import block_reference as ref
    words = lambda b: [int(b[2 * i + 1]) << 16 | int(b[2 * i]) for i in range(4)]
    assert words(ref.random_bits(0, 0, 1, 8)[0]) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_norm_gradient_of_rows_without_elements():
    """Rows of no elements have no threads to plan for: done before a GPU is asked for anything."""
    none = dict(D=0, y=(P, 1, 1), n=(P, 1, 1), dh=(P, 1, 1), dn=(P, 1, 1), dy=(P, 1, 1))
    assert ng(**none) == N.IRIS_OK
    kw = {k: none[k] for k in ("D", "y", "n")}
    a = N.pack_norm_join_grad(*packed(stats=P, **kw), *none["dh"], *none["dn"], *none["dy"], *NO, *NO, 0, 0, 0, 0)
    n = ctypes.c_size_t()
    assert N.load().iris_b200_norm_join_grad_workspace_size(a, None, ctypes.byref(n)) == N.IRIS_OK and n.value > 0
