"""What the differentiable forms around linear layers do in Python, with the library's calls replaced.  CPU only."""
import struct
import weakref

import pytest
import torch

from gemm_collective_tiles_gb300 import _native as N
from gemm_collective_tiles_gb300 import block

GRAD = "@23q2d10i19q"  # the packed arguments of norm_join_grad: dh's matrix is word 35, dn's word 38
DH, DN = 35, 38


class Library:
    """Stands in for the calls of a forward and a backward pass: notes every matrix that _rows has to copy, and at the backward
    call which of these are still held, and the packed arguments."""

    def __init__(self, monkeypatch):
        self.copies, self.packed = [], None
        rows = block._rows

        def noted(t, cols):
            m = rows(t, cols)
            if t is not None and m.data_ptr() != t.data_ptr():
                self.copies.append((weakref.ref(m), m.data_ptr()))
            return m

        def forward(y, h, n, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps, stats, stream=None):
            for t in (h, n, stats):
                if t is not None:
                    t.zero_()
            one = N.IRIS_F32
            return (*block._m(y), *block._m(x), *block._m(gate), *block._m(h), *block._m(n), *map(block._ptr, (post_weight, post_bias)),
                    *map(block._ptr, (weight, bias, stats)), y.shape[0], y.shape[1], 0, scale, eps, one, one, 0, 0, 0, 0, 0,
                    block._NORMS[post], block._NORMS[pre], 0)

        def backward(name, packed, workspace, index):
            assert name == "norm_join_grad"
            self.held = [(at, ref() is not None) for ref, at in self.copies]
            self.packed = struct.unpack(GRAD, packed)

        monkeypatch.setattr(block, "_rows", noted)
        monkeypatch.setattr(block, "_norm_join", forward)
        monkeypatch.setattr(block, "_call", backward)
        monkeypatch.setattr(block, "_layer_workspace", lambda workspace, device: None)


def test_gradients_that_are_copied_are_held(monkeypatch):
    """Incoming gradients that are no matrix as they lie are copied, and each copy lives until the call has been made."""
    lib = Library(monkeypatch)
    y, x = (torch.randn(3, 4, 8, requires_grad=True) for _ in range(2))
    h, n = block.block_norm(y, x=x, pre="rms")
    lib.copies.clear()
    dh, dn = (torch.randn(4, 3, 8).transpose(0, 1) for _ in range(2))
    torch.autograd.grad([h, n], [y, x], [dh, dn])
    assert len(lib.held) == 2 and all(alive for _, alive in lib.held)
    at = [a for a, _ in lib.held]
    assert [lib.packed[DH], lib.packed[DN]] == at and at[0] != at[1]
    assert lib.packed[DH + 1:DH + 3] == (8, 1) == lib.packed[DN + 1:DN + 3]


@pytest.mark.parametrize("which", ["y", "x", "both"])
def test_inputs_that_are_copied_are_held(monkeypatch, which):
    """The same of the saved inputs, with an allocator that gives released memory out again, so that the backward pass's
    copies lie where the forward pass's lay."""
    lib = Library(monkeypatch)
    rows, memory, handed_on = block._rows, {}, []

    def recycled(t, cols):
        m = rows(t, cols)
        if t is None or m.data_ptr() == t.data_ptr():
            return m
        for i in range(8):
            buf, ref = memory.get((m.numel(), i), (None, None))
            if buf is None or ref() is None:
                buf = torch.empty_like(m) if buf is None else buf
                v = buf.view(m.shape).copy_(m).view(m.shape)
                memory[m.numel(), i] = buf, weakref.ref(v)
                handed_on.append((v.data_ptr(), weakref.ref(v)))
                return v

    def gradient(y, stats, dh, dn, x=None, **kw):
        lib.packed = (y.data_ptr(), 0, 0, x.data_ptr())
        call("norm_join_grad", None, None, None)

    def call(name, packed, workspace, index):
        lib.alive = [at for at, ref in handed_on if ref() is not None]
        if packed is not None:
            lib.packed = struct.unpack(GRAD, packed)

    monkeypatch.setattr(block, "_rows", recycled)
    monkeypatch.setattr(block, "_call", call)
    monkeypatch.setattr(block, "norm_join_grad", gradient)
    lay = lambda swap: (torch.randn(4, 3, 8).transpose(0, 1) if swap else torch.randn(3, 4, 8)).requires_grad_()
    y, x = lay(which != "x"), lay(which != "y")
    h, n = block.block_norm(y, x=x, pre="rms")
    torch.autograd.grad([h, n], [y, x], [torch.randn(3, 4, 8) for _ in range(2)])
    for name, t, at in (("y", y, lib.packed[0]), ("x", x, lib.packed[3])):
        assert at == t.data_ptr() if which not in (name, "both") else at in lib.alive


def test_tangents_are_refused(monkeypatch):
    """There is no forward-mode derivative: an input with a tangent is an error, not an output without one.  Without a tangent
    a dual level changes nothing."""
    import torch.autograd.forward_ad as fw
    monkeypatch.setattr(block, "_dropped", lambda x, p, rng, residual=None: x.detach().clone())
    monkeypatch.setattr(block, "_joined", lambda y, *a: (y.detach().clone(), y.detach().clone(), torch.zeros(2, 4), ()))
    monkeypatch.setattr(block, "_linear", lambda x, weight, *a: (x.detach() @ weight.detach(), None))
    x, w = torch.randn(2, 4), torch.randn(4)
    calls = [lambda t, v: block.dropout(t, 0.5, None), lambda t, v: block.dropout(x, 0.5, None, residual=t),
             lambda t, v: block.block_norm(t, pre="rms"), lambda t, v: block.block_norm(x, x=t, pre="rms"),
             lambda t, v: block.block_norm(x, gate=t, pre="rms"), lambda t, v: block.block_norm(x, pre="rms", weight=v),
             lambda t, v: block.block_norm(x, pre="rms", bias=v), lambda t, v: block.block_norm(x, post="rms", post_weight=v),
             lambda t, v: block.block_norm(x, post="layer", post_bias=v)]
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones_like(x)), fw.make_dual(w, torch.ones_like(w))
        for call in calls:
            for mode in (torch.enable_grad, torch.no_grad):
                with mode():
                    with pytest.raises(NotImplementedError):
                        call(*dual)
                    call(x, w)
        for i in range(4):
            with pytest.raises(NotImplementedError):
                args = [x.clone(), torch.randn(4, 3), w[:3], torch.randn(2, 3)]
                args[i] = fw.make_dual(args[i], torch.ones_like(args[i]))
                block._LinearAct.apply(*args[:3], None, args[3], 0.0, None, None) if block._graph_of(*args) else None
    for call in calls:
        call(x, w)
    assert not block._graph_of(x, w, None)


def test_gates_of_no_rows():
    """A row per token, or per sequence, of a batch without any: no gate rows."""
    from test_block_abi import NO, P, nj
    none = (0, 1, 1)
    for gate in (NO, none, (P, 64, 1)):
        assert nj(M=0, y=none, n=none, gate=gate, gate_rows=0) == N.IRIS_OK
    assert nj(M=0, y=none, n=none, gate=(P, 64, 1), gate_rows=1) == N.IRIS_OK
    for rows in (-1, 2):
        assert nj(M=0, y=none, n=none, gate=(P, 64, 1), gate_rows=rows) == N.IRIS_EINVAL
    assert nj(gate=(P, 64, 1), gate_rows=0) == N.IRIS_EINVAL


def test_config_of_the_products():
    """As every op's: a dict of fields, "auto" (which for these is the default, an estimate from the sizes), nothing else."""
    from gemm_collective_tiles_gb300 import fp8, make_config
    assert fp8._cfgp(None) is None and fp8._cfgp("auto") is None
    assert fp8._cfgp(dict(tile_m=128))._obj.tile_m == 128 == fp8._cfgp(make_config(tile_m=128))._obj.tile_m
    with pytest.raises(ValueError, match="unknown config"):
        fp8._cfgp("fast")


def test_workspaces_that_grow_little_by_little():
    """Batches that get longer step by step: what is held, with all that was outgrown, stays within a few times the need."""
    import gemm_collective_tiles_gb300 as gct
    ws, grown = gct.Workspace(256, "cpu"), 0
    ws.buf[5] = 1  # the header moves along
    for need in range(300, 1 << 20, 512):
        if need > ws.nbytes:
            ws._grow(need)
            grown += 1
        assert ws.nbytes >= need and sum(b.numel() for b, _ in ws._outgrown) + ws.nbytes <= 4.5 * need + 4096
    assert grown < 25 and ws.buf[5] == 1 and ws.buf.sum() == 1
    size = ws.nbytes
    ws._grow(size)  # other memory of the same size
    assert ws.nbytes == size
    ws._grow(10 * size)  # one that is far too small: no more than is asked for
    assert ws.nbytes == 10 * size


def test_capture_id_refuses_nothing_to_write():
    assert N.load().iris_b200_capture_id(None, None) == N.IRIS_EINVAL
