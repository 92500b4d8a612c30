"""The operators around linear layers together: a block's second half as a model uses them, trained and served, in a
graph, on another stream, from threads."""
import threading

import pytest
import torch

import block_reference as ref
import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def parameters(D, H, dtype=BF, seed=0, grad=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p = dict(w1=rand(D, H) / D ** 0.5, b1=0.1 * rand(H), w2=rand(H, D) / H ** 0.5, b2=0.1 * rand(D), n1=1 + 0.1 * rand(D),
             n2=1 + 0.1 * rand(D), n3=1 + 0.1 * rand(D), gate=0.5 + 0.1 * rand(1, D))
    return {k: v.to(dtype).requires_grad_(grad) for k, v in p.items()}


def block(p, x, y, rng, workspace=None, drop=0.25):
    """y joins x, the sum's norm goes through the perceptron, whose output joins in turn; returns the stream and its norm."""
    h, n = gct.block_norm(y, x=x, post="rms", post_weight=p["n1"], gate=p["gate"], pre="rms", weight=p["n2"], workspace=workspace)
    a = gct.linear_act(n, p["w1"], p["b1"], act="gelu_tanh", workspace=workspace)
    m = gct.linear_act(a, p["w2"], p["b2"], residual=h, p=drop, rng=rng, workspace=workspace)
    return gct.block_norm(gct.dropout(m, drop, rng), x=m, scale=0.5, pre="layer", weight=p["n3"], workspace=workspace)


def reference(p, x, y, rng, drop=0.25):
    p = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    x, y = x.detach().double().requires_grad_(), y.detach().double().requires_grad_()
    h = x + p["gate"] * ref.norm(y, "rms", p["n1"], None, 1e-6)[0]
    n = ref.norm(h, "rms", p["n2"], None, 1e-6)[0]
    m = h + ref.drop(ref.act(n @ p["w1"] + p["b1"], "gelu_tanh") @ p["w2"] + p["b2"], drop, rng)
    h2 = m + 0.5 * ref.drop(m, drop, rng)
    return p, x, y, h2, ref.norm(h2, "layer", p["n3"], None, 1e-6)[0]


def inputs(M, D, dtype=BF, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(M, D, generator=g, device="cuda").to(dtype).requires_grad_() for _ in range(2)]


@pytest.mark.parametrize("dtype", [BF, torch.float16])
@pytest.mark.parametrize("M,D,H", [(1, 64, 256), (70, 264, 1000), (300, 256, 1024), (33, 131, 517)])
def test_block_trains(M, D, H, dtype):
    """Five roundings to 16 bits lie between the inputs and the outputs, and as many on the way back; each is a half step of
    values of the size of one, the products and norms pass such errors on at about their own size, and the gradients' sizes
    are those of their largest elements: 24 half steps of those."""
    p, (x, y), rng = parameters(D, H, dtype), inputs(M, D, dtype), (77, 5)
    out = block(p, x, y, torch.tensor(rng, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(9)
    d = [torch.randn(M, D, generator=g, device="cuda").to(dtype) for _ in out]
    leaves = [x, y, *p.values()]
    got = [o.detach() for o in out] + list(torch.autograd.grad(out, leaves, d))
    wp, wx, wy, h2, n2 = reference(p, x, y, rng)
    want = [h2.detach(), n2.detach()] + list(torch.autograd.grad([h2, n2], [wx, wy, *wp.values()], [v.double() for v in d]))
    for a, b in zip(got, want):
        assert a.shape == b.shape and a.dtype == dtype
        assert (a.double() - b).abs().max() <= 24 * ref.half_step(dtype) * b.abs().max()


def test_decoding_equals_its_rows_of_a_prompt():
    """One token at a time against all at once: other kernels, sums in another order, the same formulas."""
    p, (x, y) = parameters(256, 1024, grad=False), inputs(40, 256)
    with torch.no_grad():
        whole = block(p, x, y, None, drop=0.0)
        for i in (0, 17, 39):
            one = block(p, x[i:i + 1], y[i:i + 1], None, drop=0.0)
            for a, b in zip(one, whole):
                assert (a.float() - b[i:i + 1].float()).abs().max() <= 8 * 2.0 ** -8 * b.float().abs().max()


def test_streams_graphs_and_repeats():
    p, (x, y) = parameters(264, 512), inputs(200, 264)
    rng = torch.tensor([3, 4], device="cuda")
    ws = gct.Workspace(256)
    leaves = [x, y, *p.values()]

    def step(workspace=ws):
        out = block(p, x, y, rng, workspace)
        return [o.detach() for o in out] + list(torch.autograd.grad(out, leaves, [torch.ones_like(o) for o in out]))

    want = [t.clone() for t in step()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(None)  # the stream's own workspace
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for i in range(3):
        rng[1] = 4 + i  # a replay reads what the tensor holds then
        graph.replay()
        torch.cuda.synchronize()
        same = all(torch.equal(a, b) for a, b in zip(got, want))
        assert same == (i == 0)
    rng[1] = 4
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gct.query_status(ws)[0] == 0


def test_dependent_calls_equal_calls_one_at_a_time():
    """Kernels start while the one before them ends: nothing may be read before it is written."""
    for M in (1, 50, 300, 2000):
        p, (x, y) = parameters(512, 1024, grad=False), inputs(M, 512)
        rng = torch.tensor([1, 2], device="cuda")
        with torch.no_grad():
            def chain(wait):
                a, b = x.detach().clone(), y.detach().clone()
                for _ in range(6):
                    n = torch.empty_like(b)
                    gct.norm_join(b, a, n, x=a, post="rms", pre="rms", weight=p["n2"], scale=0.5)
                    wait()
                    u = torch.empty(M, 1024, dtype=BF, device="cuda")
                    gct.matmul_act(n, p["w1"], u, act="silu", workspace=ws)
                    wait()
                    gct.matmul_act(u, p["w2"], b, bias=p["b2"], residual=n, p=0.1, rng=rng, workspace=ws)
                    wait()
                    gct.dropout_add(b, b, 0.1, rng)
                    wait()
                    gct.act_grad(b, n, b, act="gelu", workspace=ws)
                    wait()
                return a, b
            ws = gct.Workspace(1 << 20)
            want = chain(torch.cuda.synchronize)
            for _ in range(4):
                got = chain(lambda: None)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_threads():
    """Two threads with a workspace between them on one stream, and each as a thread's first work."""
    p, (x, y) = parameters(264, 512, grad=False), inputs(120, 264)
    ws = gct.Workspace(256)
    rng = torch.tensor([3, 4], device="cuda")
    with torch.no_grad():
        want = block(p, x, y, rng, ws)
    torch.cuda.synchronize()
    results, errors = [], []

    def work():
        try:
            with torch.no_grad():
                for _ in range(20):
                    results.append(block(p, x, y, rng, ws))
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors and len(results) == 40
    assert all(torch.equal(a, b) for r in results for a, b in zip(r, want))
    assert gct.query_status(ws)[0] == 0


def test_offsets_past_32_bits():
    """Rows that lie more than 2^31 elements, and 2^32 bytes, into their tensors."""
    rows, D = 2100, 1 << 20
    big = torch.empty(rows, D, dtype=torch.float16, device="cuda")
    view = big[:, 8:520]  # 512 columns, rows 2^20 elements apart
    g = torch.Generator(device="cuda").manual_seed(1)
    small = torch.randn(rows, 512, generator=g, device="cuda").half()
    view.copy_(small)
    rng, key = torch.tensor([5, 6], device="cuda"), (5, 6)
    out = torch.empty_like(small)
    gct.dropout_add(view, out, 0.5, rng)
    assert torch.equal(out, ref.drop(small.double(), 0.5, key).half())
    w = torch.eye(512, device="cuda").half()
    gct.matmul_act(view, w, out)
    assert torch.equal(out, small)
    target = big[:, 1024:1536]
    gct.matmul_act(small, w, target, residual=view)
    assert torch.equal(target, (small.float() * 2).half())
    n = torch.empty_like(small)
    gct.norm_join(view, target, n, x=view, pre="rms")
    want = torch.empty_like(small)
    gct.norm_join(small, None, want, x=small, pre="rms")
    assert torch.equal(n, want) and torch.equal(target, (small.float() * 2).half())
    gct.act_grad(view, None, target, p=0.5, rng=rng)
    assert torch.equal(target, ref.drop(small.double(), 0.5, key).half())
    odd = big[:, 3:516]
    odd.copy_(torch.randn(rows, 513, generator=g, device="cuda"))
    flat = odd.contiguous()
    n, want = torch.empty_like(flat), torch.empty_like(flat)
    gct.norm_join(odd, None, n, pre="layer")
    gct.norm_join(flat, None, want, pre="layer")
    assert torch.equal(n, want)
