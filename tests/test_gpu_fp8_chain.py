"""Chains of 8-bit float ops, each on what the one before wrote: kernels start
while their forerunner still runs, so a chain must give what the same calls
give one at a time, eagerly and from a graph, with other kernels in between."""
import pytest
import torch

import gemm_collective_tiles_gb300 as gct

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [512, 1000])
@pytest.mark.parametrize("M", [1, 7, 64, 300, 1500])
def test_chain_equals_its_calls_one_at_a_time(M, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    weights = []
    for _ in range(6):
        w = gct.empty_fp8(K, K, "tiles")
        gct.quantize_fp8(torch.randn(K, K, generator=g, device="cuda") * 0.05, *w, block="tiles")
        weights.append(w)
    x0 = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    codes, scales = gct.empty_fp8(M, K)
    outs = [torch.empty(M, K, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    grad = torch.empty(K, K, device="cuda")
    ws = [None, None]

    def chain(wait=lambda: None):
        x = x0
        for i, w in enumerate(weights):
            gct.quantize_fp8(x, codes, scales)
            wait()
            ws[0] = gct.matmul_fp8(codes, scales, *w, outs[i & 1], workspace=ws[0])
            wait()
            x = outs[i & 1]
            if i & 1:
                x.mul_(0.5)
                wait()
        ws[1] = gct.weight_grad_fp8(codes, scales, x, grad, workspace=ws[1])
        return x.clone(), grad.clone()

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = chain()
        for _ in range(5):
            got[0].zero_()
            got[1].zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for w in ws:
        assert gct.query_status(w)[0] == 0
