"""The MoE step's calls captured in graphs."""
import numpy as np
import pytest
import torch

import grouped_fp8_weight_gb300 as dg
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def routing(T, topk, G, seed):
    r = np.random.default_rng(seed)
    idx = r.integers(0, G, (T, topk))
    idx[r.random(idx.shape) < 0.1] = -1
    return idx


@pytest.mark.parametrize("T,topk,G,align", [(100, 4, 16, 16), (8192, 5, 64, 128), (70000, 2, 300, 1)])
def test_sort_in_a_graph(T, topk, G, align):
    """Replays, with other routings in the same memory, of few and of many pairs."""
    idx = torch.from_numpy(routing(T, topk, G, 0)).to(DEV, torch.int32)
    dg.dg_moe_sort(idx, G, align)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dg.dg_moe_sort(idx, G, align, with_src=True)
    for seed in (1, 2):
        host = routing(T, topk, G, seed)
        idx.copy_(torch.from_numpy(host))
        graph.replay()
        dg.dg_sync_check()
        c, r, p = oracle.moe_sort(host, G, align)
        for got, want in zip(out, (c, r, p, np.where(p >= 0, p // topk, -1))):
            assert np.array_equal(got.cpu().numpy(), want)


def test_a_layer_s_forward_calls_in_a_graph():
    """Sort, cast and dispatch, product and combine of more than 2^15 pairs in one
    graph give what the calls give one by one."""
    T, topk, G, C, N = 9000, 4, 8, 256, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, C, generator=g, device=DEV).bfloat16()
    weight = torch.rand(T, topk, generator=g, device=DEV)
    w = torch.randint(0, 120, (G, N, C), generator=g, device=DEV, dtype=torch.uint8)
    sw = torch.rand(G, 1, C // 128, generator=g, device=DEV) * 0.01
    idx = torch.from_numpy(routing(T, topk, G, 4)).to(DEV, torch.int32)

    def forward():
        counts, rows, pairs = dg.dg_moe_sort(idx, G, 16)
        R = pairs.shape[0]
        q = torch.empty(R, C, dtype=torch.uint8, device=DEV)
        s = torch.empty(R, C // 128, device=DEV)
        dg.dg_quant_rows_fp8(x, q, s, rows, pairs)
        ye = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
        dg.dg_m_grouped_fp8_linear(q, s, w, sw, ye, counts)
        y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        dg.dg_moe_combine(ye, rows, weight, y)
        return y

    forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward()
    for seed in (5, 6):
        idx.copy_(torch.from_numpy(routing(T, topk, G, seed)))
        x.copy_(torch.randn(T, C, generator=g, device=DEV))
        graph.replay()
        dg.dg_sync_check()
        got = out.clone()
        assert torch.equal(got, forward()) and bool(got.any())


def test_replays_of_an_optimizer_step_are_the_same_call_again():
    """Step number, rates and seed are the captured call's; the tensors and the
    gradient's scale are read when it runs."""
    def state():
        g = torch.Generator(device=DEV).manual_seed(8)
        n = 1000
        t = [torch.randn(n, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)]
        t += [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
        t += [torch.zeros(8, dtype=torch.uint8, device=DEV) for _ in range(2)]
        return t, dg.dg_adamw_plan(*[[a] for a in t])
    (a, pa), (b, pb) = state(), state()
    scale = torch.ones(1, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_adamw_step(pa, 2, 1e-2, grad_scale=scale, seed=9)
    for k in (1.0, 0.25, 3.0):
        scale.fill_(k)
        graph.replay()
        dg.dg_adamw_step(pb, 2, 1e-2, grad_scale=scale, seed=9)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x, y)
