"""The operators around the matmuls where element offsets pass 32 bits, with two
calls in flight at once, and with many tokens: each against the same call on a
part of the rows, or against plain arithmetic on a sample of them."""
import math

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.fixture(scope="module")
def uw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    from decode_gemm_exponent_b200 import uw as U
    yield U
    torch.cuda.empty_cache()


def test_route_beyond_32_bits_of_logits(uw):
    t, e, top_k = (1 << 31) // 256 + 5000, 256, 8
    logits = torch.empty(t, e, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, t, 1 << 20):
        logits[i:i + (1 << 20)].normal_(generator=g)
    r = uw.route_experts(logits, top_k)
    tail = uw.route_experts(logits[-3000:].contiguous(), top_k)
    assert torch.equal(r.ids[-3000:], tail.ids) and torch.equal(r.weights[-3000:], tail.weights)
    assert torch.equal(r.ids[:2000], uw.route_experts(logits[:2000].contiguous(), top_k).ids)
    counts = torch.bincount(r.ids.reshape(-1), minlength=e)
    assert torch.equal(r.offsets[1:].long(), torch.cumsum(counts, 0)) and int(r.offsets[0]) == 0
    # the order is a stable sort: places of one expert rise, and slot inverts it
    expert = r.ids.reshape(-1)[r.order.long()]
    same = expert[1:] == expert[:-1]
    assert bool((expert[1:] >= expert[:-1]).all()) and bool((r.order[1:] > r.order[:-1])[same].all())
    assert torch.equal(r.slot.reshape(-1)[r.order.long()], torch.arange(t * top_k, device="cuda", dtype=torch.int32))


@pytest.mark.parametrize("kernel,bn,rows", [(2, 256, 128), (2, 128, 64), (2, 256, 256), (3, 4, 0)])
def test_expert_products_beyond_32_bits_of_outputs(uw, kernel, bn, rows):
    e, n, k = 3, 4096, 64
    t = (1 << 31) // n + 3000
    if kernel == 3:
        t, n = (1 << 31) // 16384 + 300, 16384          # one pass per 16 rows: fewer, wider rows
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, k, device="cuda", generator=g).bfloat16()
    w = torch.randn(e, n, k, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, e, (t, 1), device="cuda", generator=g).int()
    r = uw.group_rows(ids, e)
    routing = uw.Routing(ids, torch.full((t, 1), 0.5, device="cuda"), r.offsets, r.order, r.slot)
    y = uw.expert_matmul(x, w, routing, gather=True, plan=uw.make_expert_plan(kernel, bn, rows, sort=int(rows == 256)))
    out = uw.expert_combine(y, routing)
    for i in list(range(0, 40)) + list(range(t - 40, t)):
        want = w[int(ids[i, 0])].double() @ x[i].double()
        size = w[int(ids[i, 0])].double().abs() @ x[i].double().abs()
        # 64 of K: 4 truncations and a few roundings of the absolute sum
        assert bool(((y[int(r.slot[i, 0])].double() - want).abs() <= 32 * 2.0 ** -24 * size).all())
        assert torch.equal(out[i], y[int(r.slot[i, 0])] * 0.5)


def test_adapters_beyond_32_bits_of_outputs(uw):
    n, k, a, rank = 4096, 64, 3, 8
    t = (1 << 31) // n + 3000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(t, k, device="cuda", generator=g).bfloat16()
    A = torch.randn(a, rank, k, device="cuda", generator=g).bfloat16()
    B = torch.randn(a, n, rank, device="cuda", generator=g).bfloat16()
    y = torch.empty(t, n, device="cuda")
    for i in range(0, t, 1 << 16):
        y[i:i + (1 << 16)].normal_(generator=g)
    ids = torch.randint(-1, a, (t,), device="cuda", generator=g).int()
    out = uw.lora_add(x, A, B, ids, y)
    rows = torch.cat([torch.arange(0, 50), torch.arange(t - 50, t)]).cuda()
    for i in rows.tolist():
        j = int(ids[i])
        want = y[i].double()
        size = want.abs()
        if j >= 0:
            v = A[j].double() @ x[i].double()
            want = want + B[j].double() @ v
            size = size + B[j].double().abs() @ (A[j].double().abs() @ x[i].double().abs())
        assert bool(((out[i].double() - want).abs() <= 64 * 2.0 ** -24 * size).all())
    rest = (ids < 0).nonzero()[-200:, 0]
    assert torch.equal(out[rest], y[rest])


def test_two_calls_at_once(uw):
    """Calls on two streams with their own outputs and workspaces do not disturb
    each other."""
    g = torch.Generator(device="cuda").manual_seed(4)
    e, n, k, top_k = 16, 256, 512, 4
    w = torch.randn(e, 2 * n, k, device="cuda", generator=g).bfloat16()
    down = torch.randn(e, k, n, device="cuda", generator=g).bfloat16()
    A = torch.randn(6, 16, k, device="cuda", generator=g).bfloat16()
    B = torch.randn(6, k, 16, device="cuda", generator=g).bfloat16()
    data = []
    for t in (700, 900):
        data.append((torch.randn(t, k, device="cuda", generator=g).bfloat16(), torch.randn(t, e, device="cuda", generator=g),
                     torch.randint(-1, 6, (t,), device="cuda", generator=g).int(), torch.randn(t, k, device="cuda", generator=g)))

    def layer(d, stream=None):
        x, logits, ids, base = d
        r = uw.route_experts(logits, top_k, score="sigmoid", n_groups=4, top_groups=2, stream=stream)
        h = uw.expert_gate_up(x, w[:, :n], w[:, n:], r, stream=stream)
        y = uw.expert_matmul(h, down, r, stream=stream)
        out = uw.expert_combine(y, r, base=base, stream=stream)
        return uw.lora_add(x, A, B, ids, out, stream=stream)

    want = [layer(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(10):
        got = [layer(d, s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_replayed_in_turn(uw):
    """Two captured graphs of the whole path, each with its own outputs."""
    g = torch.Generator(device="cuda").manual_seed(5)
    e, n, k = 8, 128, 256
    w = torch.randn(e, 2 * n, k, device="cuda", generator=g).bfloat16()
    graphs = []
    for t in (40, 600):
        x = torch.randn(t, k, device="cuda", generator=g).bfloat16()
        logits = torch.randn(t, e, device="cuda", generator=g)
        r = uw.route_experts(logits, 2)
        h = uw.expert_gate_up(x, w[:, :n], w[:, n:], r)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            uw.route_experts(logits, 2, out=r)
            uw.expert_gate_up(x, w[:, :n], w[:, n:], r, out=h)
        graphs.append((graph, x, logits, r, h))
    for seed in range(3):
        for graph, x, logits, r, h in graphs:
            gen = torch.Generator(device="cuda").manual_seed(100 + seed)
            logits.copy_(torch.randn(logits.shape, device="cuda", generator=gen))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, logits, r, h in graphs:
            fresh = uw.route_experts(logits.clone(), 2)
            assert torch.equal(fresh.order, r.order) and torch.equal(fresh.offsets, r.offsets)
            assert torch.equal(uw.expert_gate_up(x, w[:, :n], w[:, n:], fresh).view(torch.int16), h.view(torch.int16))
