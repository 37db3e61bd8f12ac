"""Products of routed rows with their experts' weights, with the token counts on
the device (uw_expert_matmul, uw_expert_gate_up, uw_expert_combine), against
float64 with bounds from the arithmetic (u = 2^-24).

FP32 sums: the MMA truncates when it accumulates, at most 4 u of the absolute
sum per 16 of K; the chains are 512 of K long in the tcgen05 kernel (32 steps)
and K / (2 warps) in the warp-MMA kernel, their sums are rounded additions:
error <= (4 steps + sums) u sum|w x|.  The gated activation: the error of g and
up through h = silu(g) up, |silu'| <= 1.1, a few units for exp and the division
((8 + 2 |g|) u: the exponent's argument is rounded), and one rounding to BF16, 2^-8 of half a step: eps / 2."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def uw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from decode_gemm_exponent_b200 import uw as U_
    return U_


def routed(uw, t, e, top_k, seed, drop=0.0, crowd=None):
    """A Routing of distinct random experts per token; `drop` of the slots have none;
    `crowd`: an expert that every token goes to."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand(t, e, device="cuda", generator=g).argsort(1)[:, :top_k].int()
    if crowd is not None:
        hit = (ids == crowd).any(1)
        ids[~hit, 0] = crowd
    ids[torch.rand(t, top_k, device="cuda", generator=g) < drop] = -1
    p = torch.rand(t, top_k, device="cuda", generator=g)
    r = uw.group_rows(ids.contiguous(), e)
    return uw.Routing(ids, p, r.offsets, r.order, r.slot)


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()


def plans(uw):
    P = uw.make_expert_plan
    return [P(uw.KERNEL_MMA, 4), P(uw.KERNEL_MMA, 1, width=1), P(uw.KERNEL_TC, 128, 128), P(uw.KERNEL_TC, 256, 32),
            P(uw.KERNEL_TC, 256, 64, sort=1), P(uw.KERNEL_TC, 128, 128, sort=1), P(uw.KERNEL_TC, 256, 256, sort=1), None]


def product(x, w, routing, gather, k_per_chain):
    """y, bound in float64, [places, n]; rows of no expert are NaN, 0."""
    places = routing.order.numel()
    y = torch.full((places, w.shape[1]), math.nan, device="cuda", dtype=torch.float64)
    bound = torch.zeros_like(y)
    per_row = places // x.shape[0] if gather else 1
    at = routing.offsets.tolist()
    units = 4 * (k_per_chain / 16 + 1) + w.shape[2] / k_per_chain + 8
    for i in range(w.shape[0]):
        j = torch.arange(at[i], at[i + 1], device="cuda")
        rows = x[routing.order[j].long() // per_row if gather else j].double()
        y[j] = rows @ w[i].double().T
        bound[j] = units * U * (rows.abs() @ w[i].double().abs().T)
    return y, bound


def chain(plan, k):
    return max(512, k if plan is None or plan.kernel == 3 else 0)


def check(got, want, bound):
    live = ~want.isnan()
    err = (got.double() - want).abs()[live]
    assert bool((err <= bound[live] + 1e-30).all()), float((err / (bound[live] + 1e-30)).max())


SHAPES = [(1, 4, 64, 64, 2), (3, 8, 192, 128, 3), (40, 16, 320, 256, 4), (33, 2, 64, 576, 1), (200, 5, 448, 192, 2),
          (700, 8, 256, 1024, 2), (300, 130, 64, 128, 8), (900, 2, 192, 640, 1), (520, 1, 320, 2112, 1)]


@pytest.mark.parametrize("which", range(8))
@pytest.mark.parametrize("t,e,n,k,top_k", SHAPES)
def test_matmul(uw, which, t, e, n, k, top_k):
    plan = plans(uw)[which]
    r = routed(uw, t, e, top_k, t + e)
    w, x = normal(n, e, n, k, std=0.05), normal(k, t, k)
    want, bound = product(x, w, r, True, chain(plan, k))
    check(uw.expert_matmul(x, w, r, gather=True, plan=plan), want, bound)
    xs = x[r.order.long() // top_k].contiguous()
    check(uw.expert_matmul(xs, w, r, plan=plan), want, bound)


@pytest.mark.parametrize("which", range(8))
@pytest.mark.parametrize("t,e,n,k,top_k", SHAPES)
def test_gate_up(uw, which, t, e, n, k, top_k):
    plan = plans(uw)[which]
    r = routed(uw, t, e, top_k, t + e)
    w, x = normal(n, e, 2 * n, k, std=0.05), normal(k, t, k)
    g, dg = product(x, w[:, :n], r, True, max(512, k))
    u, du = product(x, w[:, n:], r, True, max(512, k))
    s = g * torch.sigmoid(g)
    want = s * u
    bound = 1.1 * dg * (u.abs() + du) + s.abs() * du + (8 + 2 * g.abs()) * U * want.abs()
    bound = bound + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + bound) + 1e-38
    got = uw.expert_gate_up(x, w[:, :n], w[:, n:], r, plan=plan)
    check(got, want, bound)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    again = uw.expert_gate_up(x.view(torch.int16), w[:, :n], w[:, n:], r, plan=plan, status=status)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16)) and int(status) == 0
    if plan is not None and plan.rows == 256:             # gathered rows of x: the same products
        plan = uw.make_expert_plan(uw.KERNEL_TC, 256, 256)
        again = uw.expert_gate_up(x, w[:, :n], w[:, n:], r, plan=plan, status=status)
        check(again, want, bound)
        assert int(status) == 0


@pytest.mark.parametrize("k", [64, 832])
def test_uneven_experts_over_many_tiles(uw, k):
    """From one row to several tiles per expert, more tiles than SMs, so that every
    stage and queue of the kernels is used again with another number of rows."""
    g = torch.Generator().manual_seed(k)
    counts = torch.cat([torch.randint(1, 40, (60,), generator=g), torch.randint(40, 700, (30,), generator=g)])
    counts = counts[torch.randperm(90, generator=g)]
    ids = torch.repeat_interleave(torch.arange(90), counts)
    ids = ids[torch.randperm(len(ids), generator=g)].int().cuda()[:, None].contiguous()
    r = uw.group_rows(ids, 90)
    w, x = normal(1, 90, 2 * 192, k, std=0.05), normal(2, len(ids), k)
    gate, dg = product(x, w[:, :192], r, True, max(512, k))
    up, du = product(x, w[:, 192:], r, True, max(512, k))
    s = gate * torch.sigmoid(gate)
    want = s * up
    bound = 1.1 * dg * (up.abs() + du) + s.abs() * du + (8 + 2 * gate.abs()) * U * want.abs()
    bound = bound + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + bound) + 1e-38
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for rows in (64, 256):
        plan = uw.make_expert_plan(uw.KERNEL_TC, 256, rows)
        for _ in range(3):
            check(uw.expert_gate_up(x, w[:, :192], w[:, 192:], r, plan=plan, status=status), want, bound)
    y, dy = product(x, w, r, True, 512)
    xs = x[r.order.long()].contiguous()
    check(uw.expert_matmul(xs, w, r, plan=uw.make_expert_plan(uw.KERNEL_TC, 256, 256), status=status), y, dy)
    assert int(status) == 0


@pytest.mark.parametrize("which", range(8))
def test_crowded_and_empty_experts_and_dropped_slots(uw, which):
    plan = plans(uw)[which]
    t, e, n, k = 150, 40, 128, 192
    r = routed(uw, t, e, 2, 7, drop=0.4, crowd=11)
    w, x = normal(1, e, n, k, std=0.1), normal(2, t, k)
    want, bound = product(x, w, r, True, chain(plan, k))
    y = torch.full((2 * t, n), 7.0, device="cuda")
    uw.expert_matmul(x, w, r, gather=True, plan=plan, out=y)
    check(y, want, bound)
    last = int(r.offsets[-1])
    assert last < 2 * t and bool((y[last:] == 7.0).all())      # rows behind the last expert are left as they were


@pytest.mark.parametrize("which", range(8))
def test_no_slot_has_an_expert_and_no_tokens(uw, which):
    plan = plans(uw)[which]
    r = routed(uw, 20, 6, 2, 3, drop=1.1)
    y = torch.full((40, 64), 3.0, device="cuda")
    w = normal(1, 6, 64, 64)
    uw.expert_matmul(normal(2, 20, 64), w, r, gather=True, plan=plan, out=y)
    assert bool((y == 3.0).all())
    none = uw.route_experts(torch.empty(0, 6, device="cuda"), 2)
    assert uw.expert_matmul(normal(2, 20, 64)[:0], w, none, gather=True, plan=plan).shape == (0, 64)
    assert uw.expert_combine(torch.empty(0, 64, device="cuda"), none).shape == (0, 64)


@pytest.mark.parametrize("which", [0, 2, 3, 4, 6])
def test_strides_and_guard_rows(uw, which):
    plan = plans(uw)[which]
    t, e, n, k = 90, 3, 128, 128
    r = routed(uw, t, e, 1, 5)
    store = normal(4, e, n + 64, k)
    x = normal(6, t, 320)[:, 64:192]
    want = uw.expert_matmul(x.contiguous(), store[:, 64:].contiguous(), r, gather=True, plan=plan)
    y = torch.full((t + 2, n + 8), math.inf, device="cuda")
    uw.expert_matmul(x, store[:, 64:], r, gather=True, plan=plan, out=y[1:-1, 4:-4])
    assert torch.equal(y[1:-1, 4:-4], want)
    y[1:-1, 4:-4] = math.inf
    assert bool(y.isinf().all())


@pytest.mark.parametrize("rows", [64, 256])
def test_a_short_limit_is_long_enough_for_copies_to_land(uw, rows):
    r = routed(uw, 300, 4, 2, 3)
    x, w = normal(1, 300, 512), normal(2, 4, 256, 512)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = uw.expert_gate_up(x, w[:, :128], w[:, 128:], r, plan=uw.make_expert_plan(uw.KERNEL_TC, 256, rows))
    got = uw.expert_gate_up(x, w[:, :128], w[:, 128:], r, plan=uw.make_expert_plan(uw.KERNEL_TC, 256, rows, timeout_ns=1),
                            status=status)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and int(status) == 0


def test_nan_rows_stay_with_their_tokens(uw):
    r = routed(uw, 60, 2, 1, 9)
    w = normal(4, 2, 128, 128)
    x = normal(6, 60, 128)
    for plan in plans(uw):
        want = uw.expert_matmul(x, w, r, gather=True, plan=plan)
        bad = x.clone()
        bad[13] = math.nan
        got = uw.expert_matmul(bad, w, r, gather=True, plan=plan)
        at = int(r.slot[13])
        assert bool(got[at].isnan().all())
        keep = torch.arange(60, device="cuda") != at
        assert torch.equal(got[keep], want[keep])
    for plan in plans(uw) + [uw.make_expert_plan(uw.KERNEL_TC, 256, 256)]:
        want = uw.expert_gate_up(x, w, w, r, plan=plan)
        got = uw.expert_gate_up(bad, w, w, r, plan=plan)
        assert bool(got[at].isnan().all()) and torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("kernel,bn,kw", [(3, 1, dict(width=1)), (3, 4, dict(width=2)), (3, 8, {}), (3, 3, dict(width=1)),
                                          (2, 128, dict(rows=32)), (2, 256, dict(rows=128, sort=1)), (2, 256, dict(rows=256, sort=1))])
@pytest.mark.parametrize("k", [256, 1152])
def test_compressed_equals_plain_bit_for_bit(uw, kernel, bn, kw, k):
    from decode_gemm_exponent_b200 import synth
    t, e, n = 23, 6, 192
    plan = uw.make_expert_plan(kernel, bn, **kw)
    ws = [[synth.weights_bf16(n, k, 0.01 + 0.004 * i, 0.004, 1.0, seed=100 * j + i) for i in range(e)] for j in range(2)]
    sets = [uw.ExpertSet([uw.Matrix(uw.encode(w)) for w in row]) for row in ws]
    plain = [torch.from_numpy(np.stack(row).view(np.int16)).cuda() for row in ws]
    r = routed(uw, t, e, 2, 5, drop=0.1, crowd=2)
    x = normal(8, t, k)
    last = int(r.offsets[-1])
    a = uw.expert_matmul(x, sets[0], r, gather=True, plan=plan)[:last]
    b = uw.expert_matmul(x, plain[0], r, gather=True, plan=plan)[:last]
    assert torch.equal(a, b)
    a = uw.expert_gate_up(x, sets[0], sets[1], r, plan=plan)[:last]
    b = uw.expert_gate_up(x, plain[0], plain[1], r, plan=plan)[:last]
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # and the default plan runs on the set
    uw.expert_matmul(x, sets[0], r, gather=True)


@pytest.mark.parametrize("t,top_k,n", [(1, 1, 4), (5, 3, 64), (100, 8, 1028), (3, 32, 2048)])
@pytest.mark.parametrize("based", [False, True])
def test_combine(uw, t, top_k, n, based):
    r = routed(uw, t, 64, top_k, t + n, drop=0.2)
    y = torch.randn(t * top_k, n, device="cuda")
    y[int(r.offsets[-1]):] = math.nan                     # rows of no expert are never read into a sum
    base = torch.randn(t, n, device="cuda") if based else None
    live = (r.slot >= 0)[:, :, None]
    rows = torch.where(live, y[r.slot.clamp(min=0).long()].double(), 0.0) * r.weights[:, :, None].double()
    want = rows.sum(1) + (base.double() if based else 0.0)
    bound = (top_k + 1) * U * (rows.abs().sum(1) + (base.abs().double() if based else 0.0)) + 1e-30
    got = uw.expert_combine(y, r, base=base)
    assert bool(((got.double() - want).abs() <= bound).all())
    if based:
        place = base.clone()
        assert torch.equal(uw.expert_combine(y, r, base=place, out=place), got)


@pytest.mark.parametrize("t", [1, 6, 500, 1500])
@pytest.mark.parametrize("compressed", [False, True])
def test_a_layer_from_the_logits_to_the_output(uw, t, compressed):
    """Router, experts and join in one run, captured into a graph and replayed
    with other tokens; padding tokens come out zero."""
    from decode_gemm_exponent_b200 import synth
    e, n, k, top_k = 12, 128, 256, 3
    ws = [[synth.weights_bf16(*s, 0.04, 0.0, 1.0, seed=31 * j + i) for i in range(e)] for j, s in enumerate([(n, k), (n, k), (k, n)])]
    plain = [torch.from_numpy(np.stack(row).view(np.int16)).cuda().view(torch.bfloat16) for row in ws]
    gate, up, down = [uw.ExpertSet([uw.Matrix(uw.encode(w)) for w in row]) for row in ws] if compressed else plain
    x, logits = normal(3, t, k), torch.randn(t, e, device="cuda")
    out = torch.empty(t, k, device="cuda")
    r = uw.route_experts(logits, top_k, score="sigmoid", scale=1.5)
    h = torch.zeros(t * top_k, n, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(t * top_k, k, device="cuda")

    def layer():
        uw.route_experts(logits, top_k, score="sigmoid", scale=1.5, out=r)
        uw.expert_gate_up(x, gate, up, r, out=h)
        uw.expert_matmul(h, down, r, out=y)
        uw.expert_combine(y, r, out=out)

    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (1, 2):
        x.copy_(normal(50 + seed, t, k))
        logits.copy_(torch.randn(t, e, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        if t > 1:
            logits[t // 2:] = -math.inf
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for s in range(top_k):
            for i in range(e):
                rows = (r.ids[:, s] == i).nonzero()[:, 0]
                xs = x[rows].double()
                a, b = xs @ plain[0][i].double().T, xs @ plain[1][i].double().T
                hh = a * torch.sigmoid(a) * b
                want[rows] += r.weights[rows, s, None].double() * (hh @ plain[2][i].double().T)
                size[rows] += r.weights[rows, s, None].double() * (hh.abs() @ plain[2][i].double().abs().T)
        # h is rounded to BF16 once (eps / 2), all else is 32 bits: far below 1e-4 of the absolute sum
        assert bool(((out.double() - want).abs() <= (torch.finfo(torch.bfloat16).eps / 2 + 1e-4) * size + 1e-30).all())
        if t > 1:
            assert bool((out[t // 2:] == 0).all())


def test_refusals(uw):
    r = routed(uw, 8, 4, 2, 1)
    x, w = normal(1, 8, 128), normal(2, 4, 64, 128)
    for kw in (dict(x=x.float()), dict(x=x[:5]), dict(x=x[:, :64].contiguous()), dict(w=w[:3]), dict(w=w.float()),
               dict(w=w.transpose(1, 2)), dict(w=w[0]), dict(x=x.cpu()), dict(out=torch.empty(16, 32, device="cuda")),
               dict(out=torch.empty(16, 64, device="cuda", dtype=torch.bfloat16)), dict(gather=False)):
        full = dict(x=x, w=w, gather=True)
        full.update(kw)
        with pytest.raises(ValueError):
            uw.expert_matmul(full.pop("x"), full.pop("w"), r, **full)
    with pytest.raises(ValueError):
        uw.expert_gate_up(x, w, w[:, :32], r)
    P = uw.make_expert_plan
    for plan in (P(uw.KERNEL_FMA, 1, 0), P(uw.KERNEL_TC, 64), P(uw.KERNEL_TC, 128, 16), P(uw.KERNEL_TC, 128, width=1),
                 P(uw.KERNEL_MMA, 9), P(uw.KERNEL_MMA, 4, 32), P(uw.KERNEL_MMA, 4, sort=1)):
        with pytest.raises(uw.UwError) as err:
            uw.expert_matmul(x, w, r, gather=True, plan=plan)
        assert err.value.status == uw.ERR_INVALID_ARG
    with pytest.raises(uw.UwError) as err:     # 256 places per tile take rows in expert order
        uw.expert_matmul(x, w, r, gather=True, plan=P(uw.KERNEL_TC, 256, 256))
    assert err.value.status == uw.ERR_INVALID_ARG
    from decode_gemm_exponent_b200 import synth
    mats = [uw.Matrix(uw.encode(synth.weights_bf16(64, 128, 0.02, 0.0, 1.0, seed=i))) for i in range(4)]
    s = uw.ExpertSet(mats)
    with pytest.raises(uw.UwError) as err:     # rebuilt weights need a workspace
        uw.expert_matmul(x, s, r, gather=True, plan=P(uw.KERNEL_TC, 128), ws=torch.empty(512, device="cuda").byte())
    assert err.value.status == uw.ERR_WORKSPACE
    with pytest.raises(uw.UwError) as err:     # the sorted rows need a workspace
        uw.expert_matmul(x, w, r, gather=True, plan=P(uw.KERNEL_TC, 128, sort=1), ws=torch.empty(512, device="cuda").byte())
    assert err.value.status == uw.ERR_WORKSPACE
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):        # a workspace that the kernel could not use
            uw.expert_matmul(x, w, r, gather=True, plan=P(uw.KERNEL_TC, 128, sort=1), ws=ws)
    with pytest.raises(uw.UwError):            # one form for both
        uw.expert_gate_up(x, s, w, r)
    other = uw.Matrix(uw.encode(synth.weights_bf16(128, 128, 0.02, 0.0, 1.0, seed=9)))
    with pytest.raises(uw.UwError):
        uw.ExpertSet(mats[:3] + [other])
    huff = uw.Matrix(uw.encode(synth.weights_bf16(64, 128, 0.02, 0.0, 1.0, seed=9), uw.EMIT_HUFFMAN))
    with pytest.raises(uw.UwError):
        uw.ExpertSet([huff])
