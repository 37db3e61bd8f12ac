"""Low-rank adapters beside a projection (uw_lora_add) against float64.

Bound, per element, from the arithmetic (u = 2^-24).  V = A x: the MMA's
accumulation truncates, at most 2 u of the absolute sum per 16 of K, twice for
its inner alignment; no chain is longer than 512 of K (32 steps), then at most
8 + splits rounded additions: dV <= (128 + 8 + splits) u sum|a x|.  V times
scale is rounded once and kept as three BF16 parts up to u |V|.  The second
product accumulates 3 parts x ranks / 16 steps: 4 u each of sum|b v|; the sum
with y is rounded once."""
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


def make(t, k, n, count, rank, seed, ids=None, odd_ranks=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x = rnd(t, k).bfloat16()
    a = (rnd(count, rank, k) / math.sqrt(k)).bfloat16()
    b = (rnd(count, n, rank) * 0.2).bfloat16()
    y = rnd(t, n)
    ranks = torch.randint(0 if odd_ranks else rank, rank + 1, (count,), device="cuda", generator=g).int()
    scales = torch.rand(count, device="cuda", generator=g) + 0.5
    if ids is None:
        ids = torch.randint(-1, count + 1, (t,), device="cuda", generator=g).int()
    return x, a, b, ids, y, ranks, scales


def plain(x, a, b, ids, y, ranks, scales):
    """out, bound in float64."""
    out, bound = y.double().clone(), torch.zeros_like(y, dtype=torch.float64)
    k = x.shape[1]
    splits = max(16, -(-k // 4096))
    for i in range(a.shape[0]):
        r = a.shape[1] if ranks is None else int(ranks[i])
        s = 1.0 if scales is None else float(scales[i])
        rows = (ids == i).nonzero()[:, 0]
        if r == 0 or rows.numel() == 0:
            continue
        xs, as_, bs = x[rows].double(), a[i, :r].double(), b[i, :, :r].double()
        v = xs @ as_.T * s
        dv = (128 + 8 + splits + 2) * U * (xs.abs() @ as_.abs().T) * s
        out[rows] += v @ bs.T
        bound[rows] = dv @ bs.abs().T + 4 * 3 * (-(-r // 16)) * U * (v.abs() @ bs.abs().T)
    return out, bound + U * out.abs() + 1e-30


def check(got, want, bound):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), "error %g of the bound" % float((err / bound).max())


@pytest.mark.parametrize("t,k,n,count,rank", [
    (1, 64, 64, 1, 8), (1, 4096, 1024, 8, 64), (1, 4096, 14336, 3, 256), (3, 65536, 128, 2, 16), (31, 640, 2048, 1, 72), (32, 192, 320, 40, 8), (2, 128, 192, 3, 16), (17, 512, 320, 40, 24), (32, 4096, 512, 48, 16),
    (64, 1024, 256, 2, 8), (65, 1024, 256, 3, 32), (333, 2048, 448, 5, 40), (130, 14336, 128, 4, 64), (300, 192, 640, 1, 256),
    (1000, 256, 64, 1000, 8), (1024, 128, 128, 1024, 8), (1025, 128, 128, 7, 16), (900, 192, 64, 1, 24), (33, 4096, 512, 64, 16)])
def test_against_float64(uw, t, k, n, count, rank):
    x, a, b, ids, y, ranks, scales = make(t, k, n, count, rank, t + k + n)
    want, bound = plain(x, a, b, ids, y, ranks, scales)
    got = uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales)
    check(got, want, bound)
    rest = (ids < 0) | (ids >= count)
    assert torch.equal(got[rest], y[rest])
    # the same bits from given groups, in place, and again
    groups = uw.group_rows(ids, count)
    assert torch.equal(uw.lora_add(x, a, b, None, y, ranks=ranks, scales=scales, groups=groups), got)
    place = y.clone()
    assert uw.lora_add(x, a, b, ids, place, ranks=ranks, scales=scales, out=place) is place
    assert torch.equal(place, got)


@pytest.mark.parametrize("t", [5, 200])
def test_whole_slots_without_ranks_or_scales(uw, t):
    x, a, b, ids, y, _, _ = make(t, 256, 128, 4, 16, 3)
    want, bound = plain(x, a, b, ids, y, None, None)
    check(uw.lora_add(x.view(torch.int16), a.view(torch.int16), b.view(torch.int16), ids, y), want, bound)


@pytest.mark.parametrize("rank", [1, 2, 3, 4, 5, 7, 8, 15, 17, 23])
@pytest.mark.parametrize("t", [3, 100])
def test_what_a_slot_holds_beyond_its_rank_is_never_used(uw, rank, t):
    x, a, b, _, y, _, scales = make(t, 128, 128, 2, 24, rank)
    ids = torch.zeros(t, dtype=torch.int32, device="cuda")
    ranks = torch.full((2,), rank, dtype=torch.int32, device="cuda")
    want, bound = plain(x, a, b, ids, y, ranks, scales)
    a[:, rank:], b[:, :, rank:] = math.nan, math.inf
    check(uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales), want, bound)


def test_ranks_outside_the_slots_are_clamped(uw):
    x, a, b, ids, y, _, scales = make(40, 128, 128, 3, 16, 9)
    ranks = torch.tensor([-5, 99, 16], dtype=torch.int32, device="cuda")
    want, bound = plain(x, a, b, ids, y, ranks.clamp(0, 16), scales)
    check(uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales), want, bound)


@pytest.mark.parametrize("value", [-1, 0])
def test_no_row_has_an_adapter_and_all_have_one(uw, value):
    x, a, b, ids, y, ranks, scales = make(90, 192, 128, 2, 8, 4, ids=torch.full((90,), value, dtype=torch.int32, device="cuda"))
    want, bound = plain(x, a, b, ids, y, ranks, scales)
    got = uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales)
    check(got, want, bound)
    if value < 0:
        assert torch.equal(got, y)


def test_no_rows(uw):
    x, a, b, ids, y, ranks, scales = make(4, 64, 64, 2, 8, 1)
    assert uw.lora_add(x[:0], a, b, ids[:0], y[:0]).shape == (0, 64)


def test_strided_rows_and_columns_of_a_wider_buffer(uw):
    x, a, b, ids, y, ranks, scales = make(50, 128, 192, 3, 8, 8)
    want = uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales)
    wide_x = torch.randn(50, 320, device="cuda").bfloat16()
    wide_x[:, 64:192] = x
    both = torch.full((50, 448), math.nan, device="cuda")
    both[:, 4:196] = y
    got = uw.lora_add(wide_x[:, 64:192], a, b, ids, both[:, 4:196], ranks=ranks, scales=scales, out=both[:, 200:392])
    assert torch.equal(got, want) and torch.equal(both[:, 4:196], y)
    assert bool(both[:, :4].isnan().all() and both[:, 196:200].isnan().all() and both[:, 392:].isnan().all())


def test_infinite_activations_reach_their_row_only(uw):
    x, a, b, _, y, _, scales = make(20, 128, 64, 1, 8, 12)
    ids = torch.zeros(20, dtype=torch.int32, device="cuda")
    want = uw.lora_add(x, a, b, ids, y)
    x[7, 3], x[9, 5] = math.inf, math.nan
    got = uw.lora_add(x, a, b, ids, y)
    keep = [i for i in range(20) if i not in (7, 9)]
    assert torch.equal(got[keep], want[keep])
    assert not bool(got[7].isfinite().any()) and bool(got[9].isnan().all())


@pytest.mark.parametrize("t", [3, 100])
def test_inner_products_near_the_largest_float(uw, t):
    """A x just above the largest BF16, which rounding to BF16 would make infinite."""
    x, a, b, _, y, _, _ = make(t, 128, 64, 1, 8, 13)
    ids = torch.zeros(t, dtype=torch.int32, device="cuda")
    top = torch.finfo(torch.bfloat16).max                     # (2 - 2^-7) 2^127
    x.zero_(), a.zero_(), y.zero_(), b.zero_()
    x[:, 0], x[:, 1] = top, 2.0 ** 119                        # the sum is half way to 2^128
    a[0, 0, :2] = 1.0
    b[0, :, 0] = 2.0 ** -100
    got = uw.lora_add(x, a, b, ids, y)
    want = (top + 2.0 ** 119) * 2.0 ** -100                   # every sum and piece is exact
    assert bool((got.double() == want).all())


def test_another_stream_and_a_replayed_graph(uw):
    x, a, b, ids, y, ranks, scales = make(100, 256, 192, 6, 16, 77)
    want = uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(y)
    ws = uw.new_workspace(uw.lora_workspace_size(100, 256, 192, 6, 16), "cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        uw.lora_add(x, a, b, ids, y, ranks=ranks, scales=scales, out=out, ws=ws)
    for seed in (1, 2):
        x2, _, _, ids2, y2, _, _ = make(100, 256, 192, 6, 16, seed)
        want = uw.lora_add(x2, a, b, ids2, y2, ranks=ranks, scales=scales)
        x.copy_(x2), ids.copy_(ids2), y.copy_(y2)
        ws.fill_(0xFF)       # its contents do not matter
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_beside_a_compressed_projection(uw):
    """The projection's matmul, then the adapters in place on its result, one
    call after the other on a stream."""
    from decode_gemm_exponent_b200 import synth
    n, k, m = 512, 1024, 12
    mat = uw.Matrix(uw.encode(synth.weights_bf16(n, k, 0.02, 0.002, 1.0, seed=5)))
    x, a, b, ids, _, ranks, scales = make(m, k, n, 5, 16, 31)
    plan = uw.make_plan(uw.PIPE_DIRECT_PALETTE, uw.KERNEL_MMA, 4)
    groups = uw.group_rows(ids, 5)
    y = torch.empty(m, n, device="cuda")
    ws = uw.new_workspace(uw.lora_workspace_size(m, k, n, 5, 16), "cuda")     # None: few rows need none
    base = mat.matmul(x.view(torch.int16), plan)
    want, bound = plain(x, a, b, ids, base, ranks, scales)
    for _ in range(20):
        mat.matmul(x.view(torch.int16), plan, y=y)
        uw.lora_add(x, a, b, None, y, ranks=ranks, scales=scales, groups=groups, out=y, ws=ws)
    check(y, want, bound)
    assert mat.device_status() == 0


def test_refusals(uw):
    x, a, b, ids, y, ranks, scales = make(48, 128, 128, 2, 16, 2)
    for args, kw in (((x.float(), a, b, ids, y), {}), ((x, a[:, :, :64], b, ids, y), {}), ((x, a, b[:1], ids, y), {}),
                     ((x, a, b, ids.long(), y), {}), ((x, a, b, ids[:4], y), {}), ((x, a, b, ids, y.double()), {}),
                     ((x, a, b, ids, y), dict(ranks=ranks.long())), ((x, a, b, ids, y), dict(scales=scales.cpu())),
                     ((x, a, b, ids, y.T.contiguous().T), {}), ((x, a, b, ids, y), dict(out=y[:4])),
                     ((x, a, b, None, y), {}), ((x, a, b, ids, y), dict(ws=torch.empty(1 << 20, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            uw.lora_add(*args, **kw)
    with pytest.raises(uw.UwError) as e:       # ranks in eights
        uw.lora_add(x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), ids, y)
    assert e.value.status == uw.ERR_INVALID_ARG
    with pytest.raises(uw.UwError) as e:
        uw.lora_add(x[:, :96].contiguous(), a[:, :, :96].contiguous(), b, ids, y)
    assert e.value.status == uw.ERR_UNSUPPORTED_SHAPE
    with pytest.raises(uw.UwError) as e:
        uw.lora_add(x, a, b, ids, y, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == uw.ERR_WORKSPACE
    wide = torch.zeros(48, 256, device="cuda")
    with pytest.raises(uw.UwError):            # result overlaps the input
        uw.lora_add(x, a, b, ids, wide[:, :128], out=wide[:, 64:192])
