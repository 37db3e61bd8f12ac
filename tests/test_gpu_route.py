"""Routing of tokens to experts and grouping of rows (uw_route_experts,
uw_group_rows) against a plain float64 implementation, one token at a time.

Ids, offsets, order and slots are whole numbers and must be equal.  Weights are
float32: the final rounding is 2^-24 of the value, the exponentials of the
64-bit path add nothing to that, and the 32-bit sum of the softmax without a
bias adds at most 4 (expf, 2 units) + 7 (argument rounding, 2^-24 times the mean
distance to the maximum, below ln 1024) + experts / 32 + 5 (additions of positive
terms) further units of 2^-24."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def uw():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from decode_gemm_exponent_b200 import uw as U
    return U


def plain_route(logits, top_k, score, bias, n_groups, top_groups, group_score, renormalize, scale):
    """ids int [t, top_k], weights float64 [t, top_k]; logits float64, bias float64 or None."""
    t, e = logits.shape
    ids = np.full((t, top_k), -1, np.int64)
    weights = np.zeros((t, top_k))
    size = e // n_groups
    for i in range(t):
        l = np.array([min(v, float(np.finfo(np.float32).max)) if v > -math.inf else -math.inf for v in logits[i]])
        alive = l > -math.inf
        s = np.zeros(e)
        if alive.any():
            if score == "softmax":
                s[alive] = np.exp(l[alive] - l[alive].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[alive] = 1.0 / (1.0 + np.exp(-l[alive]))
        value = s + (0.0 if bias is None else bias)
        alive &= value > -math.inf
        rank = l if bias is None else value
        allowed = set(range(e))
        if n_groups > 1:
            v = []
            for g in range(n_groups):
                mine = [j for j in range(g * size, g * size + size) if alive[j]]
                if not mine:
                    v.append(-math.inf)
                elif group_score == "max":
                    v.append(max(rank[j] for j in mine))
                else:
                    v.append(sum(sorted((value[j] for j in mine), reverse=True)[:2]))
            best = sorted(range(n_groups), key=lambda g: (-v[g], g))[:top_groups]
            allowed = {j for g in best for j in range(g * size, g * size + size)}
        order = sorted((j for j in allowed if alive[j]), key=lambda j: (-rank[j], j))[:top_k]
        ids[i, :len(order)] = order
        weights[i, :len(order)] = s[order]
    if renormalize:
        weights /= weights.sum(1, keepdims=True) + 1e-20
    return ids, weights * scale


def plain_group(ids, groups):
    flat = ids.reshape(-1)
    key = np.where((flat < 0) | (flat >= groups), groups, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(groups + 1))
    slot = np.empty(flat.size, np.int64)
    slot[order] = np.arange(flat.size)
    return offsets, order, np.where(key < groups, slot, -1).reshape(ids.shape)


def check_group(r, ids, groups):
    offsets, order, slot = plain_group(ids, groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.slot.cpu().numpy(), slot)


def check_route(uw, logits, top_k, bias=None, **kw):
    full = dict(score="softmax", n_groups=1, top_groups=1, group_score="max", renormalize=True, scale=1.0)
    full.update(kw)
    r = uw.route_experts(logits, top_k, bias=bias, **full)
    ids, weights = plain_route(logits.double().cpu().numpy(), top_k, full["score"],
                               None if bias is None else bias.double().cpu().numpy(), full["n_groups"],
                               full["top_groups"], full["group_score"], full["renormalize"],
                               float(np.float32(full["scale"])))
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = r.weights.cpu().numpy().astype(np.float64)
    units = 1 + 4 + 7 + logits.shape[1] / 32 + 5
    assert (np.abs(got - weights) <= units * 2.0 ** -24 * np.abs(weights) + 1e-45).all()
    check_group(r, ids, logits.shape[1])
    return r


def random_logits(t, e, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(t, e, generator=g) * 1.5
    return l.to(dtype).cuda()


@pytest.mark.parametrize("t", [1, 3, 64, 65, 200, 1500])
@pytest.mark.parametrize("e,top_k", [(1, 1), (8, 2), (60, 4), (128, 8), (256, 8), (513, 32), (1024, 10)])
def test_softmax(uw, t, e, top_k):
    if t * e > 500_000:
        t = 300
    check_route(uw, random_logits(t, e, 10 * t + e), top_k, renormalize=(t % 2 == 0))


@pytest.mark.parametrize("t,e,top_k,n_groups,top_groups", [
    (5, 16, 4, 4, 2), (70, 64, 6, 8, 3), (300, 256, 8, 8, 4), (33, 160, 6, 8, 3), (9, 30, 2, 30, 5), (20, 1024, 16, 32, 1),
    (12, 96, 3, 3, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(uw, t, e, top_k, n_groups, top_groups, score, group_score, biased):
    bias = torch.randn(e, generator=torch.Generator().manual_seed(e)).mul(0.05).cuda() if biased else None
    check_route(uw, random_logits(t, e, t + e), top_k, bias, score=score, n_groups=n_groups, top_groups=top_groups,
                group_score=group_score, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_bf16_logits_tie_to_the_lowest_index(uw, score, biased):
    # 256 values of 8 bits of mantissa in a narrow range: many are equal
    logits = (random_logits(90, 256, 5) * 0.2).to(torch.bfloat16)
    bias = torch.zeros(256, device="cuda") if biased else None
    check_route(uw, logits, 8, bias, score=score)
    check_route(uw, torch.zeros(70, 40, device="cuda"), 5, None if bias is None else bias[:40].contiguous(), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [7, 200])
def test_masked_and_extreme_logits(uw, score, t):
    inf, nan = math.inf, math.nan
    logits = random_logits(t, 24, 3)
    logits[0] = -inf                       # a padding token
    logits[1, 2:] = -inf                   # fewer experts left than slots
    logits[2] = nan
    logits[3, ::2] = nan
    logits[4, 5] = inf
    logits[5] = torch.linspace(-3e38, 3e38, 24, device="cuda")
    logits[6] = torch.linspace(-200.0, -100.0, 24, device="cuda")
    check_route(uw, logits, 4, score=score)
    check_route(uw, logits, 4, torch.zeros(24, device="cuda"), score=score)
    check_route(uw, logits, 4, score=score, n_groups=4, top_groups=2, group_score="top2")
    bias = torch.zeros(24, device="cuda")
    bias[3], bias[7] = -inf, nan           # experts taken out
    check_route(uw, logits, 4, bias, score=score, n_groups=2, top_groups=2)


def test_negative_zero_ties_with_zero(uw):
    logits = torch.full((3, 8), -1.0, device="cuda")
    logits[:, 2], logits[:, 5] = -0.0, 0.0
    assert check_route(uw, logits, 2).ids.tolist() == [[2, 5]] * 3


def test_scores_a_unit_apart_are_told_apart(uw):
    # sigmoid(l) + bias with gaps far below 2^-24: a 32-bit choice would tie
    logits = torch.zeros(40, 32, device="cuda")
    logits += torch.arange(32, device="cuda") * 1e-8
    check_route(uw, logits, 6, torch.full((32,), 0.25, device="cuda"), score="sigmoid")


def test_strided_rows_and_reused_buffers(uw):
    wide = random_logits(100, 300, 9)
    r = uw.route_experts(wide[:, 40:104], 6)
    again = uw.route_experts(wide[:, 40:104].contiguous(), 6)
    for f in ("ids", "weights", "offsets", "order", "slot"):
        assert torch.equal(getattr(r, f), getattr(again, f))
    other = random_logits(100, 64, 11)
    assert uw.route_experts(other, 6, out=r) is r
    check_route(uw, other, 6)
    assert torch.equal(r.ids, uw.route_experts(other, 6).ids)


def test_no_tokens(uw):
    r = uw.route_experts(torch.empty(0, 16, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 17 and r.ids.shape == (0, 2)
    g = uw.group_rows(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert g.offsets.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("rows,per_row,groups", [(1, 1, 1), (31, 1, 5), (700, 3, 7), (2048, 1, 1024), (2049, 1, 1024),
                                                 (5000, 8, 128), (100000, 1, 300), (9, 64, 2), (40, 64, 1000)])
def test_group_rows(uw, rows, per_row, groups):
    rng = np.random.default_rng(rows + groups)
    ids = rng.integers(-2, groups + 2, (rows, per_row)).astype(np.int32)   # the same id several times in a row too
    ids[rng.random(ids.shape) < 0.3] = groups // 2
    ids[0, 0] = np.iinfo(np.int32).min
    check_group(uw.group_rows(torch.from_numpy(ids).cuda(), groups), ids, groups)


def test_all_rows_in_one_group_and_in_none(uw):
    for value in (4, -1):
        ids = np.full((6000,), value, np.int32)
        check_group(uw.group_rows(torch.from_numpy(ids).cuda(), 9), ids, 9)


@pytest.mark.parametrize("t", [16, 3000])
def test_another_stream_and_a_replayed_graph(uw, t):
    logits = random_logits(t, 64, 21)
    want = uw.route_experts(logits, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = uw.route_experts(logits, 4, stream=s)
    s.synchronize()
    for f in ("ids", "weights", "offsets", "order", "slot"):
        assert torch.equal(getattr(got, f), getattr(want, f))
    static = logits.clone()
    out = uw.route_experts(static, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        uw.route_experts(static, 4, out=out)
    for seed in (1, 2):
        fresh = random_logits(t, 64, 100 + seed)
        static.copy_(fresh)
        g.replay()
        torch.cuda.synchronize()
        want = uw.route_experts(fresh, 4)
        for f in ("ids", "weights", "offsets", "order", "slot"):
            assert torch.equal(getattr(out, f), getattr(want, f))


def test_refusals(uw):
    x = torch.zeros(4, 16, device="cuda")
    for bad in (dict(top_k=0), dict(top_k=17), dict(top_k=33), dict(top_k=2, n_groups=3), dict(top_k=2, n_groups=0),
                dict(top_k=2, n_groups=4, top_groups=5), dict(top_k=5, n_groups=8, top_groups=2),
                dict(top_k=2, scale=math.nan)):
        with pytest.raises(uw.UwError) as err:
            uw.route_experts(x, **bad)
        assert err.value.status == uw.ERR_INVALID_ARG
    for bad in (dict(score="exp"), dict(group_score="mean"), dict(bias=torch.zeros(15, device="cuda")),
                dict(bias=torch.zeros(16)), dict(bias=torch.zeros(16, device="cuda", dtype=torch.float64))):
        with pytest.raises(ValueError):
            uw.route_experts(x, 2, **bad)
    for logits in (x.double(), x.T, x[0], x.cpu()):
        with pytest.raises(ValueError):
            uw.route_experts(logits, 2)
    with pytest.raises(ValueError):
        uw.route_experts(x, 2, out=uw.route_experts(x[:2].contiguous(), 2))
    with pytest.raises(ValueError):
        uw.group_rows(torch.zeros(4, device="cuda"), 2)
    with pytest.raises(uw.UwError):
        uw.group_rows(torch.zeros(4, device="cuda", dtype=torch.int32), uw.MAX_GROUPS + 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("top_k", [3, 32])
def test_choices_nearer_than_32_bits_tell_apart(uw, score, group_score, top_k):
    """Scores plus biases that differ by less than 2^-24, in one group and across
    groups: the order and the kept groups are those of 64 bits."""
    g = torch.Generator().manual_seed(top_k)
    logits = (torch.randint(0, 3, (60, 128), generator=g) * 1e-7 + torch.randn(60, 1, generator=g)).cuda()
    for bias in (torch.full((128,), 0.5), torch.randint(0, 2, (128,), generator=g) * 2.0 ** -24 + 0.25):
        check_route(uw, logits, top_k, bias.cuda(), score=score)
        check_route(uw, logits, top_k, bias.cuda(), score=score, n_groups=8, top_groups=3, group_score=group_score)
    check_route(uw, logits, top_k, score=score, n_groups=16, top_groups=5, group_score=group_score)


@pytest.mark.parametrize("n_groups", [1, 3, 5, 7, 12, 20, 31])
def test_odd_group_counts(uw, n_groups):
    e = n_groups * 11
    bias = torch.randn(e, generator=torch.Generator().manual_seed(e)).mul(0.1).cuda()
    for group_score in ("max", "top2"):
        check_route(uw, random_logits(75, e, e), 4, bias, score="sigmoid", n_groups=n_groups, top_groups=(n_groups + 1) // 2,
                    group_score=group_score)
