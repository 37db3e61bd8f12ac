"""Arguments that the operators around the matmuls refuse, before anything is
launched: through the C ABI with device addresses that are never read, on a
host without a GPU."""
import ctypes

import pytest

FAKE = 1 << 40


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exponent_b200 import uw as U
    return U


def router(uw, **kw):
    base = dict(experts=16, top_k=2, n_groups=1, top_groups=1, score=1, group_score=1, renormalize=1, logits_type=1, scale=1.0)
    base.update(kw)
    return uw.Router(**base)


def test_route(uw):
    L = uw.lib()
    size = ctypes.c_size_t()
    good = router(uw)
    assert L.uw_route_workspace_size(8, ctypes.byref(good), ctypes.byref(size)) == 0 and size.value == 0
    assert L.uw_route_workspace_size(4096, ctypes.byref(good), ctypes.byref(size)) == 0 and size.value > 0
    for bad in (dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=33, experts=64), dict(top_k=17),
                dict(n_groups=0), dict(n_groups=5), dict(n_groups=64, experts=64), dict(top_groups=2), dict(top_groups=0),
                dict(n_groups=8, top_groups=1, top_k=3), dict(score=0), dict(score=3), dict(group_score=3),
                dict(logits_type=0), dict(logits_type=3), dict(scale=float("inf")), dict(scale=float("nan"))):
        r = router(uw, **bad)
        assert L.uw_route_workspace_size(8, ctypes.byref(r), ctypes.byref(size)) == uw.ERR_INVALID_ARG, bad
    assert L.uw_route_workspace_size(-1, ctypes.byref(good), ctypes.byref(size)) == uw.ERR_INVALID_ARG
    assert L.uw_route_workspace_size(1 << 30, ctypes.byref(good), ctypes.byref(size)) == uw.ERR_UNSUPPORTED_SHAPE
    assert L.uw_route_workspace_size(8, None, ctypes.byref(size)) == uw.ERR_INVALID_ARG
    assert L.uw_route_workspace_size(8, ctypes.byref(good), None) == uw.ERR_INVALID_ARG

    def run(logits=FAKE, t=4096, stride=16, bias=None, ids=FAKE, w=FAKE, off=FAKE, order=FAKE, slot=FAKE, ws=FAKE,
            nbytes=1 << 30):
        return L.uw_route_experts(logits, t, stride, bias, ctypes.byref(good), ids, w, off, order, slot, ws, nbytes, None)
    for kw in (dict(logits=None), dict(t=-1), dict(stride=15), dict(ids=None), dict(w=None), dict(off=None),
               dict(order=None), dict(slot=None), dict(logits=FAKE + 2), dict(bias=FAKE + 1), dict(ids=FAKE + 2)):
        assert run(**kw) == uw.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(nbytes=size.value - 1)):
        assert run(**kw) == uw.ERR_WORKSPACE, kw


def test_group_rows(uw):
    L = uw.lib()
    size = ctypes.c_size_t()
    assert L.uw_group_workspace_size(10, 1, 5, ctypes.byref(size)) == 0 and size.value == 0
    assert L.uw_group_workspace_size(100000, 8, 128, ctypes.byref(size)) == 0 and size.value > 0
    for rows, per_row, groups in ((-1, 1, 4), (4, 0, 4), (4, 65, 4), (4, 1, 0), (4, 1, 1025)):
        assert L.uw_group_workspace_size(rows, per_row, groups, ctypes.byref(size)) == uw.ERR_INVALID_ARG
    assert L.uw_group_workspace_size(1 << 31, 1, 4, ctypes.byref(size)) == uw.ERR_UNSUPPORTED_SHAPE
    run = lambda ids, off, order, slot, ws, n: L.uw_group_rows(ids, 100000, 8, 128, off, order, slot, ws, n, None)
    assert run(None, FAKE, FAKE, FAKE, FAKE, 1 << 30) == uw.ERR_INVALID_ARG
    assert run(FAKE, None, FAKE, FAKE, FAKE, 1 << 30) == uw.ERR_INVALID_ARG
    assert run(FAKE, FAKE, None, FAKE, FAKE, 1 << 30) == uw.ERR_INVALID_ARG
    assert run(FAKE, FAKE, FAKE, FAKE + 1, FAKE, 1 << 30) == uw.ERR_INVALID_ARG
    assert run(FAKE, FAKE, FAKE, None, None, 0) == uw.ERR_WORKSPACE
    assert run(FAKE, FAKE, FAKE, None, FAKE, 100) == uw.ERR_WORKSPACE


def test_lora(uw):
    L = uw.lib()
    size = ctypes.c_size_t()

    def adapters(n=128, k=256, count=4, rank=16, a=FAKE, b=FAKE, ranks=None, scales=None):
        return uw.Adapters(n, k, count, rank, a, b, ranks, scales)

    for kw, status in ((dict(n=0), 1), (dict(k=-64), 1), (dict(n=100), 2), (dict(k=100), 2), (dict(count=0), 1),
                       (dict(count=1025), 1), (dict(rank=0), 1), (dict(rank=12), 1), (dict(rank=264), 1),
                       (dict(k=1 << 40), 2)):
        assert L.uw_lora_workspace_size(8, ctypes.byref(adapters(**kw)), ctypes.byref(size)) == status, kw
    assert L.uw_lora_workspace_size(-1, ctypes.byref(adapters()), ctypes.byref(size)) == 1
    assert L.uw_lora_workspace_size(0, ctypes.byref(adapters()), ctypes.byref(size)) == 0 and size.value == 0
    assert L.uw_lora_workspace_size(8, ctypes.byref(adapters()), ctypes.byref(size)) == 0 and size.value > 0

    def run(d=None, x=FAKE, xs=256, t=8, ids=FAKE, off=None, order=None, y=FAKE, ys=128, out=FAKE, os_=128, ws=FAKE,
            nbytes=1 << 30):
        d = d or adapters()
        return L.uw_lora_add(x, xs, t, ctypes.byref(d), ids, off, order, y, ys, out, os_, ws, nbytes, None)
    for kw in (dict(x=None), dict(y=None), dict(out=None), dict(x=FAKE + 8), dict(y=FAKE + 8, out=FAKE + 8), dict(xs=248),
               dict(xs=260), dict(ys=124, os_=124), dict(ys=130, os_=130), dict(os_=132), dict(ids=None),
               dict(ids=None, off=FAKE), dict(ids=FAKE + 2), dict(t=-1), dict(d=adapters(a=None)), dict(d=adapters(b=None)),
               dict(d=adapters(a=FAKE + 8)), dict(d=adapters(ranks=FAKE + 1)), dict(out=FAKE + 16),
               dict(out=FAKE + 4 * 128)):
        assert run(**kw) == uw.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(nbytes=size.value - 1)):
        assert run(**kw) == uw.ERR_WORKSPACE, kw
    assert run(t=0, x=None, ids=None, y=None, out=None, ws=None, nbytes=0) == uw.UW_OK    # nothing to launch
