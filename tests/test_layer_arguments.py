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
                       (dict(k=1 << 40), 2), (dict(n=1 << 24), 2)):
        assert L.uw_lora_workspace_size(8, ctypes.byref(adapters(**kw)), ctypes.byref(size)) == status, kw
    assert L.uw_lora_workspace_size(-1, ctypes.byref(adapters()), ctypes.byref(size)) == 1
    assert L.uw_lora_workspace_size(0, ctypes.byref(adapters()), ctypes.byref(size)) == 0 and size.value == 0
    assert L.uw_lora_workspace_size(8, ctypes.byref(adapters()), ctypes.byref(size)) == 0 and size.value == 0    # one launch
    assert L.uw_lora_workspace_size(8, ctypes.byref(adapters(k=65536)), ctypes.byref(size)) == 0 and size.value > 0
    assert L.uw_lora_workspace_size(80, ctypes.byref(adapters()), ctypes.byref(size)) == 0 and size.value > 0

    def run(d=None, x=FAKE, xs=256, t=80, ids=FAKE, off=None, order=None, y=FAKE, ys=128, out=FAKE, os_=128, ws=FAKE,
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
    for kw in (dict(ys=1 << 28, os_=1 << 28), dict(os_=1 << 28, out=FAKE << 4), dict(t=4096, ys=1 << 22, os_=1 << 22)):
        assert run(**kw) == uw.ERR_UNSUPPORTED_SHAPE, kw          # more than 64 GB


def test_expert_calls(uw):
    L = uw.lib()

    def rows(places=16, per_row=2, off=FAKE, order=FAKE, x=FAKE, x_rows=8, xs=128):
        return uw.ExpertRows(places, per_row, off, order, x, x_rows, xs)

    def wset(n=64, k=128, e=4, w=FAKE, stride=64 * 128, table=None):
        return uw.ExpertSetArgs(n, k, e, w, stride, table)

    P = uw.make_expert_plan
    ok = P(uw.KERNEL_MMA, 4)

    def run(r=None, w=None, y=FAKE, ys=64, plan=ok, ws=None, nbytes=0):
        r, w = r or rows(), w or wset()
        return L.uw_expert_matmul(ctypes.byref(r), ctypes.byref(w), y, ys, ctypes.byref(plan), ws, nbytes, None, None)

    assert run(rows(places=0, off=None, order=None, x=None, x_rows=0)) == uw.UW_OK
    for r in (rows(places=-1), rows(per_row=0), rows(off=None), rows(x=None), rows(x_rows=0), rows(order=None), rows(xs=120),
              rows(xs=132), rows(x=FAKE + 8), rows(off=FAKE + 2)):
        assert run(r) == uw.ERR_INVALID_ARG
    assert run(rows(places=1 << 31)) == uw.ERR_UNSUPPORTED_SHAPE
    for w, status in ((wset(n=0), 1), (wset(n=96), 2), (wset(k=100), 2), (wset(e=0), 1), (wset(e=1025), 1), (wset(w=None), 1),
                      (wset(table=FAKE), 1), (wset(w=FAKE + 8), 1), (wset(stride=64 * 127), 1), (wset(stride=64 * 128 + 4), 1),
                      (wset(w=None, table=FAKE + 8), 1)):
        assert run(w=w) == status
    assert run(y=None) == uw.ERR_INVALID_ARG and run(y=FAKE + 8) == uw.ERR_INVALID_ARG
    assert run(ys=60) == uw.ERR_INVALID_ARG and run(ys=66) == uw.ERR_INVALID_ARG
    for plan in (P(uw.KERNEL_MMA, 0), P(uw.KERNEL_MMA, 9), P(uw.KERNEL_MMA, 4, 32), P(uw.KERNEL_MMA, 4, width=3),
                 P(uw.KERNEL_MMA, 4, sort=1), P(uw.KERNEL_TC, 64), P(uw.KERNEL_TC, 256, 0), P(uw.KERNEL_TC, 256, 256), P(uw.KERNEL_TC, 128, 256), P(uw.KERNEL_TC, 128, 256, sort=1),
                 P(uw.KERNEL_TC, 256, width=1), P(uw.KERNEL_TC_SK, 16), P(uw.KERNEL_MMA, 4, timeout_ns=-1)):
        assert run(plan=plan) == uw.ERR_INVALID_ARG
    assert run(w=wset(k=192, stride=64 * 192), r=rows(xs=192), plan=P(uw.KERNEL_MMA, 4, width=2)) == uw.ERR_INVALID_ARG
    tc = P(uw.KERNEL_TC, 256)
    assert run(w=wset(w=None, table=FAKE), plan=tc) == uw.ERR_WORKSPACE       # rebuilt weights need one
    assert run(w=wset(stride=1 << 39), plan=tc) == uw.ERR_UNSUPPORTED_SHAPE
    sort, size = P(uw.KERNEL_TC, 256, sort=1), ctypes.c_size_t()
    for r, want in ((rows(), 16 * 128 * 2), (rows(order=None), 0)):
        assert L.uw_expert_workspace_size(ctypes.byref(r), ctypes.byref(wset()), 1, ctypes.byref(sort), ctypes.byref(size)) == 0
        assert size.value == want
        compressed = wset(w=None, table=FAKE)
        for gated in (0, 1):
            assert L.uw_expert_workspace_size(ctypes.byref(r), ctypes.byref(compressed), gated, ctypes.byref(sort), ctypes.byref(size)) == 0
            assert size.value == want + (1 + gated) * 4 * 64 * 128 * 2
    for ws, nbytes in ((None, 0), (FAKE, 4095), (FAKE + 16, 1 << 20)):
        assert run(plan=sort, ws=ws, nbytes=nbytes) == uw.ERR_WORKSPACE

    def gate_up(a, b, hs=64):
        r = rows()
        return L.uw_expert_gate_up(ctypes.byref(r), ctypes.byref(a), ctypes.byref(b) if b else None, FAKE, hs, ctypes.byref(ok),
                                   None, 0, None, None)
    for b in (None, wset(n=128, stride=1 << 20), wset(k=64), wset(e=5), wset(w=None, table=FAKE)):
        assert gate_up(wset(), b) == uw.ERR_INVALID_ARG
    assert gate_up(wset(), wset(), 68) == uw.ERR_INVALID_ARG

    p = uw.ExpertPlan()
    for w, places, gated, kernel in ((wset(), 4, 0, uw.KERNEL_MMA), (wset(), 100000, 0, uw.KERNEL_TC), (wset(), 100, 1, uw.KERNEL_TC),
                                     (wset(w=None, table=FAKE), 64, 0, uw.KERNEL_MMA), (wset(w=None, table=FAKE), 65, 0, uw.KERNEL_TC), (wset(k=192, stride=64 * 192), 1, 1, uw.KERNEL_MMA)):
        assert L.uw_expert_plan_default(ctypes.byref(w), places, gated, ctypes.byref(p)) == 0 and p.kernel == kernel
        # every default is a valid plan
        size = ctypes.c_size_t()
        assert L.uw_expert_workspace_size(ctypes.byref(rows(places=places)), ctypes.byref(w), gated, ctypes.byref(p), ctypes.byref(size)) == 0
    assert L.uw_expert_plan_default(ctypes.byref(wset()), -1, 0, ctypes.byref(p)) == uw.ERR_INVALID_ARG
    assert L.uw_expert_plan_default(ctypes.byref(wset()), 1, 0, None) == uw.ERR_INVALID_ARG


def test_expert_table(uw):
    import numpy as np
    from decode_gemm_exponent_b200 import synth
    L = uw.lib()
    dms = []
    for n, flags in ((64, 0), (64, 0), (128, 0), (64, uw.EMIT_HUFFMAN)):
        host = np.frombuffer(uw.encode(synth.weights_bf16(n, 128, 0.02, 0.002, 1.0, seed=n), flags), np.uint8)
        dm = uw.DMat()
        uw.check(L.uw_matrix_bind(host.ctypes.data, host.size, FAKE, FAKE, 0, ctypes.byref(dm)), "uw_matrix_bind")
        dms.append(dm)
    arr = lambda *i: (ctypes.POINTER(uw.DMat) * len(i))(*[ctypes.pointer(dms[j]) for j in i])
    table = np.zeros(4 * uw.EXPERT_ENTRY_BYTES, np.uint8)
    run = lambda a, n, size=table.size: L.uw_expert_table(a, n, table.ctypes.data, size)
    assert run(arr(0, 1), 2) == uw.UW_OK and table.any()
    assert run(arr(0, 1), 2, 127) == uw.ERR_WORKSPACE
    assert run(arr(0, 2), 2) == uw.ERR_INVALID_ARG           # another size
    assert run(arr(0, 3), 2) == uw.ERR_INVALID_ARG           # no palette plane
    assert run(arr(0), 0) == uw.ERR_INVALID_ARG
    assert run(None, 1) == uw.ERR_INVALID_ARG


def test_expert_combine(uw):
    L = uw.lib()

    def run(y=FAKE, ys=64, slot=FAKE, w=FAKE, t=8, k=2, n=64, base=None, bs=0, out=FAKE, os_=64):
        return L.uw_expert_combine(y, ys, slot, w, t, k, n, base, bs, out, os_, None)
    assert run(t=0, y=None, slot=None, w=None, out=None) == uw.UW_OK
    for kw in (dict(t=-1), dict(k=0), dict(n=0), dict(ys=60), dict(ys=66), dict(os_=60), dict(y=None), dict(slot=None),
               dict(w=None), dict(out=None), dict(y=FAKE + 4), dict(out=FAKE + 8), dict(base=FAKE, bs=60),
               dict(base=FAKE + 4, bs=64), dict(base=FAKE, bs=68), dict(slot=FAKE + 2)):
        assert run(**kw) == uw.ERR_INVALID_ARG, kw
    assert run(n=66, ys=68, os_=68) == uw.ERR_UNSUPPORTED_SHAPE
    assert run(t=1 << 31) == uw.ERR_UNSUPPORTED_SHAPE


def test_packed_structs_equal_the_declared_ones(uw):
    for packed, declared, values in ((uw._SET, uw.ExpertSetArgs, (64, 128, 5, FAKE, 64 * 128, FAKE + 16)),
                                     (uw._ROWS, uw.ExpertRows, (70, 7, FAKE, FAKE + 4, FAKE + 16, 10, 128)),
                                     (uw._ADAPTERS, uw.Adapters, (64, 128, 3, 16, FAKE, FAKE + 16, FAKE + 32, FAKE + 48))):
        s = declared(*values)
        got = declared.from_buffer_copy(packed.pack(*values))
        assert packed.size == ctypes.sizeof(declared)
        for name, _ in declared._fields_:
            assert getattr(got, name) == getattr(s, name), name
