"""Host side of the 4-bit cache and the step tables: refusals (found before
anything is enqueued), the plan's sizes, and the tests' own reference.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import q4_support as ref

OK, INVALID, SHAPE, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, -1, -2, -4, -6, -7
# addresses that pass a null and alignment check and are never read
A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def daa():
    from decode_attention_append_gb300 import build
    build.build()
    import decode_attention_append_gb300 as m
    m.load_library()
    return m


def _d(daa, hq=4, hkv=2, d=64, p=16, n=64):
    return daa._Dims(hq, hkv, d, p, n)


@pytest.mark.parametrize("change,expect", [
    (dict(k=None), INVALID), (dict(pool=None), INVALID), (dict(table=None), INVALID),
    (dict(batch=-1), INVALID), (dict(nnz=-1), INVALID), (dict(batch=0), SHAPE),
    (dict(k=ODD), ALIGNMENT), (dict(pool=ODD), ALIGNMENT),
    (dict(dims=dict(d=96)), UNSUPPORTED), (dict(dims=dict(p=32)), UNSUPPORTED),
    (dict(dims=dict(hq=34)), UNSUPPORTED), (dict(dims=dict(hq=3)), INVALID), (dict(dims=dict(n=0)), INVALID),
    (dict(nnz=0), OK), (dict(nnz=0, batch=0), OK),
])
def test_append_refusals(daa, change, expect):
    c = dict(k=A, pool=A, table=A, batch=2, nnz=3, dims={})
    c.update(change)
    lib = daa.load_library()
    assert lib.daa_kv_append_q4(c["k"], A, c["pool"], None, c["table"], A, A, A, c["batch"], c["nnz"],
                                _d(daa, **c["dims"]), None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(pool=None), INVALID), (dict(ids=None), INVALID), (dict(out=None), INVALID), (dict(n=-1), INVALID),
    (dict(out=ODD), ALIGNMENT), (dict(dims=dict(d=32)), UNSUPPORTED), (dict(n=0), OK),
])
def test_dequant_refusals(daa, change, expect):
    c = dict(pool=A, ids=A, out=A, n=3, dims={})
    c.update(change)
    lib = daa.load_library()
    assert lib.daa_kv_dequant_q4(c["pool"], None, c["ids"], c["n"], c["out"], _d(daa, **c["dims"]), None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(pool=dict(seq_len=None)), INVALID), (dict(pool=dict(counters=None)), INVALID),
    (dict(pool=dict(num_slots=0)), INVALID), (dict(pool=dict(max_pages=0)), INVALID),
    (dict(pool=dict(page_size=32)), UNSUPPORTED), (dict(pool=dict(num_slots=65537)), UNSUPPORTED),
    (dict(batch=-1), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(advance=2), INVALID),
    (dict(slots=None), INVALID), (dict(qo=None), INVALID), (dict(pages=None), INVALID),
    (dict(cap=-1), INVALID), (dict(slot_map=ctypes.c_void_p(0x10004)), ALIGNMENT),
])
def test_step_table_refusals(daa, change, expect):
    c = dict(pool={}, batch=2, advance=1, slots=A, qo=A, pages=A, cap=8, slot_map=A)
    c.update(change)
    pool = dict(seq_len=0x10000, held=0x10000, block_table=0x10000, free_pages=0x10000, counters=0x10000,
                num_slots=4, max_pages=4, num_pages=16, page_size=16)
    pool.update(c["pool"])
    lib = daa.load_library()
    st = daa._Pool(*pool.values())
    assert lib.daa_step_table(ctypes.byref(st), c["slots"], A, c["batch"], c["advance"], c["qo"], A, c["pages"],
                              c["cap"], A, c["slot_map"], A, 8, None) == expect
    assert lib.daa_step_table(None, A, A, 1, 1, A, A, A, 8, A, A, A, 8, None) == INVALID
    if "pool" in change:
        assert lib.daa_release_pages(ctypes.byref(st), A, 2, None) == expect
    st = daa._Pool(*dict(pool, num_slots=4, max_pages=4, page_size=16, seq_len=0x10000, counters=0x10000).values())
    assert lib.daa_release_pages(ctypes.byref(st), None, 2, None) == INVALID
    assert lib.daa_release_pages(ctypes.byref(st), A, -1, None) == INVALID
    assert lib.daa_release_pages(ctypes.byref(st), None, 0, None) == OK


def _ws(daa, qo, kv, last, **dims):
    st = ctypes.c_int32(0)
    p = [np.asarray(x, np.int32) for x in (qo, kv, last)]
    n = daa.load_library().daa_batch_attention_q4_workspace_size(*(x.ctypes.data_as(ctypes.c_void_p) for x in p),
                                                                 len(qo) - 1, _d(daa, **dims), ctypes.byref(st))
    return n, st.value


@pytest.mark.parametrize("qo,kv,last,dims,expect", [
    ([0, 2], [0, 1], [1], {}, SHAPE), ([0, 1], [0, 1], [0], {}, SHAPE), ([0, 1], [0, 1], [17], {}, SHAPE),
    ([1, 1], [0, 1], [1], {}, SHAPE), ([0, 3, 2], [0, 1, 2], [16, 16], {}, SHAPE), ([0, 1], [0, 0], [0], {}, SHAPE),
    ([0, 1], [0, 1], [3], dict(d=80), UNSUPPORTED), ([0, 1], [0, 1], [3], {}, OK),
    ([0, 0, 0], [0, 0, 4], [0, 3], {}, OK), ([0], [0], [], {}, OK),
    ([0, 900, 901], [0, 60, 80], [16, 1], dict(hq=32, hkv=8, d=128), OK),
])
def test_workspace_size(daa, qo, kv, last, dims, expect):
    n, st = _ws(daa, qo, kv, last, **dims)
    assert st == expect
    assert (n > 0) == (expect == OK and qo[-1] > 0)
    assert n == _ws(daa, qo, kv, last, **dims)[0]


def test_run_refusals(daa):
    lib = daa.load_library()
    info = daa.PlanInfo()
    run = lambda i, scale=1.0: lib.daa_batch_attention_q4_run(  # noqa: E731
        A, A, None, A, ctypes.byref(i) if i is not None else None, 1, scale, A, None, A, 1 << 20, _d(daa), None)
    assert run(None) == INVALID
    assert run(info) == INVALID  # no plan wrote it
    h = [np.asarray(x, np.int32) for x in ([0, 1], [0, 1], [3])]
    hp = [x.ctypes.data_as(ctypes.c_void_p) for x in h]
    plan = lambda ws, n, i=info: lib.daa_batch_attention_q4_plan(  # noqa: E731
        *hp, 1, _d(daa), ws, n, ctypes.byref(i) if i is not None else None, None)
    assert plan(A, 1 << 24, None) == INVALID
    assert plan(None, 0) == WORKSPACE
    assert plan(A, 16) == WORKSPACE
    assert plan(ctypes.c_void_p(0x10010), 1 << 24) == ALIGNMENT
    # a plan of nothing needs no workspace, and its run launches nothing
    e = [np.asarray(x, np.int32) for x in ([0, 0], [0, 2], [3])]
    assert lib.daa_batch_attention_q4_plan(*(x.ctypes.data_as(ctypes.c_void_p) for x in e), 1, _d(daa), None, 0,
                                           ctypes.byref(info), None) == OK
    assert run(info) == OK
    assert run(info, float("nan")) == INVALID and run(info, 0.0) == INVALID
    assert lib.daa_batch_attention_q4_run(A, A, None, A, ctypes.byref(info), 1, 1.0, A, None, A, 1 << 20,
                                          _d(daa, hq=2), None) == INVALID
    # a plan record of the bf16 calls is not one of these
    other = daa.PlanInfo()
    assert lib.daa_batch_attention_plan(*(x.ctypes.data_as(ctypes.c_void_p) for x in e), 1, None, None, 0, _d(daa),
                                        None, 0, ctypes.byref(other), None) == OK
    assert run(other) == INVALID


def test_binding_refuses_host_tensors(daa):
    pool = torch.zeros(4, 2, 2, 9 * 64, dtype=torch.uint8)
    ids = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        daa.kv_dequant_q4(pool, ids)
    with pytest.raises(TypeError):
        daa.PagePool.from_tensors(ids, ids, ids.view(1, 1), ids, torch.zeros(2, dtype=torch.int32))


def test_reference_rounds_to_nearest_even():
    """The reference against a search over every code, ties and cut-offs included."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((400, 64)) * 2.0 ** rng.integers(-14, 14, (400, 1))).bfloat16().double().numpy()
    x[0] = 0.0
    x[1, :16] = np.arange(16) * 0.25  # scale 0.625: exact midpoints among them
    x[2] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -0.0] * 4
    code, sc = ref.quantise(x, np.zeros(400))
    assert (code[2] == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 10, 12, 12, 14, 14, 8] * 4).all() and (sc[2] == 56).all()
    y = np.abs(x.reshape(400, 4, 16))
    full = np.concatenate([[0], ref.E4M3[1:]])
    d = np.abs(y.max(-1)[..., None] / 6 - full[1:])
    assert (np.abs(full[sc] - y.max(-1) / 6) <= d.min(-1) * (1 + 1e-12)).all()
    dist = np.abs(y[..., None] - full[sc][..., None, None] * ref.E2M1)
    got = np.take_along_axis(dist, (code.reshape(400, 4, 16) & 7)[..., None].astype(int), -1)[..., 0]
    assert (got <= dist.min(-1) + 1e-15 * y).all()


def test_reference_append_reads_back():
    rng = np.random.default_rng(2)
    t, n = ref.make_table(rng, [3, 0, 20], [15, 4, 0])
    k, v = (torch.from_numpy(rng.standard_normal((19, 2, 64))).bfloat16().double().numpy() for _ in range(2))
    pool = np.full((n, 2, 2, 9 * 64), 0xAB, np.uint8)
    ref.append(pool, k, v, t, [[1, 0], [0, -2]])
    vals = ref.decode_pages(pool, 64, [[1, 0], [0, -2]])
    page = t["page_indices"]
    got = np.stack([vals[page[t["kv_indptr"][0] + p // 16], :, :, p % 16] for p in range(3, 18)])
    for i, x in enumerate((k, v)):
        amax = np.abs(x[:15].reshape(15, 2, 4, 16)).max(-1)[..., None]
        # a step of the largest codes is a third of the block's maximum, its scale is off by at most 2^-4
        assert (np.abs(got[:, i] - x[:15]).reshape(15, 2, 4, 16) <= amax * (1 / 6 + 1 / 16)).all()
