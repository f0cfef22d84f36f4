"""The 4-bit cache and the step tables on the GPU against plain restatements in
64 bits: append and dequant bit by bit, tables entry by entry, attention within
the bounds that q4_support.check_attention derives from its roundings."""
import numpy as np
import pytest
import torch

import q4_support as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def daa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_append_gb300 as m
    m.device_error(reset=True)
    return m


@pytest.fixture(autouse=True)
def no_device_error(daa):
    yield
    assert daa.device_error(reset=True) == 0


DEV = "cuda"


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).bfloat16()


def _exps(rng, hkv, on):
    return rng.integers(-4, 5, (2, hkv)).astype(np.int32) if on else None


def _dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _pool(rng, n, hkv, d):
    """Slices of quantised values, as the append writes them (host uint8)."""
    body = rng.integers(0, 256, (n, hkv, 2, 8 * d), dtype=np.uint8)
    sc = rng.integers(40, 64, (n, hkv, 2, d), dtype=np.uint8)  # scales 0.16 .. 1.9
    return np.concatenate([body, sc], -1)


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("hkv,d,cached,new,exps", [
    (1, 64, [0], [1], False), (2, 64, [15, 16, 0, 3], [1, 1, 0, 33], True), (8, 128, [5] * 9, [1] * 9, False),
    (3, 128, [0, 100, 7], [200, 0, 9], True), (5, 64, [0, 1], [517, 16], False), (32, 128, [31], [40], True),
])
def test_append_bits(daa, hkv, d, cached, new, exps):
    rng = np.random.default_rng(hkv * 1000 + d + len(new))
    t, n = ref.make_table(rng, cached, new)
    e = _exps(rng, hkv, exps)
    rows = int(t["qo_indptr"][-1])
    k, v = _bf16(rng, (rows, hkv, d)), _bf16(rng, (rows, hkv, d), 1e-3)
    k[0, 0, :16] = torch.arange(16) * 0.25                          # exact midpoints
    k[0, 0, 16:32] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0])
    v[0, 0, :16] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1, -1, 3e38, -3e38, 1e-38, 9e-41, 0, -0.0, 100, 2688, 2000, 5, -7])
    v[0, 0, 16:32] = torch.tensor([float("nan"), 1, 2, 3, -4, 5, 6, 0.1, -0.2, 0.3, 1e-30, 0, -0.0, 1e-3, 2, 3])
    v[rows - 1, hkv - 1] = 0.0
    k[rows - 1, hkv - 1] *= 2.0 ** -12                               # below the smallest scale
    pool = np.full((n, hkv, 2, 9 * d), 0xA5, np.uint8)
    gpool = _dev(pool)
    g = {x: _dev(y) for x, y in t.items()}
    daa.kv_append_q4(k.to(DEV), v.to(DEV), gpool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"],
                     kv_exp=_dev(e))
    ref.append(pool, k.double().numpy(), v.double().numpy(), t, e)
    assert np.array_equal(gpool.cpu().numpy(), pool)  # untouched bytes among them


def test_append_bad_page_and_lengths(daa):
    rng = np.random.default_rng(3)
    t, n = ref.make_table(rng, [0, 4], [17, 2])
    k = _bf16(rng, (19, 2, 64)).to(DEV)
    pool = torch.full((n, 2, 2, 9 * 64), 7, dtype=torch.uint8, device=DEV)
    bad = dict(t, page_indices=t["page_indices"].copy())
    bad["page_indices"][1] = n  # the page of row 16
    g = {x: _dev(y) for x, y in bad.items()}
    daa.kv_append_q4(k, k, pool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"])
    assert daa.device_error(reset=True) == 1
    host = np.full((n, 2, 2, 9 * 64), 7, np.uint8)
    ref.append(host, k.double().cpu().numpy(), k.double().cpu().numpy(), t, None)
    host[t["page_indices"][1]] = 7  # that row is skipped, the others are written
    assert np.array_equal(pool.cpu().numpy(), host)
    bad = dict(t, last_page_len=np.array([1, 17], np.int32))
    g = {x: _dev(y) for x, y in bad.items()}
    daa.kv_append_q4(k, k, pool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"])
    assert daa.device_error(reset=True) == 3


# ------------------------------------------------------------------- dequant
@pytest.mark.parametrize("n,hkv,d,exps", [(1, 1, 64, False), (7, 3, 128, True), (33, 8, 64, True), (130, 5, 128, False)])
def test_dequant_exact(daa, n, hkv, d, exps):
    rng = np.random.default_rng(n)
    pool = rng.integers(0, 256, (n + 4, hkv, 2, 9 * d), dtype=np.uint8)
    pool[..., 8 * d:] &= 0x7F
    pool[..., 8 * d:][pool[..., 8 * d:] == 0x7F] = 0x7E  # every scale but NaN
    e = _exps(rng, hkv, exps)
    ids = rng.permutation(n + 4)[:n].astype(np.int32)
    out = daa.kv_dequant_q4(_dev(pool), _dev(ids), kv_exp=_dev(e))
    assert np.array_equal(out.double().cpu().numpy(), ref.decode_pages(pool[ids], d, e))


def test_dequant_page_twice_and_out_of_range(daa):
    rng = np.random.default_rng(4)
    pool = _pool(rng, 5, 2, 64)
    ids = np.array([3, -1, 3, 5, 0], np.int32)
    out = daa.kv_dequant_q4(_dev(pool), _dev(ids)).double().cpu().numpy()
    assert daa.device_error(reset=True) == 1
    want = ref.decode_pages(pool[np.clip(ids, 0, 4)], 64, None)
    want[[1, 3]] = 0
    assert np.array_equal(out, want)


# -------------------------------------------------------------------- tables
def _state(rng, slots, width, num_pages, lens):
    free = list(rng.permutation(num_pages))
    st = {"seq_len": np.zeros(slots, np.int32), "held": np.zeros(slots, np.int32),
          "block_table": np.full((slots, width), -1, np.int32)}
    for s, ln in lens.items():
        st["seq_len"][s] = ln
        st["held"][s] = -(-ln // 16)
        st["block_table"][s, :st["held"][s]] = [free.pop() for _ in range(st["held"][s])]
    st["free"] = free
    return st


def _device_pool(daa, st, num_pages):
    stack = np.full(num_pages, -1, np.int32)
    stack[:len(st["free"])] = st["free"]
    return daa.PagePool.from_tensors(_dev(st["seq_len"]), _dev(st["held"]), _dev(st["block_table"]), _dev(stack),
                                     torch.tensor([len(st["free"]), 0], dtype=torch.int32, device=DEV))


def _outs(batch, pages, rows, fill=-7):
    f = lambda n, dt=torch.int32: torch.full((n,), fill, dtype=dt, device=DEV)  # noqa: E731
    return dict(qo_indptr=f(batch + 1), kv_indptr=f(batch + 1), page_indices=f(pages), last_page_len=f(batch),
                slot_map=f(rows, torch.int64), positions=f(rows))


def _same_state(pool, st):
    n = len(st["free"])
    assert np.array_equal(pool.seq_len.cpu().numpy(), st["seq_len"])
    assert np.array_equal(pool.held.cpu().numpy(), st["held"])
    assert np.array_equal(pool.block_table.cpu().numpy(), st["block_table"])
    assert pool.counters.tolist() == [n, 0]
    assert pool.free_pages[:n].tolist() == [int(x) for x in st["free"]]


@pytest.mark.parametrize("batch,hi,new_hi,advance,spare", [
    (1, 1, 1, True, 0), (1, 40, 300, False, 3), (5, 100, 40, True, 2), (64, 300, 1, True, 40),
    (600, 40, 3, False, 9), (513, 3000, 2, True, 1), (1500, 20, 20, True, 100),
])
def test_step_table(daa, batch, hi, new_hi, advance, spare):
    rng = np.random.default_rng(batch + hi)
    slots = rng.permutation(batch + spare)[:batch]
    lens = {int(s): int(rng.integers(0, hi + 1)) for s in slots}
    width = -(-(hi + new_hi) // 16) + 1
    num_pages = (batch + 1) * width
    st = _state(rng, batch + spare, width, num_pages, lens)
    st["held"][slots[0]] = min(width, st["held"][slots[0]] + 1)  # cut back earlier: holds a page more than its length
    if st["block_table"][slots[0], st["held"][slots[0]] - 1] < 0:
        st["block_table"][slots[0], st["held"][slots[0]] - 1] = st["free"].pop()
    pool = _device_pool(daa, st, num_pages)
    for step in range(2):
        new = rng.integers(0, new_hi + 1, batch) // (1 + step)
        want = ref.step_table(st, slots, new, advance)
        n_pages, n_rows = want["kv_indptr"][-1], want["qo_indptr"][-1]
        # room for more than the step has: what lies behind is left alone
        out = _outs(batch, n_pages + (5000 if step else 3), n_rows + 2)
        pool.build(_dev(slots.astype(np.int32)), _dev(new.astype(np.int32)), advance=advance, **out)
        for name, w in want.items():
            assert np.array_equal(out[name].cpu().numpy()[:len(w)], w), name
            assert (out[name][len(w):] == -7).all(), name
        _same_state(pool, st)
    if not advance:  # the same step again takes no pages and says the same
        again = _outs(batch, n_pages, n_rows)
        pool.build(_dev(slots.astype(np.int32)), _dev(new.astype(np.int32)), **again)
        for name, w in want.items():
            assert np.array_equal(again[name].cpu().numpy(), w), name
        _same_state(pool, st)


def test_step_table_refuses_as_a_whole(daa):
    rng = np.random.default_rng(5)
    st = _state(rng, 6, 4, 12, {0: 30, 1: 16, 2: 1, 4: 0})
    pool = _device_pool(daa, st, 12)

    def refused(slots, new, code, pages=12, rows=200):
        out = _outs(len(slots), pages, rows)
        pool.build(_dev(np.array(slots, np.int32)), _dev(np.array(new, np.int32)), advance=True, **out)
        assert daa.device_error(reset=True) == code
        for n in ("qo_indptr", "kv_indptr", "last_page_len"):
            assert (out[n] == 0).all()
        for n in ("page_indices", "slot_map", "positions"):
            assert (out[n] == -7).all()
        _same_state(pool, st)

    refused([0, 6], [1, 1], 3)
    refused([0, -1], [1, 1], 3)
    refused([0, 1, 0], [1, 1, 1], 3)      # a slot twice
    refused([0, 1], [1, -1], 3)
    refused([0, 1], [35, 1], 3)           # 65 tokens in a row of 64
    refused([0, 1], [2 ** 31 - 1, 2 ** 31 - 1], 3)
    refused([0, 1], [1, 1], 3, pages=3)   # 4 pages
    refused([0, 1], [5, 5], 3, rows=9)
    refused([4, 5, 3], [64, 64, 1], 4)    # 9 pages, 8 free
    out = _outs(3, 9, 113)
    pool.build(_dev(np.array([4, 5, 3], np.int32)), _dev(np.array([64, 48, 1], np.int32)), advance=True, **out)
    ref.step_table(st, [4, 5, 3], [64, 48, 1], True)
    assert pool.counters.tolist() == [0, 0]
    _same_state(pool, st)


def test_empty_step(daa):
    pool = daa.PagePool(8, 3, 4)
    out = _outs(0, 4, 4)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    pool.build(e, e, **out)
    assert out["qo_indptr"].tolist() == [0] and out["kv_indptr"].tolist() == [0]
    t = pool.step([1, 2], [0, 0])
    assert t.qo_indptr.tolist() == [0, 0, 0] and t.page_indices.numel() == 0 and t.last_page_len.tolist() == [0, 0]


def test_page_pool_serving_loop(daa):
    """Admit, decode, cut back, release: host copies and device state agree throughout."""
    rng = np.random.default_rng(6)
    pool = daa.PagePool(400, 20, 40)
    st = {"seq_len": np.zeros(20, np.int32), "held": np.zeros(20, np.int32),
          "block_table": np.full((20, 40), -1, np.int32), "free": list(range(399, -1, -1))}
    live = []
    for step in range(30):
        idle = [s for s in range(20) if s not in live]
        admit = idle[:int(rng.integers(0, 4))]
        slots = live + admit
        rng.shuffle(slots)
        new = [int(rng.integers(1, 90)) if s in admit else int(rng.integers(0, 6)) for s in slots]
        advance = bool(step % 3)
        t = pool.step(slots, new, advance=advance)
        want = ref.step_table(st, slots, new, advance)
        for name, w in want.items():
            assert np.array_equal(getattr(t, name).cpu().numpy(), w), name
        assert np.array_equal(t.h_qo_indptr, want["qo_indptr"]) and np.array_equal(t.h_kv_indptr, want["kv_indptr"])
        assert np.array_equal(t.h_last_page_len, want["last_page_len"])
        live = slots
        if not advance:
            kept = [int(st["seq_len"][s]) + (n if s in admit else n // 2) for s, n in zip(slots, new)]
            pool.set_lengths(slots, kept)
            for s, k in zip(slots, kept):
                st["seq_len"][s] = k
        gone = [s for s in live if rng.random() < 0.15]
        before = list(st["free"])
        pool.release(gone)
        back = [int(x) for s in gone for x in st["block_table"][s, :st["held"][s]]]
        st["free"] = before + back[::-1]
        for s in gone:
            st["seq_len"][s] = st["held"][s] = 0
            live.remove(s)
        _same_state(pool, st)
        assert pool.h_free == len(st["free"]) and np.array_equal(pool.h_len, st["seq_len"])
    with pytest.raises(daa.DaaError):
        pool.step([0], [40 * 16 + 1])
    with pytest.raises(ValueError):
        pool.step([0, 0], [1, 1])
    with pytest.raises(ValueError):
        pool.release([20])
    _same_state(pool, st)


def test_release_refuses(daa):
    rng = np.random.default_rng(7)
    st = _state(rng, 4, 3, 9, {0: 30, 2: 16})
    pool = _device_pool(daa, st, 9)
    lib = daa.load_library()
    import ctypes
    for slots in ([0, 0], [4], [-1]):
        s = _dev(np.array(slots, np.int32))
        assert lib.daa_release_pages(ctypes.byref(pool._pool), ctypes.c_void_p(s.data_ptr()), len(slots),
                                     ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        assert daa.device_error(reset=True) == 3
        _same_state(pool, st)


# ----------------------------------------------------------------- attention
def _attend(daa, rng, hq, hkv, d, cached, new, causal=True, exps=False, scale=None, poison=True, spare=5):
    t, n = ref.make_table(rng, cached, new, spare)
    e = _exps(rng, hkv, exps)
    pool = _pool(rng, n, hkv, d)
    clean = pool.copy()
    if poison:  # slots past the last token hold NaN scales and any codes
        for r in range(len(new)):
            ln = int(t["last_page_len"][r])
            if 0 < ln < 16:
                p = t["page_indices"][t["kv_indptr"][r + 1] - 1]
                nb = d // 16
                pool[p, :, :, ln * (d // 2):8 * d] = 0xFF
                pool[p, :, 0, 8 * d + ln * nb:] = 0x7F
                pool[p, :, 1, 8 * d:].reshape(hkv, nb, 16)[:, :, ln:] = 0xFF
    rows = int(t["qo_indptr"][-1])
    q = _bf16(rng, (rows, hq, d))
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    attn = daa.BatchAttentionQ4(table, hq, _dev(pool), causal=causal, sm_scale=scale, kv_exp=_dev(e))
    out = torch.full((rows, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows, hq), float("nan"), device=DEV)
    attn.run(q.to(DEV), out=out, lse=lse)
    sc = scale if scale is not None else 1.0 / d ** 0.5
    want = ref.attention(q.double().numpy(), clean, t, e, d, sc, causal)
    return attn, q, out, lse, want


def _check(daa, *args, **kw):
    attn, q, out, lse, want = _attend(daa, *args, **kw)
    ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, out.shape[2])
    return attn, q, out, lse, want


LENS = [  # (cached, new)
    ([0], [1]), ([15], [1]), ([16], [1]), ([130, 0, 3, 700], [1, 1, 0, 1]), ([40, 127, 128, 5], [1, 2, 3, 4]),
    ([0, 33, 64], [5, 16, 7]), ([300], [40]), ([70, 12], [1, 300]),
]


@pytest.mark.parametrize("cached,new", LENS)
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (4, 2, 64), (8, 1, 128), (6, 2, 128)])
def test_attention_lengths(daa, hq, hkv, d, cached, new):
    _check(daa, np.random.default_rng(sum(cached) + 7 * hq), hq, hkv, d, cached, new, exps=bool(hq & 2))


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_groups(daa, g, d):
    _check(daa, np.random.default_rng(g), 2 * g, 2, d, [90, 500, 17], [1, 1, 3], exps=bool(g & 1))


@pytest.mark.parametrize("cached,new", [([20, 0], [1, 1]), ([31, 3, 0], [2, 9, 4]), ([5], [130])])
def test_attention_not_causal(daa, cached, new):
    _check(daa, np.random.default_rng(9), 8, 2, 128, cached, new, causal=False)


def test_attention_long_split(daa):
    """Few requests, many keys: the splits of one request are joined, for one and for several tokens."""
    _check(daa, np.random.default_rng(10), 4, 1, 128, [9001, 4095], [1, 1])
    _check(daa, np.random.default_rng(11), 8, 1, 64, [6000, 77], [5, 2], exps=True)
    _check(daa, np.random.default_rng(12), 2, 2, 128, [5003], [1])


def test_attention_large_scores(daa):
    """Scores of hundreds: the running maximum moves, and most weights vanish."""
    _check(daa, np.random.default_rng(13), 8, 2, 128, [700, 90], [1, 4], scale=1.0)
    _check(daa, np.random.default_rng(14), 3, 1, 64, [2100], [1], scale=2.5)


@pytest.mark.parametrize("mag", [1e-30, 1e-6, 1e4, 1e30])
def test_attention_query_range(daa, mag):
    """Queries of any bf16 size (the scale makes up for it)."""
    rng = np.random.default_rng(15)
    t, n = ref.make_table(rng, [100, 30], [1, 3])
    pool = _pool(rng, n, 2, 128)
    q = _bf16(rng, (4, 8, 128), mag)
    q[0, 0] = 0  # a row of zeros: every key weighs the same
    q[1, 1, ::2] *= 2.0 ** -20
    scale = 0.1 / mag
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    attn = daa.BatchAttentionQ4(table, 8, _dev(pool), sm_scale=scale)
    lse = torch.empty(4, 8, device=DEV)
    out = attn.run(q.to(DEV), lse=lse)
    ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                        ref.attention(q.double().numpy(), pool, t, None, 128, scale), 128)


def test_attention_bad_page(daa):
    rng = np.random.default_rng(16)
    t, n = ref.make_table(rng, [100, 50], [1, 70])
    t["page_indices"][2] = n + 100
    t["page_indices"][-1] = -5
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    attn = daa.BatchAttentionQ4(table, 4, _dev(_pool(rng, n, 2, 64)))
    attn.run(_bf16(rng, (71, 4, 64)).to(DEV))
    assert daa.device_error(reset=True) == 1


def test_attention_binding_refusals(daa):
    rng = np.random.default_rng(17)
    attn, q, out, lse, _ = _attend(daa, rng, 4, 2, 64, [10], [2])
    qd = q.to(DEV)
    with pytest.raises(ValueError):
        attn.run(qd[:1].contiguous())
    with pytest.raises(TypeError):
        attn.run(qd.float())
    with pytest.raises(TypeError):
        attn.run(qd, out=out.transpose(0, 1))
    with pytest.raises(ValueError):
        attn.run(qd, lse=lse[:1])
    with pytest.raises(ValueError):
        daa.BatchAttentionQ4(attn.t, 4, attn.kv_pages, kv_exp=torch.zeros(2, 3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        daa.BatchAttentionQ4(attn.t, 4, attn.kv_pages[..., :-1].contiguous())
    with pytest.raises(daa.DaaError):
        daa.BatchAttentionQ4(attn.t, 3, attn.kv_pages)
    with pytest.raises(TypeError):
        daa.BatchAttentionQ4(attn.t, 4, attn.kv_pages[:, :1])


# ------------------------------------------------------- streams, graphs, runs
def test_run_in_graphs(daa):
    rng = np.random.default_rng(18)
    attn, q, out, lse, want = _attend(daa, rng, 8, 2, 128, [700, 20, 33], [1, 1, 40])
    other, q2, out2, lse2, want2 = _attend(daa, rng, 8, 2, 128, [300, 2000], [4, 1])
    with pytest.raises(daa.DaaError):
        fresh = daa.BatchAttentionQ4(attn.t, 8, attn.kv_pages)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fresh.plan()
    torch.cuda.synchronize()
    qs, graphs = [q.to(DEV), q2.to(DEV)], []
    for a, x, o, l in ((attn, qs[0], out, lse), (other, qs[1], out2, lse2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.run(x, out=o, lse=l)
        graphs.append(g)
    for _ in range(3):  # two graphs in turn, each on its own workspace
        for o, l in ((out, lse), (out2, lse2)):
            o.fill_(float("nan"))
            l.fill_(float("nan"))
        for g in graphs:
            g.replay()
        for o, l, w in ((out, lse, want), (out2, lse2, want2)):
            ref.check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(), w, 128)


def test_own_stream_and_repeatable(daa):
    rng = np.random.default_rng(19)
    attn, q, out, lse, want = _attend(daa, rng, 12, 3, 128, [3000, 20, 500, 64], [1, 1, 5, 200])
    qd, s = q.to(DEV), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    for stream in (s, s.cuda_stream):
        out2.fill_(0)
        s.wait_stream(torch.cuda.current_stream())
        attn.run(qd, out=out2, lse=lse2, stream=stream)
        s.synchronize()
        assert torch.equal(out2, out) and torch.equal(lse2, lse)  # bit by bit


@pytest.mark.parametrize("hq,hkv,d,exps", [(4, 2, 64, True), (16, 2, 128, False), (2, 2, 128, True)])
def test_serving_steps_together(daa, hq, hkv, d, exps):
    """Tables from lengths, append and attention over several steps: chunks, decodes, and a request that leaves."""
    rng = np.random.default_rng(20 + d)
    e = _exps(rng, hkv, exps)
    pool = daa.PagePool(300, 6, 60)
    cache = daa.new_q4_pool(300, hkv, d)
    host = np.zeros((300, hkv, 2, 9 * d), np.uint8)
    plan = [([0, 1, 2], [70, 1, 300]), ([0, 1, 2], [1, 1, 1]), ([3, 2, 0, 1], [90, 4, 1, 1]), ([3, 0], [1, 5]), ([4, 3, 0], [33, 1, 1])]
    for i, (slots, new) in enumerate(plan):
        t = pool.step(slots, new)
        rows = sum(new)
        q, k, v = _bf16(rng, (rows, hq, d)), _bf16(rng, (rows, hkv, d)), _bf16(rng, (rows, hkv, d))
        lse = torch.empty(rows, hq, device=DEV)
        out = daa.BatchAttentionQ4(t, hq, cache, kv_exp=_dev(e)).step(k.to(DEV), v.to(DEV), q.to(DEV), lse=lse)
        ht = {n: getattr(t, n).cpu().numpy() for n in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")}
        ref.append(host, k.double().numpy(), v.double().numpy(), ht, e)
        assert np.array_equal(cache.cpu().numpy(), host)
        ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                            ref.attention(q.double().numpy(), host, ht, e, d, 1 / d ** 0.5), d)
        # the places that the tables name are those of the append
        vals = daa.kv_dequant_q4(cache, t.page_indices, kv_exp=_dev(e)).transpose(1, 2)
        assert t.slot_map.numel() == rows and vals.shape[0] == int(ht["kv_indptr"][-1])
        if i == 2:
            pool.release([1, 2])
    assert np.isin(t.slot_map.cpu().numpy() // 16, t.page_indices.cpu().numpy()).all()


@pytest.mark.parametrize("hq,hkv,new", [(8, 1, [12]), (8, 1, [13]), (4, 1, [24, 25]), (16, 1, [6, 7, 1])])
def test_attention_around_the_row_threshold(daa, hq, hkv, new):
    """Around the rows from which a request counts as a long chunk."""
    _check(daa, np.random.default_rng(21), hq, hkv, 128, [333] * len(new), new)
    _check(daa, np.random.default_rng(22), hq, hkv, 64, [90] * len(new), new, causal=False)


def test_attention_many_small_requests(daa):
    rng = np.random.default_rng(23)
    n = 1500
    _check(daa, rng, 6, 3, 64, rng.integers(0, 40, n).tolist(), rng.integers(0, 3, n).tolist())


def test_offsets_past_32_bits(daa):
    """Pages whose bytes lie past 4 GB: appended, read back and attended to."""
    rng = np.random.default_rng(24)
    hkv, d = 4, 128
    n = (1 << 32) // (hkv * 2 * 9 * d) + 100
    pool = torch.zeros(n, hkv, 2, 9 * d, dtype=torch.uint8, device=DEV)
    t, used = ref.make_table(rng, [0, 0], [50, 129], spare=0)
    low = t["page_indices"].copy()
    t["page_indices"] = (n - used + low).astype(np.int32)
    g = {x: _dev(y) for x, y in t.items()}
    k, v, q = _bf16(rng, (179, hkv, d)), _bf16(rng, (179, hkv, d)), _bf16(rng, (179, 2 * hkv, d))
    daa.kv_append_q4(k.to(DEV), v.to(DEV), pool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"])
    host = np.zeros((used, hkv, 2, 9 * d), np.uint8)
    small = dict(t, page_indices=low)
    ref.append(host, k.double().numpy(), v.double().numpy(), small, None)
    assert np.array_equal(pool[n - used:].cpu().numpy(), host)
    assert not pool[:n - used].any()
    back = daa.kv_dequant_q4(pool, g["page_indices"])
    assert np.array_equal(back.double().cpu().numpy(), ref.decode_pages(host[low], d, None))
    for rows, tab in ((slice(0, 179), small), (slice(49, 50), None)):
        if tab is None:  # the first request's last token alone: a decode step
            tab = {"qo_indptr": np.array([0, 1], np.int32), "kv_indptr": t["kv_indptr"][:2],
                   "page_indices": low[:t["kv_indptr"][1]], "last_page_len": t["last_page_len"][:1]}
        table = daa.PageTable.from_host(tab["qo_indptr"], tab["kv_indptr"], n - used + tab["page_indices"],
                                        tab["last_page_len"], DEV)
        lse = torch.empty(q[rows].shape[0], 2 * hkv, device=DEV)
        out = daa.BatchAttentionQ4(table, 2 * hkv, pool).run(q[rows].to(DEV), lse=lse)
        ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                            ref.attention(q[rows].double().numpy(), host, tab, None, d, 1 / d ** 0.5), d)


def test_two_streams_at_once(daa):
    """Two batches with workspaces of their own, many runs under way at the same time."""
    rng = np.random.default_rng(25)
    made = [_attend(daa, rng, 8, 2, 128, [3000, 40, 900], [1, 5, 30]), _attend(daa, rng, 16, 1, 64, [5000, 7], [1, 1])]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    outs = []
    for (attn, q, out, lse, want), s in zip(made, streams):
        qd, o, l = q.to(DEV), torch.zeros_like(out), torch.zeros_like(lse)
        torch.cuda.synchronize()
        outs.append((attn, qd, o, l, s))
    for _ in range(20):
        for attn, qd, o, l, s in outs:
            attn.run(qd, out=o, lse=l, stream=s)
    torch.cuda.synchronize()
    for (attn, q, out, lse, want), (_, _, o, l, _) in zip(made, outs):
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_step_in_a_graph(daa):
    """Tables, append and attention of a step captured as one graph and replayed with new values."""
    rng = np.random.default_rng(26)
    hq, hkv, d = 8, 2, 128
    slots, cached, new = [3, 0, 2], [100, 33, 700], [1, 2, 1]
    st = _state(rng, 4, 60, 150, dict(zip(slots, cached)))
    pool = _device_pool(daa, st, 150)
    want = ref.step_table({**st, "free": list(st["free"]), "held": st["held"].copy(), "block_table": st["block_table"].copy()},
                          slots, new, False)
    ht = {x: np.array(want[x], np.int32) for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")}
    o = _outs(3, len(want["page_indices"]), 4)
    table = daa.PageTable(o["qo_indptr"], o["kv_indptr"], o["page_indices"], o["last_page_len"], ht["qo_indptr"],
                          ht["kv_indptr"], ht["last_page_len"])
    cache = _dev(_pool(rng, 150, hkv, d))
    first = cache.clone()
    attn = daa.BatchAttentionQ4(table, hq, cache)
    attn.plan()
    q, k, v = (torch.zeros(4, h, d, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv))
    out, lse = torch.empty_like(q), torch.empty(4, hq, device=DEV)
    s_dev, n_dev = _dev(np.array(slots, np.int32)), _dev(np.array(new, np.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.build(s_dev, n_dev, **o)
        attn.append(k, v)
        attn.run(q, out=out, lse=lse)
    for _ in range(3):
        cache.copy_(first)
        hq_, hk_, hv_ = _bf16(rng, q.shape), _bf16(rng, k.shape), _bf16(rng, v.shape)
        q.copy_(hq_), k.copy_(hk_), v.copy_(hv_)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len", "slot_map", "positions"):
            assert np.array_equal(o[name].cpu().numpy(), want[name]), name
        host = first.cpu().numpy()
        ref.append(host, hk_.double().numpy(), hv_.double().numpy(), ht, None)
        assert np.array_equal(cache.cpu().numpy(), host)
        ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                            ref.attention(hq_.double().numpy(), host, ht, None, d, 1 / d ** 0.5), d)


def test_traced_runs(daa):
    """Under the tracer every kernel runs alone; the results are the same, and the kernels have names."""
    rng = np.random.default_rng(27)
    attn, q, out, lse, want = _attend(daa, rng, 12, 3, 128, [3000, 20, 64], [1, 1, 200])
    qd, o2 = q.to(DEV), torch.zeros_like(out)
    daa.trace_enable(64)
    try:
        attn.run(qd, out=o2)
        daa.kv_dequant_q4(attn.kv_pages, attn.t.page_indices)
        names = [n for n, _ in daa.trace_read()]
    finally:
        daa.trace_disable()
    assert torch.equal(o2, out)
    assert names[0] == "kv_dequant_q4" and names[-1] == "kv_dequant_q4" and "attention_q4" in names


def test_append_after_other_kernels(daa):
    """Launches overlap the kernel before them: values written just before are the ones that are used."""
    rng = np.random.default_rng(28)
    hkv, d = 2, 128
    t, n = ref.make_table(rng, [0, 5], [300, 40])
    g = {x: _dev(y) for x, y in t.items()}
    src = [_bf16(rng, (340, hkv, d)).to(DEV) for _ in range(4)]
    k = torch.empty_like(src[0])
    pool = daa.new_q4_pool(n, hkv, d)
    reads = []
    for x in src:
        k.copy_(x)
        daa.kv_append_q4(k, k, pool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"])
        reads.append(daa.kv_dequant_q4(pool, g["page_indices"]))
    for x, r in zip(src, reads):
        host = np.zeros((n, hkv, 2, 9 * d), np.uint8)
        ref.append(host, x.double().cpu().numpy(), x.double().cpu().numpy(), t, None)
        assert np.array_equal(r.double().cpu().numpy(), ref.decode_pages(host[t["page_indices"]], d, None))


@pytest.mark.parametrize("e", [0, -3])
def test_append_every_block_maximum(daa, e):
    """Every finite bf16 as a block's largest value, the rest of the block on and
    beside the midpoints between codes: bit by bit as the exact quotients round."""
    rng = np.random.default_rng(30)
    top = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 0 .. the largest
    rows = -(-len(top) // 8)
    top = torch.cat([top, top[:8 * rows - len(top)]])
    t, n = ref.make_table(rng, [0], [rows], spare=0)
    g = {x: _dev(y) for x, y in t.items()}
    scale = ref.E4M3[ref.quantise(top.double().numpy()[:, None].repeat(16, 1), np.full(len(top), e))[1][:, 0]]
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * scale[:, None] * 2.0 ** e  # 7 bits at most: exact where normal
    on = torch.from_numpy(np.clip(mid, 0, 3e38)).bfloat16()
    bits = on.view(torch.int16)
    block = torch.cat([top[:, None], on, (bits + 1).view(torch.bfloat16), (bits - 1).clamp(min=0).view(torch.bfloat16)[:, :1]], 1)
    block = torch.where(block.abs() > top[:, None].abs(), top[:, None], block)
    block = block * torch.from_numpy(rng.choice([-1.0, 1.0], (len(top), 16))).bfloat16()
    k = block.reshape(rows, 1, 128)
    exps = np.full((2, 1), e, np.int32)
    pool = np.zeros((n, 1, 2, 9 * 128), np.uint8)
    gpool = _dev(pool)
    daa.kv_append_q4(k.to(DEV), k.to(DEV), gpool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"],
                     kv_exp=_dev(exps))
    ref.append(pool, k.double().numpy(), k.double().numpy(), t, exps)
    assert np.array_equal(gpool.cpu().numpy(), pool)


def test_append_many_requests_and_offset_rows(daa):
    """More requests than a CTA keeps in shared memory; K on a 16-byte boundary that is none of 32."""
    rng = np.random.default_rng(31)
    hkv, d = 2, 64
    t, n = ref.make_table(rng, rng.integers(0, 20, 1400), rng.integers(0, 3, 1400))
    rows = int(t["qo_indptr"][-1])
    k, v = _bf16(rng, (rows, hkv, d)), _bf16(rng, (rows, hkv, d))
    room = torch.zeros(k.numel() + 8, dtype=torch.bfloat16, device=DEV)
    kd = room[8:].view(rows, hkv, d)
    kd.copy_(k)
    assert kd.data_ptr() % 32 == 16
    g = {x: _dev(y) for x, y in t.items()}
    gpool = daa.new_q4_pool(n, hkv, d)
    daa.kv_append_q4(kd, v.to(DEV), gpool, g["qo_indptr"], g["page_indices"], g["kv_indptr"], g["last_page_len"])
    pool = np.zeros((n, hkv, 2, 9 * d), np.uint8)
    ref.append(pool, k.double().numpy(), v.double().numpy(), t, None)
    assert np.array_equal(gpool.cpu().numpy(), pool)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_step_table_into_a_buffer_at_any_place(daa, off):
    rng = np.random.default_rng(32)
    lens = {i: int(x) for i, x in enumerate(rng.integers(0, 700, 40))}
    st = _state(rng, 40, 60, 2400, lens)
    pool = _device_pool(daa, st, 2400)
    new = rng.integers(0, 60, 40)
    want = ref.step_table(st, list(range(40)), new, True)
    pages = len(want["page_indices"])
    out = _outs(40, pages + 9, len(want["positions"]))
    buf = out["page_indices"]
    out["page_indices"] = buf[off:off + pages]
    pool.build(_dev(np.arange(40, dtype=np.int32)), _dev(new.astype(np.int32)), advance=True, **out)
    for name, w in want.items():
        assert np.array_equal(out[name].cpu().numpy(), w), name
    assert (buf[:off] == -7).all() and (buf[off + pages:] == -7).all()
    _same_state(pool, st)


def test_attention_refuses_a_short_page_list(daa):
    t, n = ref.make_table(np.random.default_rng(33), [40, 3], [1, 1])
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    table.page_indices = table.page_indices[:-1]
    with pytest.raises(ValueError):
        daa.BatchAttentionQ4(table, 2, daa.new_q4_pool(n, 2, 64))


@pytest.mark.parametrize("hq,hkv,d,cached,new,causal,exps,bf16", [
    (32, 8, 128, [300, 20, 0], [512, 1, 0], True, True, True),       # four-tile items, a decode beside
    (32, 8, 64, [77, 900], [500, 6], True, False, True),
    (16, 16, 128, [100, 0], [260, 259], False, True, True),
    (8, 8, 64, [5, 700, 3], [700, 1, 1], False, False, True),
    (24, 8, 128, [2500, 40], [85, 1], True, False, False),           # a token more than two tiles of 42
    (24, 8, 128, [2500, 40], [84, 1], True, False, True),            # two tiles, keys cut
    (7, 1, 64, [3860, 40], [108, 1], True, True, False), (4, 1, 128, [1500], [512], True, False, False),
    (8, 2, 128, [1000, 9, 100], [128, 1, 30], False, True, False), (1, 1, 64, [0], [1500], True, False, False),
])
def test_attention_long_chunks(daa, hq, hkv, d, cached, new, causal, exps, bf16):
    """Chunks by way of bf16 pages, and few ones that are read from the 4-bit pages."""
    attn, q, out, _, _ = _check(daa, np.random.default_rng(34), hq, hkv, d, cached, new, causal=causal, exps=exps)
    daa.trace_enable(16)
    try:
        again = attn.run(q.to(DEV))
        names = [n for n, _ in daa.trace_read()]
    finally:
        daa.trace_disable()
    assert ("kv_dequant_q4" in names) == bf16
    assert torch.equal(again, out)
