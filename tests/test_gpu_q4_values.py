"""Attention over the 4-bit cache where wrong values are small next to a context, or scales
leave fp32's range; and the places that step tables name, against what the append wrote there."""
import numpy as np
import pytest
import torch

import q4_bounds
import q4_support as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _pool(rng, n, hkv, d):
    return np.concatenate([rng.integers(0, 256, (n, hkv, 2, 8 * d), dtype=np.uint8),
                           rng.integers(40, 64, (n, hkv, 2, d), dtype=np.uint8)], -1)


def _table(daa, t):
    return daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).bfloat16()


@pytest.mark.parametrize("hq,hkv,d,cached,new,causal,bf16", [
    (2, 2, 128, [5003], [1], True, False), (4, 1, 128, [9001, 4095], [1, 1], True, False),
    (16, 1, 64, [3001], [4], True, False), (8, 1, 128, [2500], [3], True, False),
    (12, 4, 64, [1500, 700, 0], [1, 5, 3], True, False), (8, 1, 128, [700], [12], False, False),
    (7, 1, 64, [3860], [108], True, False),
    (24, 8, 64, [1700], [84], True, True), (32, 8, 64, [77], [500], True, True), (16, 4, 128, [100], [300], True, True),
])
def test_every_v_page_counts_once(daa, hq, hkv, d, cached, new, causal, bf16):
    """V zero but for one page, at every page in turn: left out, counted twice, negated or taken from elsewhere it is off
    by more than the bounds, which are relative to that page."""
    rng = np.random.default_rng(40 + hq)
    t, n = ref.make_table(rng, cached, new)
    pool = _pool(rng, n, hkv, d)
    q = _bf16(rng, (int(t["qo_indptr"][-1]), hq, d))
    scale = 1 / d ** 0.5
    B = ref.attention(q.double().numpy(), pool, t, None, d, scale, causal)[3].max()
    dev = _dev(pool)
    scales = dev[:, :, 1, 8 * d:].clone()
    dev[:, :, 1, 8 * d:] = 0
    attn = daa.BatchAttentionQ4(_table(daa, t), hq, dev, causal=causal)
    qd = q.to(DEV)
    daa.trace_enable(16)
    try:
        attn.run(qd)
        assert ("kv_dequant_q4" in [x for x, _ in daa.trace_read()]) == bf16
    finally:
        daa.trace_disable()
    for r in range(len(new)):
        rows = slice(t["qo_indptr"][r], t["qo_indptr"][r + 1])
        outs = []
        for page in t["page_indices"][t["kv_indptr"][r]:t["kv_indptr"][r + 1]].tolist():
            dev[page, :, 1, 8 * d:] = scales[page]
            out = attn.run(qd)
            dev[page, :, 1, 8 * d:] = 0
            outs.append(out[rows].clone())
            out[rows] = 0
            assert not out.any()  # nobody else's page
        want = q4_bounds.by_page(q.double().numpy(), pool, t, r, d, scale, causal)
        q4_bounds.check_by_page(torch.stack(outs).double().cpu().numpy(), want, B, d, q4_bounds.BF16 if bf16 else q4_bounds.FP16)


@pytest.mark.parametrize("size,scale,e,zero_keys", [
    (-122, None, -32, False), (-30, 2.0 ** -100, -32, False), (126, 2.0 ** -126, -20, False), (110, 2.0 ** -120, 12, False),
    (-100, 2.0 ** 100, -8, False), (-126, 2.9e38, -6, False), (100, 2.0 ** 20, 32, True), (120, 2.0 ** 120, 0, True),
])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 1), (6, 1)])
def test_scales_at_the_ends_of_their_range(daa, hq, hkv, size, scale, e, zero_keys):
    """Queries, sm_scale and exponents whose product leaves fp32's range or its normal numbers, in part or as a whole, while
    the scores themselves are ordinary or vanish."""
    rng = np.random.default_rng(41)
    d = 128
    t, n = ref.make_table(rng, [37, 5, 130], [1, 4, 3])
    pool = _pool(rng, n, hkv, d)
    if zero_keys:
        pool[:, :, 0, :8 * d] = 0
    exps = np.stack([np.full(hkv, e), np.arange(hkv) - 1]).astype(np.int32)
    q = _bf16(rng, (8, hq, d)).clamp(-1.9, 1.9).double() * 2.0 ** size
    q = q.bfloat16()
    attn = daa.BatchAttentionQ4(_table(daa, t), hq, _dev(pool), sm_scale=scale, kv_exp=_dev(exps))
    lse = torch.empty(8, hq, device=DEV)
    out = attn.run(q.to(DEV), lse=lse)
    used = 1 / d ** 0.5 if scale is None else float(np.float32(scale))
    want = ref.attention(q.double().numpy(), pool, t, exps, d, used)
    ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, d)


def test_slot_map_names_the_appended_rows(daa):
    """Every new token's quantised K and V at the page and slot that its step's table names."""
    rng = np.random.default_rng(42)
    hkv, d = 3, 64
    pool, cache = daa.PagePool(90, 5, 30), daa.new_q4_pool(90, hkv, d)
    exps = rng.integers(-3, 4, (2, hkv)).astype(np.int32)
    for slots, new in (([2, 0], [37, 1]), ([0, 3, 2], [16, 50, 1]), ([3, 0], [1, 9])):
        table = pool.step(slots, new)
        rows = sum(new)
        k, v = _bf16(rng, (rows, hkv, d)), _bf16(rng, (rows, hkv, d), 0.1)
        daa.kv_append_q4(k.to(DEV), v.to(DEV), cache, table.qo_indptr, table.page_indices, table.kv_indptr,
                         table.last_page_len, kv_exp=_dev(exps))
        page, slot = np.divmod(table.slot_map.cpu().numpy(), 16)
        got = daa.kv_dequant_q4(cache, _dev(page.astype(np.int32)), kv_exp=_dev(exps)).double().cpu().numpy()
        got = got[np.arange(rows), :, :, slot]  # [rows, 2, Hkv, d]
        for i, x in enumerate((k, v)):
            code, sc = ref.quantise(x.double().numpy(), np.broadcast_to(exps[i], (rows, hkv)))
            val = np.where(code >= 8, -1.0, 1.0) * ref.E2M1[code & 7] * np.repeat(ref.E4M3[sc], 16, -1) * 2.0 ** exps[i][:, None]
            assert np.array_equal(got[:, i], val)
