"""Rotary positions and the appends that apply them against float64 (rope_support), and against the framework's
own appends on the rotated rows, byte for byte."""
import numpy as np
import pytest
import torch

import q4_support
import rope_support as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = 0x7FC1  # of unused and stale slots: a NaN, as bits


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


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).bfloat16().to(DEV)


def _np(x):
    return x.double().cpu().numpy()


def _rows(rng, rows, hq, hk, d, how):
    """q, k, v rows: contiguous, views of one projection, heads interleaved as [q, k, v] (equal counts), or heads outermost."""
    if how == "fused":
        x = _bf16(rng, (rows, hq + 2 * hk, d))
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if how == "between":
        x = _bf16(rng, (rows, max(hq, hk), 3, d))
        return x[:, :hq, 0], x[:, :hk, 1], x[:, :hk, 2]
    if how == "heads":
        return tuple(_bf16(rng, (h, rows, d)).transpose(0, 1) for h in (hq, hk, hk))
    return tuple(_bf16(rng, (rows, h, d)) for h in (hq, hk, hk))


def _norms(rng, d, norm):
    return (_bf16(rng, (d,)), _bf16(rng, (d,))) if norm else (None, None)


def _check(got, x, pos, rope, weight, eps):
    w = None if weight is None else _np(weight)
    want = ref.rotate(_np(x), pos, rope.frequencies, rope.rotary_dim, rope.interleaved, rope.magnitude, w, eps)
    ref.check(_np(got), want, weight is not None)


@pytest.mark.parametrize("rows,hq,hk,d,rot,inter,norm,how", [
    (1, 1, 0, 64, 64, False, False, "flat"), (1, 1, 1, 128, 128, False, False, "fused"), (3, 4, 2, 64, 64, False, True, "flat"),
    (18, 4, 2, 64, 16, False, False, "fused"), (33, 12, 1, 128, 128, True, False, "fused"), (7, 5, 5, 128, 112, False, True, "fused"),
    (65, 3, 1, 64, 48, False, True, "heads"), (65, 3, 1, 64, 48, True, True, "between"), (257, 1, 0, 128, 128, False, False, "heads"),
    (300, 2, 1, 64, 16, True, False, "flat"), (1001, 7, 1, 64, 32, True, True, "fused"), (129, 32, 32, 128, 96, False, False, "between"),
    (2050, 64, 8, 128, 128, False, True, "fused"), (5003, 20, 4, 64, 32, True, False, "fused"), (40001, 1, 1, 64, 16, False, False, "flat"),
    (90001, 1, 0, 128, 128, False, True, "flat"),
])
def test_rows_against_64_bits(daa, rows, hq, hk, d, rot, inter, norm, how):
    rng = np.random.default_rng(rows + d + rot)
    q, k, _ = _rows(rng, rows, hq, max(hk, 1), d, how)
    k = k if hk else None
    rope = daa.Rope(d, 10000.0, rot, inter, dict(type="yarn", factor=8.0, original=4096))
    pos = rng.integers(0, 131072, rows).astype(np.int32)
    pos[:6] = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1_000_000])[:rows][:6]
    wq, wk = _norms(rng, d, norm)
    eps = 1e-5 if norm else 0.0
    kw = dict(q_norm=wq, k_norm=wk if hk else None, eps=eps)
    qo, ko = daa.apply_rope(q, k, _dev(pos), rope, **kw)
    assert qo.shape == q.shape and qo.is_contiguous() and (ko is None) == (k is None)
    at = np.unique(np.concatenate([np.arange(min(rows, 70)), rng.integers(0, rows, 300), [rows - 1]]))  # rows looked at
    idx = torch.from_numpy(at).to(DEV)
    _check(qo[idx], q[idx], pos[at], rope, wq, eps)
    if hk:
        _check(ko[idx], k[idx], pos[at], rope, wk, eps)
    # a row's result depends on the row alone: one at a time gives the same bits
    for r in (0, rows - 1):
        one, _ = daa.apply_rope(q[r:r + 1], None, _dev(pos[r:r + 1]), rope, q_norm=wq, eps=eps)
        assert torch.equal(one.view(torch.int16), qo[r:r + 1].view(torch.int16))
    # in place, for views of one matrix among them, with the other columns as they were
    q2, k2 = q.clone(), None
    if how in ("fused", "between"):
        base = q._base.clone()
        q2 = base.as_strided(q.shape, q.stride(), q.storage_offset())
        k2 = base.as_strided(k.shape, k.stride(), k.storage_offset()) if hk else None
        mine = torch.zeros_like(base, dtype=torch.bool)
        mine.as_strided(q.shape, q.stride(), q.storage_offset())[:] = True
        if hk:
            mine.as_strided(k.shape, k.stride(), k.storage_offset())[:] = True
        rest = base[~mine].clone()
    elif hk:
        k2 = k.clone()
    got = daa.apply_rope(q2, k2, _dev(pos), rope, q_out=q2, k_out=k2, **kw)
    assert got[0] is q2 and got[1] is k2
    assert torch.equal(q2.contiguous().view(torch.int16), qo.view(torch.int16))
    assert not hk or torch.equal(k2.contiguous().view(torch.int16), ko.view(torch.int16))
    if how in ("fused", "between"):
        assert torch.equal(base[~mine].view(torch.int16), rest.view(torch.int16))


@pytest.mark.parametrize("rows,hq,hk,d,rot,inter", [(5000, 12, 1, 128, 64, False), (5000, 13, 2, 128, 128, True), (4300, 12, 4, 128, 16, True),
                                                    (5000, 9, 0, 128, 112, False), (4257, 25, 5, 64, 32, False), (6001, 36, 6, 64, 64, True)])
def test_many_rows_give_the_bits_of_few(daa, rows, hq, hk, d, rot, inter):
    """Many rows of many heads and the same rows a few at a time go to different kernels: the same bits, and right ones."""
    rng = np.random.default_rng(rows + rot)
    q, k, _ = _rows(rng, rows, hq, max(hk, 1), d, "fused")
    k = k if hk else None
    rope = daa.Rope(d, 10000.0, rot, inter)
    pos = rng.integers(0, 131072, rows).astype(np.int32)
    p = _dev(pos)
    qo, ko = daa.apply_rope(q, k, p, rope)
    for a in range(0, rows, 499):
        b = min(a + 499, rows)
        qs, ks = daa.apply_rope(q[a:b], k[a:b] if hk else None, p[a:b], rope)
        assert torch.equal(qs.view(torch.int16), qo[a:b].view(torch.int16))
        assert not hk or torch.equal(ks.view(torch.int16), ko[a:b].view(torch.int16))
    at = rng.integers(0, rows, 60)
    _check(qo[torch.from_numpy(at).to(DEV)], q[torch.from_numpy(at).to(DEV)], pos[at], rope, None, 0.0)
    q2 = q.contiguous()  # in place
    daa.apply_rope(q2, None, p, rope, q_out=q2)
    assert torch.equal(q2.view(torch.int16), qo.view(torch.int16))


@pytest.mark.parametrize("scaling", [None, dict(type="linear", factor=4.0), dict(type="ntk", factor=8.0),
                                     dict(type="wavelength", factor=8.0, original=8192)])
def test_scalings_and_far_positions(daa, scaling):
    rng = np.random.default_rng(1)
    rope = daa.Rope(128, 500000.0, scaling=scaling, magnitude=0.75)
    pos = np.concatenate([np.arange(64) * 40_000_003 - 2 ** 30, rng.integers(-2 ** 31, 2 ** 31, 200)]).astype(np.int32)
    x = _bf16(rng, (264, 3, 128), 30.0)
    got, _ = daa.apply_rope(x, None, _dev(pos), rope)
    _check(got, x, pos, rope, None, 0.0)


def test_broadcast_rows(daa):
    """One head for all heads and one row for all rows, by strides of zero."""
    rng = np.random.default_rng(2)
    rope = daa.Rope(64)
    x = _bf16(rng, (1, 1, 64))
    pos = np.arange(50).astype(np.int32)
    got, ko = daa.apply_rope(x.expand(50, 6, 64), x.expand(50, 2, 64), _dev(pos), rope)
    want, _ = daa.apply_rope(x.expand(50, 6, 64).contiguous(), None, _dev(pos), rope)
    assert torch.equal(got, want) and torch.equal(ko, want[:, :2])


@pytest.mark.parametrize("inter", [False, True])
def test_transposed(daa, inter):
    """Negated positions are the transposed rotation, what a gradient takes: the products <g, R x> and <R^T g, x> agree, and R^T g
    is the gradient of <g, R x> by differences in float64."""
    rng = np.random.default_rng(3)
    rope = daa.Rope(64, rotary_dim=48, interleaved=inter, magnitude=1.25)
    pos = rng.integers(0, 9000, 40).astype(np.int32)
    x, g = _bf16(rng, (40, 3, 64)), _bf16(rng, (40, 3, 64))
    back, _ = daa.apply_rope(g, None, _dev(-pos), rope)
    _check(back, g, -pos, rope, None, 0.0)
    args = (rope.frequencies, 48, inter, rope.magnitude)
    xs, gs = _np(x), _np(g)
    grad, step = np.zeros_like(xs), 2.0 ** -10
    for i in range(64):
        up, down = xs.copy(), xs.copy()
        up[..., i] += step
        down[..., i] -= step
        # the function is linear: differences are exact but for float64's roundings, 2^-40 of the values
        grad[..., i] = ((ref.rotate(up, pos, *args)[0] - ref.rotate(down, pos, *args)[0]) * gs).sum(-1) / (2 * step)
    size = ref.rotate(gs, -pos, *args)[1]
    tol = size * 2.0 ** -21 + 2.0 ** -8 * (np.abs(grad) + size * 2.0 ** -21) + 2.0 ** -38
    assert (np.abs(_np(back) - grad) <= tol).all()


@pytest.mark.parametrize("inter", [False, True])
def test_values_that_are_no_numbers(daa, inter):
    """Infinities and NaN stay within their pair; what is not rotated keeps its bits, payloads too."""
    rng = np.random.default_rng(4)
    d, rot = 64, 32
    rope = daa.Rope(d, rotary_dim=rot, interleaved=inter)
    x = _bf16(rng, (9, 2, d))
    bits = x.view(torch.int16)
    clean = x.clone()
    bits[3, 1, 5] = 0x7F80  # infinity
    bits[4, 0, 7] = 0x7FC1
    bits[5, 0, rot:] = torch.arange(0x7F81, 0x7F81 + d - rot, dtype=torch.int16, device=DEV)  # NaNs, each its own
    bits[6, 1, rot] = -0x80  # -infinity
    pos = _dev(np.arange(9).astype(np.int32))
    got, _ = daa.apply_rope(x, None, pos, rope)
    want, _ = daa.apply_rope(clean, None, pos, rope)
    mates = lambda i: ([i, i ^ 1] if inter else [i, (i + rot // 2) % rot])  # noqa: E731
    odd = torch.zeros(9, 2, d, dtype=torch.bool)
    odd[3, 1, mates(5)] = odd[4, 0, mates(7)] = True
    odd[5, 0, rot:] = odd[6, 1, rot] = True
    odd = odd.to(DEV)
    assert torch.equal(got[~odd], want[~odd])
    assert torch.equal(got.view(torch.int16)[..., rot:], bits[..., rot:])
    assert not got[3, 1, mates(5)].isfinite().any() and got[4, 0, mates(7)].isnan().all()
    # a zero position turns by nothing, and infinity times zero is no number: as the formula says
    y, _ = daa.apply_rope(x[3:4], None, pos[:1], rope)
    assert torch.isinf(y[0, 1, 5]) and y[0, 1, [m for m in mates(5) if m != 5][0]].isnan()


def test_norm_of_zeros_and_large_heads(daa):
    rng = np.random.default_rng(5)
    rope = daa.Rope(64)
    x = _bf16(rng, (6, 2, 64))
    x[0] = 0
    x[1] *= 2.0 ** 50
    x[2] *= 2.0 ** -60
    w = _bf16(rng, (64,))
    pos = np.arange(6).astype(np.int32)
    got, _ = daa.apply_rope(x, None, _dev(pos), rope, q_norm=w, eps=1e-6)
    assert not got[0].any()
    _check(got, x, pos, rope, w, 1e-6)
    got, _ = daa.apply_rope(x[1:], None, _dev(pos[1:]), rope, q_norm=w, eps=0.0)
    _check(got, x[1:], pos[1:], rope, w, 0.0)


def test_one_norm_of_two(daa):
    rng = np.random.default_rng(6)
    rope = daa.Rope(128, rotary_dim=64)
    q, k, _ = _rows(rng, 21, 6, 2, 128, "fused")
    pos = _dev(np.arange(21).astype(np.int32) * 3)
    w = _bf16(rng, (128,))
    q0, k0 = daa.apply_rope(q, k, pos, rope)
    q1, k1 = daa.apply_rope(q, k, pos, rope, k_norm=w)
    q2, k2 = daa.apply_rope(q, k, pos, rope, q_norm=w)
    q3, k3 = daa.apply_rope(q, k, pos, rope, q_norm=w, k_norm=w)
    assert torch.equal(q0, q1) and torch.equal(k0, k2) and torch.equal(q2, q3) and torch.equal(k1, k3)
    assert not torch.equal(k0, k1) and not torch.equal(q0, q2)


def test_overlaps_are_refused(daa):
    rng = np.random.default_rng(7)
    rope, pos = daa.Rope(64), _dev(np.arange(8).astype(np.int32))
    x = _bf16(rng, (8, 6, 64))
    before = x.clone()
    y = torch.empty(8, 4, 64, dtype=torch.bfloat16, device=DEV)
    for q, k, qo, ko in ((x[:, :4], x[:, 4:], y, x[:, 3:5]), (x[:, :4], None, x[:, 1:5], None), (x[:, :2], x[:, 4:], x[:, 4:], x[:, 2:4]),
                         (x[:, :4], x[:, 4:], y, y[:, :2]), (y, x[:, 4:], x[:, :4], x[:, :2])):
        with pytest.raises(daa.DaaError) as e:
            daa.apply_rope(q, k, pos, rope, q_out=qo, k_out=ko)
        assert e.value.status == -1
    assert torch.equal(x, before)
    daa.apply_rope(x[:, :2], x[:, 4:], pos, rope, q_out=x[:, 2:4], k_out=x[:, 4:])  # beside one another
    want, _ = daa.apply_rope(before, None, pos, rope)
    assert torch.equal(x[:, 2:4], want[:, :2]) and torch.equal(x[:, 4:], want[:, 4:]) and torch.equal(x[:, :2], before[:, :2])


# ------------------------------------------------------------------- appends
APPENDS = [
    # hq, hk, d, rot, interleaved, norm, rows' layout, cached, new
    (4, 2, 64, 64, False, False, "flat", [48, 39, 72], [16, 1, 1]),
    (1, 1, 64, 16, False, False, "fused", [0], [1]),
    (12, 1, 128, 128, False, False, "fused", [1023, 5, 4096, 0, 31, 15, 16, 17], [1] * 8),
    (32, 8, 128, 128, False, True, "fused", [100, 7, 0], [5, 5, 5]),
    (15, 5, 64, 16, False, True, "flat", [777, 777, 3, 0], [333, 17, 3, 0]),
    (8, 8, 128, 112, False, False, "between", [0, 20, 0], [0, 41, 0]),
    (6, 2, 64, 48, True, False, "heads", [1, 2, 3], [64, 15, 33]),
    (16, 1, 128, 32, True, True, "fused", [200, 0], [2, 90]),
    (5, 5, 128, 48, False, False, "fused", [11, 1000], [37, 1]),
    (64, 8, 128, 128, False, False, "fused", [8192, 77], [1500, 1]),
    (20, 4, 64, 64, False, True, "fused", [0, 901], [5003, 1]),
    (2, 1, 64, 32, False, False, "flat", [3 + i % 40 for i in range(2000)], [1 + i % 3 // 2 for i in range(2000)]),
    (1, 1, 64, 16, False, False, "fused", [i % 50 for i in range(20000)], [(i * 7 % 5) // 3 for i in range(20000)]),
    (3, 1, 64, 64, True, False, "fused", [i % 50 for i in range(257)], [1] * 257),
    (16, 16, 64, 64, False, True, "fused", [0, 70], [0, 1300]),
    # many rows of few heads
    (12, 1, 128, 128, False, False, "fused", [900, 3], [2501, 1]), (8, 1, 128, 128, False, True, "flat", [0, 30], [2000, 700]),
    (3, 1, 128, 48, False, True, "fused", [17], [2600]), (6, 2, 64, 48, True, False, "heads", [5, 1], [2700, 3]),
]


def _case(daa, hq, hk, d, rot, inter, norm, how, cached, new):
    rng = np.random.default_rng(hq + d + rot + len(new))
    t, n = q4_support.make_table(rng, cached, new)
    rows = int(t["qo_indptr"][-1])
    q, k, v = _rows(rng, rows, hq, hk, d, how)
    wq, wk = _norms(rng, d, norm)
    rope = daa.Rope(d, 10000.0, rot, inter, dict(type="wavelength", factor=8.0, original=512))
    return t, n, q, k, v, wq, wk, rope, rng


def _dev_table(t):
    return [_dev(t[x]) for x in ("qo_indptr", "page_indices", "kv_indptr", "last_page_len")]


def _nan_pool(n, hk, d):
    return torch.full((n, 2, hk, 16, d), NAN, dtype=torch.int16, device=DEV).view(torch.bfloat16)


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}r{c[3]}")
def test_append(daa, case):
    hq, hk, d, rot, inter, norm, how, cached, new = case
    t, n, q, k, v, wq, wk, rope, rng = _case(daa, *case)
    place = ref.places(t)
    pos = _dev(place[:, 3].astype(np.int32))
    eps = 1e-6
    q_want, k_want = daa.apply_rope(q, k, pos, rope, q_norm=wq, k_norm=wk, eps=eps)  # held to float64 by the tests above
    at = rng.integers(0, len(place), 40)
    _check(k_want[torch.from_numpy(at).to(DEV)], k[torch.from_numpy(at).to(DEV)], place[at, 3], rope, wk, eps)
    want = _nan_pool(n, hk, d)
    wb, kb, vb = (x.view(torch.int16) for x in (want, k_want, v.contiguous()))
    wb[place[:, 1], 0, :, place[:, 2]] = kb
    wb[place[:, 1], 1, :, place[:, 2]] = vb
    pool = _nan_pool(n, hk, d)
    q_out = daa.append_rope(q, k, v, pool, *_dev_table(t), rope, q_norm=wq, k_norm=wk, eps=eps)
    assert torch.equal(q_out.view(torch.int16), q_want.view(torch.int16))
    assert torch.equal(pool.view(torch.int16), wb)
    # the same through kv_append, and without query rows
    daa.kv_append(k_want, v.contiguous(), pool, *_dev_table(t))
    assert torch.equal(pool.view(torch.int16), wb)
    pool = _nan_pool(n, hk, d)
    assert daa.append_rope(None, k, v, pool, *_dev_table(t), rope, k_norm=wk, eps=eps) is None
    assert torch.equal(pool.view(torch.int16), wb)


def _exact_keys(k, pos, rope, weight, eps=float(np.float32(1e-6))):
    y, _ = ref.rotate(_np(k), pos, rope.frequencies, rope.rotary_dim, rope.interleaved, rope.magnitude, None if weight is None else _np(weight), eps)
    y = torch.from_numpy(y).float().bfloat16().to(DEV)
    if weight is None:
        y[..., rope.rotary_dim:] = k[..., rope.rotary_dim:]
    return y


@pytest.mark.parametrize("exps", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}r{c[3]}")
def test_append_q4(daa, case, exps):
    hq, hk, d, rot, inter, norm, how, cached, new = case
    t, n, q, k, v, wq, wk, rope, rng = _case(daa, *case)
    at = ref.places(t)[:, 3]
    pos = _dev(at.astype(np.int32))
    e = rng.integers(-3, 4, (2, hk)).astype(np.int32)
    e_dev = _dev(e) if exps else None
    q_want, _ = daa.apply_rope(q, None, pos, rope, q_norm=wq)
    # keys by the definition alone, to fp32's nearest and then to bf16: bytes, not bounds
    k_want = _exact_keys(k, at, rope, wk)
    want = torch.full((n, hk, 2, 9 * d), 0xAB, dtype=torch.uint8, device=DEV)
    pool = want.clone()
    daa.kv_append_q4(k_want, v.contiguous(), want, *_dev_table(t), kv_exp=e_dev)
    q_out = daa.append_rope_q4(q, k, v, pool, *_dev_table(t), rope, kv_exp=e_dev, q_norm=wq, k_norm=wk)
    assert torch.equal(q_out.view(torch.int16), q_want.view(torch.int16))
    assert torch.equal(pool, want)
    if len(pos) < 500:  # and by the definition
        host = np.full((n, hk, 2, 9 * d), 0xAB, np.uint8)
        q4_support.append(host, _np(k_want), _np(v), t, e if exps else None)
        assert np.array_equal(pool.cpu().numpy(), host)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (64, 32, False)])
@pytest.mark.parametrize("at", [131_072, 2 ** 24 - 40])
def test_keys_of_far_positions_into_4_bits(daa, at, d, rot, inter, norm):
    """Byte for byte the definition's.  Angles off by 2^-36.7 together move a key to another bf16 value at one in some 2^27."""
    rng = np.random.default_rng(26)
    t, n = q4_support.make_table(rng, [0], [40])
    q, k, v = _rows(rng, 40, 4, 4, d, "fused")
    wk = _norms(rng, d, norm)[1]
    rope = daa.Rope(d, 500000.0, rot, inter, dict(type="yarn", factor=16.0, original=4096))
    pos = (at + np.arange(40)).astype(np.int32)
    pool, want = daa.new_q4_pool(n, 4, d), daa.new_q4_pool(n, 4, d)
    daa.append_rope_q4(q, k, v, pool, *_dev_table(t), rope, positions=_dev(pos), k_norm=wk)
    daa.kv_append_q4(_exact_keys(k, pos, rope, wk), v.contiguous(), want, *_dev_table(t))
    assert torch.equal(pool, want)


@pytest.mark.parametrize("q4", [False, True])
def test_given_positions_turn_but_do_not_place(daa, q4):
    """A draft tree's depths: rows go to the slots of their order, at the angles of the positions given."""
    rng = np.random.default_rng(8)
    t, n = q4_support.make_table(rng, [30, 7], [7, 6])
    q, k, v = _rows(rng, 13, 8, 2, 128, "fused")
    rope = daa.Rope(128)
    place = ref.places(t)
    depth = np.array([(i + 1).bit_length() - 1 for i in range(7)])
    pos = np.concatenate([30 + depth, 7 + depth[:6]]).astype(np.int32)
    q_want, k_want = daa.apply_rope(q, k, _dev(pos), rope)
    if q4:
        k_want = _exact_keys(k, pos, rope, None)
        pool, want = daa.new_q4_pool(n, 2, 128), daa.new_q4_pool(n, 2, 128)
        got = daa.append_rope_q4(q, k, v, pool, *_dev_table(t), rope, positions=_dev(pos))
        daa.kv_append_q4(k_want, v.contiguous(), want, *_dev_table(t))
        assert torch.equal(pool, want)
    else:
        pool = _nan_pool(n, 2, 128)
        got = daa.append_rope(q, k, v, pool, *_dev_table(t), rope, positions=_dev(pos))
        assert torch.equal(pool[place[:, 1], 0, :, place[:, 2]], k_want)
    assert torch.equal(got, q_want)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("live", [[], [3], [1, 0, 20], [40]])
def test_rows_behind_the_last_request_are_padding(daa, q4, live):
    """Buffers of 40 rows of which a step uses fewer: the rest of the outputs and the pool stay as they were, with no error."""
    rng = np.random.default_rng(9)
    new = live or [0]
    t, n = q4_support.make_table(rng, [17] * len(new), new)
    q, k, v = _rows(rng, 40, 4, 2, 64, "fused")
    rope, rows = daa.Rope(64), sum(new)
    pool = daa.new_q4_pool(n, 2, 64) if q4 else _nan_pool(n, 2, 64)
    want = pool.clone()
    out = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    call = daa.append_rope_q4 if q4 else daa.append_rope
    got = call(q, k, v, pool, *_dev_table(t), rope, q_out=out)
    assert got is out and (out[rows:] == 7).all()
    assert daa.device_error(reset=True) == 0
    if rows:
        alone = call(q[:rows], k[:rows], v[:rows], want, *_dev_table(t), rope)
        assert torch.equal(out[:rows], alone)
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("q4", [False, True])
def test_bad_pages_and_lengths(daa, q4):
    """A page id outside the pool: its rows' k and v are not written and the error word says so; lengths that cannot be: nothing
    of that request is.  The others are as ever."""
    rng = np.random.default_rng(10)
    t, n = q4_support.make_table(rng, [10, 3, 40], [12, 5, 2])
    q, k, v = _rows(rng, 19, 4, 2, 64, "flat")
    rope = daa.Rope(64)
    call = daa.append_rope_q4 if q4 else daa.append_rope
    new_pool = (lambda: daa.new_q4_pool(n, 2, 64)) if q4 else (lambda: _nan_pool(n, 2, 64))
    good, place = new_pool(), ref.places(t)
    q_want = call(q, k, v, good, *_dev_table(t), rope)
    slot_of = (lambda p, page, s: p[page, :, :, s * 32:(s + 1) * 32]) if q4 else (lambda p, page, s: p.view(torch.int16)[page, :, :, s])
    for bad in (-1, n, 2 ** 31 - 1):
        b = {x: y.copy() for x, y in t.items()}
        b["page_indices"][t["kv_indptr"][0] + 1] = bad  # rows 6 .. 11 (positions 16 .. 21)
        pool, fresh = new_pool(), new_pool()
        got = call(q, k, v, pool, *_dev_table(b), rope)
        assert daa.device_error(reset=True) == 1
        assert torch.equal(got, q_want)
        for row, page, s, _ in place.tolist():
            src = fresh if 6 <= row < 12 else good
            assert torch.equal(slot_of(pool, page, s), slot_of(src, page, s)), row
    for change in (dict(last_page_len=(1, 17)), dict(last_page_len=(1, 0)), dict(last_page_len=(1, -5)), dict(kv_indptr=None)):
        b = {x: y.copy() for x, y in t.items()}
        if "last_page_len" in change:
            i, to = change["last_page_len"]
            b["last_page_len"][i] = to
        else:
            b["kv_indptr"][2] = b["kv_indptr"][1]  # request 1 owns no page (and request 2 one more)
        pool, out = new_pool(), torch.full((19, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        call(q, k, v, pool, *_dev_table(b), rope, q_out=out)
        assert daa.device_error(reset=True) == 3
        assert (out[12:17] == 7).all() and torch.equal(out[:12], q_want[:12])
        for row, page, s, _ in place.tolist():
            if row < 12:
                assert torch.equal(slot_of(pool, page, s), slot_of(good, page, s))


def test_page_lists_that_end_too_early(daa):
    """kv_indptr that goes on past its own end: nothing behind it is read, and the request's rows are refused."""
    rng = np.random.default_rng(21)
    t, n = q4_support.make_table(rng, [20, 20], [4, 4])
    q, k, v = _rows(rng, 8, 4, 2, 64, "flat")
    rope, pool = daa.Rope(64), _nan_pool(n, 2, 64)
    b = {x: y.copy() for x, y in t.items()}
    b["kv_indptr"][1] = 10 ** 6  # request 0 owns a million pages, of four
    out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    daa.append_rope(q, k, v, pool, *_dev_table(b), rope, q_out=out)
    assert daa.device_error(reset=True) == 3
    assert (out == 7).all() and (pool.view(torch.int16) == NAN).all()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("how", ["flat", "fused", "heads"])
def test_append_in_place(daa, q4, how):
    """The rotated queries in the place of the given ones, k and v beside them untouched."""
    rng = np.random.default_rng(22)
    t, n = q4_support.make_table(rng, [20, 300], [50, 1])
    q, k, v = _rows(rng, 51, 6, 2, 128, how)
    rope, tab = daa.Rope(128, rotary_dim=96), _dev_table(t)
    call = daa.append_rope_q4 if q4 else daa.append_rope
    pool = daa.new_q4_pool(n, 2, 128) if q4 else _nan_pool(n, 2, 128)
    want, k0, v0 = pool.clone(), k.clone(), v.clone()
    q_want = call(q, k, v, want, *tab, rope)
    assert call(q, k, v, pool, *tab, rope, q_out=q) is q
    assert torch.equal(q, q_want) and torch.equal(k, k0) and torch.equal(v, v0)
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("inter,rot", [(False, 32), (True, 32), (False, 64), (True, 64), (False, 48), (True, 48)])
@pytest.mark.parametrize("norm", [False, True])
def test_keys_that_are_no_numbers_into_4_bits(daa, norm, inter, rot):
    """As the cache stores them: NaN as zero, infinities as the largest values, rotated first; and keys of any size."""
    rng = np.random.default_rng(23)
    t, n = q4_support.make_table(rng, [3], [6])
    tab, rope = _dev_table(t), daa.Rope(64, rotary_dim=rot, interleaved=inter)
    q, k, v = _rows(rng, 6, 2, 1, 64, "flat")
    k.view(torch.int16)[1, 0, 40] = 0x7F80  # rotated or not
    k.view(torch.int16)[2, 0, 3] = -0x80
    k.view(torch.int16)[3, 0, 50] = 0x7FC1
    k[4] *= 2.0 ** 101
    k[5] *= 2.0 ** -101
    v.view(torch.int16)[0, 0, 9] = 0x7F80
    pos = _dev(ref.places(t)[:, 3].astype(np.int32))
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV) if norm else None
    pool, want = daa.new_q4_pool(n, 1, 64), daa.new_q4_pool(n, 1, 64)
    daa.append_rope_q4(q, k, v, pool, *tab, rope, q_norm=w)  # the norm is q's alone
    _, k_want = daa.apply_rope(q, k, pos, rope)
    exact = _exact_keys(k[[0, 5]], ref.places(t)[[0, 5], 3], rope, None)
    k_want[[0, 5]] = exact
    daa.kv_append_q4(k_want, v, want, *tab)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("inter,rot", [(False, 64), (True, 64), (False, 32), (True, 32)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("weights", [None, 1.0, 2.0 ** 100, 2.0 ** -30])
def test_normed_keys_of_any_size_into_4_bits(daa, weights, eps, inter, rot):
    """Keys that are normalised on their way: heads with a NaN or an infinity, of zeros, of large and small values and of both,
    under ordinary, large and small weights, against the definition in 64 bits (values: a zero's sign is open)."""
    rng = np.random.default_rng(25)
    t, n = q4_support.make_table(rng, [3], [9])
    tab, rope = _dev_table(t), daa.Rope(64, rotary_dim=rot, interleaved=inter)
    q, k, v = _rows(rng, 9, 2, 1, 64, "flat")
    k.view(torch.int16)[1, 0, 40] = 0x7F80  # rotated or not
    k.view(torch.int16)[2, 0, 3] = -0x80
    k.view(torch.int16)[3, 0, 50] = 0x7FC1
    k[4] = 0
    k[5] *= 2.0 ** 50
    k[6] *= 2.0 ** -60
    k[7, 0, :32] *= 2.0 ** -40
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV) if weights is None else _bf16(rng, (64,), weights)
    place = ref.places(t)
    with np.errstate(invalid="ignore", divide="ignore"):
        k_want = _exact_keys(k, place[:, 3], rope, w, float(np.float32(eps)))
    pool, want = daa.new_q4_pool(n, 1, 64), daa.new_q4_pool(n, 1, 64)
    daa.append_rope_q4(q, k, v, pool, *tab, rope, k_norm=w, eps=eps)
    daa.kv_append_q4(k_want, v, want, *tab)
    ids = _dev(np.arange(n, dtype=np.int32))
    got, want = daa.kv_dequant_q4(pool, ids), daa.kv_dequant_q4(want, ids)
    for row, page, slot, _ in place.tolist():
        assert torch.equal(got[page, :, :, slot], want[page, :, :, slot]), row


@pytest.mark.parametrize("q4", [False, True])
def test_pages_and_rows_past_32_bits(daa, q4):
    """The last page of a pool of more than 2^32 bytes and values, and rows more than 2^31 elements apart."""
    rng = np.random.default_rng(24)
    hk, d = 16, 128
    n = (1 << 32) // (hk * 2 * (9 * d if q4 else 16 * d)) + 3
    pool = torch.empty(n, hk, 2, 9 * d, dtype=torch.uint8, device=DEV) if q4 else torch.empty(n, 2, hk, 16, d, dtype=torch.bfloat16, device=DEV)
    assert pool.numel() > 1 << 32
    pool[[0, n - 2, n - 1]] = 0
    i32 = lambda x: _dev(np.array(x, np.int32))  # noqa: E731
    tab = i32([0, 2]), i32([n - 1, n - 2]), i32([0, 2]), i32([1])
    far = (1 << 31) + 8
    x = torch.empty(far + 18 * d, dtype=torch.bfloat16, device=DEV)
    rows = _bf16(rng, (2, 48, d))
    q, k, v = (x.as_strided((2, h, d), (far, d, 1), o * d) for h, o in ((16, 0), (1, 16), (1, 17)))
    k, v = k.expand(2, hk, d), v.expand(2, hk, d)
    q.copy_(rows[:, :16])
    k[:, :1].copy_(rows[:, 16:17])
    v[:, :1].copy_(rows[:, 17:18])
    rope = daa.Rope(d)
    call = daa.append_rope_q4 if q4 else daa.append_rope
    got = call(q, k, v, pool, *tab, rope)
    small = torch.zeros_like(pool[:2])
    want = call(q.contiguous(), k.contiguous(), v.contiguous(), small, tab[0], i32([1, 0]), *tab[2:], rope)
    assert torch.equal(got, want) and torch.equal(pool[n - 2:], small) and not pool[0].any()
    daa.append_rope(q, k, v, pool, *tab, rope, q_out=q) if not q4 else daa.append_rope_q4(q, k, v, pool, *tab, rope, q_out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("q4", [False, True])
def test_empty_calls(daa, q4):
    rope = daa.Rope(64)
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = x[:, :2]
    i32 = dict(dtype=torch.int32, device=DEV)
    qo, ko = daa.apply_rope(x, k, torch.empty(0, **i32), rope)
    assert qo.shape == x.shape and ko.shape == k.shape
    pool = daa.new_q4_pool(4, 2, 64) if q4 else _nan_pool(4, 2, 64)
    call = daa.append_rope_q4 if q4 else daa.append_rope
    table = torch.zeros(2, **i32), torch.empty(0, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    assert call(x, k, k, pool, *table, rope).shape == x.shape
    with pytest.raises(daa.DaaError):  # rows of no request
        y = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
        call(y, y[:, :2], y[:, :2], pool, torch.zeros(1, **i32), torch.empty(0, **i32), torch.zeros(1, **i32), torch.empty(0, **i32), rope)


def test_argument_refusals(daa):
    rng = np.random.default_rng(11)
    rope = daa.Rope(64)
    t, n = q4_support.make_table(rng, [3], [2])
    q, k, v = _rows(rng, 2, 4, 2, 64, "flat")
    pool, tab = _nan_pool(n, 2, 64), _dev_table(t)
    pos = _dev(np.arange(2).astype(np.int32))
    for err, args, kw in (
            (TypeError, (q.float(), k, v), {}), (TypeError, (q, k.cpu(), v), {}), (ValueError, (q, k[:1], v), {}), (ValueError, (q, k, v[:, :1]), {}),
            (ValueError, (q[:1], k, v), {}), (ValueError, (q[..., ::2], k, v), {}), (ValueError, (q, k, v), dict(positions=pos[:1])),
            (TypeError, (q, k, v), dict(positions=pos.long())), (ValueError, (q, k, v), dict(q_norm=torch.ones(63, dtype=torch.bfloat16, device=DEV))),
            (TypeError, (q, k, v), dict(k_norm=torch.ones(64, device=DEV))), (ValueError, (None, k, v), dict(q_out=q)), (ValueError, (q, k, v), dict(q_out=k)),
            (ValueError, (q, k, v), dict(rope=daa.Rope(128))), (TypeError, (q, k, v), dict(rope=None)), (daa.DaaError, (q[:, :3], k, v), {}),
            (daa.DaaError, (q, k, v), dict(k_norm=torch.ones(64, dtype=torch.bfloat16, device=DEV), eps=-1.0))):
        with pytest.raises(err):
            daa.append_rope(*args, pool, *tab, **{"rope": rope, **kw})
    for err, args, kw in ((TypeError, (q, k, pos.long(), rope), {}), (ValueError, (q, k, pos[:1], rope), {}), (ValueError, (q, None, pos, rope), dict(k_out=k)),
                          (ValueError, (q[0], None, pos, rope), {}), (ValueError, (q, k, pos, daa.Rope(128)), {})):
        with pytest.raises(err):
            daa.apply_rope(*args, **kw)
    # 16-byte strides and addresses
    odd = torch.zeros(2 * 4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    for x in (odd[4:4 + 512].view(2, 4, 64), odd.as_strided((2, 4, 64), (260, 64, 1))):
        with pytest.raises(daa.DaaError) as e:
            daa.apply_rope(x, None, pos, rope)
        assert e.value.status == -7


# ------------------------------------------------------------- with attention
def _attend(q, keys, values, cached, scale):
    """float64 causal attention of one request: q [new, Hq, d] over [kv, Hkv, d]."""
    g = q.shape[1] // keys.shape[1]
    out = np.zeros(q.shape)
    for i in range(len(q)):
        for h in range(q.shape[1]):
            s = keys[:cached + i + 1, h // g] @ q[i, h] * scale
            w = np.exp(s - s.max())
            out[i, h] = w @ values[:cached + i + 1, h // g] / w.sum()
    return out


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_steps_over_a_growing_cache(daa, q4, norm):
    """Prompts in chunks, then single tokens, through PagePool and step_rope: what attention gives against float64 over all tokens'
    rotated keys at their absolute positions."""
    rng = np.random.default_rng(12)
    hq, hk, d, num = 8, 2, 64, 64
    rope = daa.Rope(d, rotary_dim=32, scaling=dict(type="linear", factor=2.0))
    pages = daa.new_q4_pool(num, hk, d) if q4 else _nan_pool(num, hk, d)
    pool = daa.PagePool(num, 4, 20)
    wq, wk = _norms(rng, d, norm)
    kw = dict(q_norm=wq, k_norm=wk, eps=1e-6)
    seen = {0: ([], []), 2: ([], [])}
    for slots, new in (([0, 2], [19, 40]), ([2], [33]), ([0, 2], [1, 1]), ([2, 0], [1, 5]), ([0], [1])):
        table = pool.step(slots, new)
        q, k, v = _rows(rng, sum(new), hq, hk, d, "fused")
        attn = (daa.BatchAttentionQ4 if q4 else daa.BatchAttention)(table, hq, pages)
        if new[0] == 1:
            attn.plan()
        lse = torch.empty(sum(new), hq, device=DEV)
        out = attn.step_rope(q, k, v, rope, lse=lse, **kw)
        # by the single calls: the same
        q_rot, k_rot = daa.apply_rope(q, k, table.positions, rope, **kw)
        assert torch.equal(attn.run(q_rot), out)
        row = 0
        for slot, n in zip(slots, new):
            sl = slice(row, row + n)
            cached = len(seen[slot][0])
            pos = np.arange(cached, cached + n)
            kk, _ = ref.rotate(_np(k[sl]), pos, rope.frequencies, 32, False, 1.0, _np(wk) if norm else None, 1e-6)
            if q4:  # the cache's own values: its rounding is another test's
                page, s = np.divmod(table.slot_map.cpu().numpy()[sl], 16)
                back = _np(daa.kv_dequant_q4(pages, _dev(page.astype(np.int32))))[np.arange(n), :, :, s]
                assert np.abs(back[:, 0] - kk).max() <= np.abs(kk).max() * (1 / 6 + 1 / 16 + 2.0 ** -7)
                kk, vv = back[:, 0], back[:, 1]
            else:
                vv = _np(v[sl])
            seen[slot][0].extend(kk)
            seen[slot][1].extend(vv)
            qq, _ = ref.rotate(_np(q[sl]), pos, rope.frequencies, 32, False, 1.0, _np(wq) if norm else None, 1e-6)
            keys, values = np.array(seen[slot][0]), np.array(seen[slot][1])
            want = _attend(qq, keys, values, cached, d ** -0.5)
            # q and k are bf16 by then: scores off by at most 2 * 2^-8 of sum |q k| (4 2^-9, and 2^-16 for their fp32), weights
            # by twice that and their own rounding (2^-8); the output's rounding 2^-8
            big = np.einsum("thd,khd->thk", np.abs(qq), np.abs(np.repeat(keys, hq // hk, 1))).max(-1)[..., None] * d ** -0.5
            dw = np.exp(2 * big * (2.0 ** -7 + 2.0 ** -15)) - 1 + 2.0 ** -8
            size = _attend_abs(qq, keys, values, cached, d ** -0.5)
            tol = 2.0 ** -8 * np.abs(want) + 2 * dw * size
            assert (np.abs(_np(out[sl]) - want) <= tol).all()
            row += n


def _attend_abs(q, keys, values, cached, scale):
    return _attend(q, keys, np.abs(values), cached, scale)


@pytest.mark.parametrize("q4", [False, True])
def test_positions_matter_by_their_distance_alone(daa, q4):
    """All positions of a step later by the same number: queries and keys turn together, and attention stays what it was to bf16."""
    rng = np.random.default_rng(13)
    hq, hk, d = 4, 1, 128
    t, n = q4_support.make_table(rng, [0], [60])
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    q, k, v = _rows(rng, 60, hq, hk, d, "fused")
    rope = daa.Rope(d)
    outs = []
    for shift in (0, 100_000):
        pages = daa.new_q4_pool(n, hk, d) if q4 else _nan_pool(n, hk, d)
        attn = (daa.BatchAttentionQ4 if q4 else daa.BatchAttention)(table, hq, pages)
        outs.append(attn.step_rope(q, k, v, rope, positions=_dev((np.arange(60) + shift).astype(np.int32))).double())
    far = (outs[0] - outs[1]).norm() / outs[0].norm()
    # bf16 keys: scores off by 2 2^-8 sum |q k| / sqrt d ~ 2^-7 * 128 * 0.64 / 11.3 = 0.06 at most, about sqrt(128) times less
    # in the mean (0.006); 4-bit keys are off by up to a sixth of their block's maximum, about 0.1 of a key in the mean
    assert far < (0.4 if q4 else 0.03)


def test_tree_verify_step(daa):
    """A draft tree: positions by depth, the ancestors' mask, against float64."""
    rng = np.random.default_rng(14)
    hq, hk, d, nodes, cached = 4, 2, 64, 7, 29
    n, pages = 9, -(-(cached + nodes) // 16)
    ids = rng.permutation(n)[:pages].astype(np.int32)
    first = daa.PageTable.from_host([0, cached], [0, -(-cached // 16)], ids[:-(-cached // 16)], [(cached - 1) % 16 + 1], DEV)
    table = daa.PageTable.from_host([0, nodes], [0, pages], ids, [(cached + nodes - 1) % 16 + 1], DEV)
    pool, rope = _nan_pool(n, hk, d), daa.Rope(d)
    q0, k0, v0 = _rows(rng, cached, hq, hk, d, "fused")
    daa.BatchAttention(first, hq, pool).append_rope(q0, k0, v0, rope)
    parent = [-1, 0, 0, 1, 1, 2, 2]
    depth = np.array([0, 1, 1, 2, 2, 2, 2])
    mask = np.zeros((nodes, 1), np.int32)
    for i in range(nodes):
        p = parent[i]
        while p >= 0:
            mask[i, 0] |= 1 << p
            p = parent[p]
    q, k, v = _rows(rng, nodes, hq, hk, d, "fused")
    pos = (cached + depth).astype(np.int32)
    out = daa.BatchAttention(table, hq, pool).step_rope(q, k, v, rope, positions=_dev(pos), tree_mask=_dev(mask))
    f = rope.frequencies
    kc, _ = ref.rotate(_np(k0), np.arange(cached), f, d, False)
    kn, _ = ref.rotate(_np(k), pos, f, d, False)
    qn, _ = ref.rotate(_np(q), pos, f, d, False)
    for i in range(nodes):
        sees = [j for j in range(i + 1) if j == i or mask[i, 0] >> j & 1]
        keys, values = np.concatenate([kc, kn[sees]]), np.concatenate([_np(v0), _np(v)[sees]])
        want = _attend(qn[i:i + 1], keys, values, len(keys) - 1, d ** -0.5)[0]
        big = np.abs(qn[i])[:, None] * np.abs(np.repeat(keys, 2, 1)).transpose(1, 0, 2)
        dw = np.exp(2 * big.sum(-1).max(-1)[:, None] * d ** -0.5 * (2.0 ** -7 + 2.0 ** -15)) - 1 + 2.0 ** -8
        size = _attend(qn[i:i + 1], keys, np.abs(values), len(keys) - 1, d ** -0.5)[0]
        assert (np.abs(_np(out[i]) - want) <= 2.0 ** -8 * np.abs(want) + 2 * dw * size).all()


# --------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("kind", ["rope", "append", "append_q4"])
def test_captured_and_replayed(daa, kind):
    """A captured call on buffers whose contents change between replays, the number of rows in use among them."""
    rng = np.random.default_rng(15)
    hq, hk, d, rows = 6, 2, 128, 50
    rope = daa.Rope(d)
    steps = []
    for cached, new in (([5, 100, 31], [1, 1, 1]), ([6, 101, 32], [20, 3, 27]), ([0, 0, 0], [0, 9, 0])):
        t, _ = q4_support.make_table(np.random.default_rng(16), cached, new, spare=0)
        x = _bf16(rng, (rows, hq + 2 * hk, d))
        pos = rng.integers(0, 9999, rows).astype(np.int32)
        steps.append((t, x, pos))
    n = max(len(t["page_indices"]) for t, _, _ in steps)
    i32 = dict(dtype=torch.int32, device=DEV)
    buf = dict(x=torch.zeros(rows, hq + 2 * hk, d, dtype=torch.bfloat16, device=DEV), pos=torch.zeros(rows, **i32), qo=torch.zeros(4, **i32),
               kv=torch.zeros(4, **i32), pi=torch.zeros(n, **i32), last=torch.zeros(3, **i32))
    pool = torch.zeros(n, hk, 2, 9 * d, dtype=torch.uint8, device=DEV) if kind == "append_q4" else torch.zeros(n, 2, hk, 16, d, dtype=torch.bfloat16, device=DEV)
    out, ko = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, hk, d, dtype=torch.bfloat16, device=DEV)

    def call(b, pool, out, ko, stream=None):
        q, k, v = b["x"][:, :hq], b["x"][:, hq:hq + hk], b["x"][:, hq + hk:]
        if kind == "rope":
            daa.apply_rope(q, k, b["pos"], rope, q_out=out, k_out=ko, stream=stream)
        else:
            (daa.append_rope_q4 if kind == "append_q4" else daa.append_rope)(q, k, v, pool, b["qo"], b["pi"], b["kv"], b["last"], rope, q_out=out, stream=stream)

    s = torch.cuda.Stream()
    call(buf, pool, out, ko, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(buf, pool, out, ko)
        call(buf, pool, out, ko)
    assert not out.any() and not pool.any()
    for t, x, pos in steps:
        b = dict(x=x, pos=_dev(pos), qo=_dev(t["qo_indptr"]), kv=_dev(t["kv_indptr"]), pi=_dev(t["page_indices"]), last=_dev(t["last_page_len"]))
        want = pool.clone(), out.clone(), ko.clone()
        call(b, *want)
        for name, y in b.items():
            buf[name][:len(y)].copy_(y)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(out, want[1]) and torch.equal(ko, want[2])


@pytest.mark.parametrize("q4", [False, True])
def test_steps_on_another_stream(daa, q4):
    """step_rope on a stream that is still busy: what it makes in between (the rotated queries) is that stream's too."""
    rng = np.random.default_rng(20)
    hq, hk, d = 16, 4, 128
    t, n = q4_support.make_table(rng, [300, 17, 900], [200, 1, 1])
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    new_pool = (lambda: torch.zeros(n, hk, 2, 9 * d, dtype=torch.uint8, device=DEV)) if q4 else (lambda: torch.zeros(n, 2, hk, 16, d, dtype=torch.bfloat16, device=DEV))
    q, k, v = _rows(rng, 202, hq, hk, d, "fused")
    rope = daa.Rope(d)
    attn = lambda p: (daa.BatchAttentionQ4 if q4 else daa.BatchAttention)(table, hq, p)  # noqa: E731
    want = attn(new_pool()).step_rope(q, k, v, rope)
    for raw in (False, True):
        s = torch.cuda.Stream()
        name = s.cuda_stream if raw else s
        a = attn(new_pool())
        late = torch.zeros_like(q._base)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)
            late.copy_(q._base)
        outs = []
        for _ in range(3):
            outs.append(a.step_rope(late[:, :hq], late[:, hq:hq + hk], late[:, hq + hk:], rope, stream=name))
            junk = [torch.full_like(q, 9.0) for _ in range(4)]  # on this stream: not in the call's memory
            del junk
        s.synchronize()
        for o in outs:
            assert torch.equal(o, want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", ["rope", "append", "append_q4"])
def test_other_streams(daa, kind, raw):
    """Inputs that the call's stream still fills behind other work, outputs made for that stream, and the call's own attention."""
    rng = np.random.default_rng(17)
    t, n = q4_support.make_table(rng, [30, 2], [3, 40])
    rope = daa.Rope(64)
    x = _bf16(rng, (43, 8, 64))
    late, pos = torch.zeros_like(x), _dev(np.arange(43).astype(np.int32))
    tab = _dev_table(t)
    s = torch.cuda.Stream()
    name = s.cuda_stream if raw else s

    def call(x, pool, stream):
        q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
        if kind == "rope":
            return daa.apply_rope(q, k, pos, rope, stream=stream)
        return ((daa.append_rope_q4 if kind == "append_q4" else daa.append_rope)(q, k, v, pool, *tab, rope, stream=stream), pool)

    new_pool = (lambda: daa.new_q4_pool(n, 2, 64)) if kind == "append_q4" else (lambda: _nan_pool(n, 2, 64))
    want, pool = call(x, new_pool(), None), new_pool()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        late.copy_(x)
    got = call(late, pool, name)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once(daa):
    """Calls share nothing: many on two streams, each with its own rows and pages."""
    rng = np.random.default_rng(18)
    jobs = []
    for hq, hk, d, cached, new in ((32, 8, 128, [100, 5], [600, 1]), (4, 4, 64, [7] * 60, [1] * 60)):
        t, n = q4_support.make_table(rng, cached, new)
        q, k, v = _rows(rng, int(t["qo_indptr"][-1]), hq, hk, d, "fused")
        rope = daa.Rope(d)
        want = _nan_pool(n, hk, d)
        q_want = daa.append_rope(q, k, v, want, *_dev_table(t), rope)
        jobs.append((q, k, v, _dev_table(t), rope, want, q_want, _nan_pool(n, hk, d), torch.empty_like(q_want), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for q, k, v, tab, rope, _, _, pool, out, s in jobs:
            daa.append_rope(q, k, v, pool, *tab, rope, q_out=out, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, _, want, q_want, pool, out, _ in jobs:
        assert torch.equal(pool.view(torch.int16), want.view(torch.int16)) and torch.equal(out, q_want)


def test_traced(daa):
    rng = np.random.default_rng(19)
    t, n = q4_support.make_table(rng, [3], [2])
    q, k, v = _rows(rng, 2, 4, 2, 64, "flat")
    rope, tab = daa.Rope(64), _dev_table(t)
    daa.trace_enable(8)
    try:
        daa.apply_rope(q, k, _dev(np.arange(2).astype(np.int32)), rope)
        daa.append_rope(q, k, v, _nan_pool(n, 2, 64), *tab, rope)
        daa.append_rope_q4(q, k, v, daa.new_q4_pool(n, 2, 64), *tab, rope)
        assert [x for x, _ in daa.trace_read()] == ["rope", "append_rope", "append_rope_q4"]
    finally:
        daa.trace_disable()
