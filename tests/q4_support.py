"""The 4-bit cache, the step tables and attention over the cache, restated in
numpy / float64 for the tests.  Shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

P = 16
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# every positive e4m3 number by its code 1 .. 126
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def _nearest(v, grid):
    """Index of the grid value nearest to v >= 0, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, v, side="left")
    tie = (i < len(mid)) & (v == mid[np.minimum(i, len(mid) - 1)])
    return i + (tie & (i % 2 == 1))


def quantise(x, e):
    """x float64 [..., d] (bf16 values), e broadcast over x[..., 0]: (codes [..., d], scale codes [..., d/16])."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(np.isnan(x), 0.0, x) * 2.0 ** -np.clip(np.asarray(e, np.float64), -32, 32)[..., None]
        y = y.reshape(*y.shape[:-1], -1, P)
        # nearest code of max / 6, compared sixfold so that ties stay exact; at least 2^-9
        sc = np.maximum(_nearest(np.minimum(np.abs(y).max(-1), 1e300), 6 * E4M3), 1)
        mag = _code(y, E4M3[sc])
    code = mag + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def _code(y, s):
    """Nearest e2m1 code of |y| / s, ties to even: |y| against the midpoints times s (exact products)."""
    a, mag = np.abs(y), np.zeros(y.shape, np.int64)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2 * s[..., None]
        mag += (a > mid) | ((a == mid) & (i % 2 == 1))
    return mag


def decode_pages(pool, d, exps):
    """Values of uint8 slices [n, Hkv, 2, 9 d]: float64 [n, 2, Hkv, 16, d]."""
    n, hkv = pool.shape[:2]
    body = pool[..., :8 * d].reshape(n, hkv, 2, P, d // 2)
    code = np.stack([body & 15, body >> 4], -1).reshape(n, hkv, 2, P, d)
    val = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    full = np.concatenate([E4M3, [np.nan]])
    full = np.concatenate([full, -full])
    sc = full[pool[..., 8 * d:]]
    sc = np.stack([sc[:, :, 0].reshape(n, hkv, P, d // 16), sc[:, :, 1].reshape(n, hkv, d // 16, P).swapaxes(2, 3)], 2)
    e = np.zeros((2, hkv)) if exps is None else np.clip(np.asarray(exps, np.float64), -32, 32)
    val = val.reshape(n, hkv, 2, P, d // 16, P) * (sc * 2.0 ** e.T[None, :, :, None, None])[..., None]
    return val.reshape(n, hkv, 2, P, d).swapaxes(1, 2)


def append(pool, k, v, t, exps):
    """kv_append_q4 on a host pool (uint8 [n, Hkv, 2, 9 d]) in place; k, v float64 [rows, Hkv, d]."""
    hkv, d = k.shape[1:]
    nb = d // 16
    e = np.zeros((2, hkv)) if exps is None else np.asarray(exps)
    for kv, x in enumerate((k, v)):
        code, sc = quantise(x, np.broadcast_to(e[kv], x.shape[:2]))
        for r in range(len(t["last_page_len"])):
            a0, a1 = t["qo_indptr"][r], t["qo_indptr"][r + 1]
            p0, np_ = t["kv_indptr"][r], t["kv_indptr"][r + 1] - t["kv_indptr"][r]
            kvlen = (np_ - 1) * P + t["last_page_len"][r] if np_ else 0
            for row in range(a0, a1):
                pos = kvlen - (a1 - a0) + row - a0
                page, s = t["page_indices"][p0 + pos // P], pos % P
                c = code[row]
                pool[page, :, kv, s * (d // 2):(s + 1) * (d // 2)] = c[:, 0::2] | (c[:, 1::2] << 4)
                at = 8 * d + (s * nb + np.arange(nb) if kv == 0 else np.arange(nb) * P + s)
                pool[page][:, kv, at] = sc[row]


def make_table(rng, cached, new, spare=5):
    """A page table (numpy int32) over shuffled pages of a pool of `num_pages`."""
    cached, new = np.asarray(cached), np.asarray(new)
    kv = cached + new
    np_ = -(-kv // P)
    n = int(np_.sum()) + spare
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return {"qo_indptr": i32(np.concatenate([[0], np.cumsum(new)])), "kv_indptr": i32(np.concatenate([[0], np.cumsum(np_)])),
            "page_indices": i32(rng.permutation(n)[:int(np_.sum())]), "last_page_len": i32(np.where(np_ > 0, kv - (np_ - 1) * P, 0))}, n


def attention(q, pool, t, exps, d, scale, causal=True):
    """float64 (out, lse, A, B, C): A = sum of weights times |v|, B = the largest scale * sum |q k| of a row's keys,
    C = sum of |v| over them -- the sizes that the error bounds of the tests are relative to.  q float64 [rows, Hq, d]."""
    hq, hkv = q.shape[1], pool.shape[1]
    g = hq // hkv
    out, A, C = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, B = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for r in range(len(t["last_page_len"])):
        a0, a1 = t["qo_indptr"][r], t["qo_indptr"][r + 1]
        if a1 == a0:
            continue
        p0, p1 = t["kv_indptr"][r], t["kv_indptr"][r + 1]
        kvlen = (p1 - p0 - 1) * P + t["last_page_len"][r]
        pages = decode_pages(pool[t["page_indices"][p0:p1]], d, exps)
        kk, vv = (torch.from_numpy(np.ascontiguousarray(pages[:, i].swapaxes(0, 1).reshape(hkv, -1, d)[:, :kvlen]))
                  for i in (0, 1))
        x = torch.from_numpy(q[a0:a1]).reshape(a1 - a0, hkv, g, d)
        s = torch.einsum("thgd,hkd->thgk", x, kk) * scale
        big = torch.einsum("thgd,hkd->thgk", x.abs(), kk.abs()) * scale
        if causal:
            hide = torch.arange(kvlen) > (kvlen - (a1 - a0) + torch.arange(a1 - a0))[:, None]
            s.masked_fill_(hide[:, None, None], -torch.inf)
            big.masked_fill_(hide[:, None, None], 0)
        z = torch.logsumexp(s, -1)
        w = (s - z[..., None]).exp()
        out[a0:a1] = torch.einsum("thgk,hkd->thgd", w, vv).reshape(a1 - a0, hq, d).numpy()
        A[a0:a1] = torch.einsum("thgk,hkd->thgd", w, vv.abs()).reshape(a1 - a0, hq, d).numpy()
        C[a0:a1] = torch.einsum("thgk,hkd->thgd", (s > -torch.inf).double(), vv.abs()).reshape(a1 - a0, hq, d).numpy()
        lse[a0:a1] = z.reshape(a1 - a0, hq).numpy()
        B[a0:a1] = big.amax(-1).reshape(a1 - a0, hq).numpy()
    return out, lse, A, B, C


def check_attention(out, lse, ref, d):
    """Against the float64 values, by the roundings on the way:
    scores   fp32 sums of d products and a scaling: off by at most ds = (d + 8) 2^-24 B
    weights  bf16 (2^-8) at the coarsest, from scores and a maximum that are off by ds each, and an exponential good to
             2^-22: relative error dw = 2^-8 + 2 ds + 2^-22, on both sides of the quotient but the rounding
             fp16 weights end at a step of 2^-24; they are held times 2^7 over a maximum that is at most the row's, so
             half a step is 2^-32 of the largest weight, and the sum of weights is at least the largest: 2^-32 C
    sums     fp32 over the keys, split and joined: 2^-16 covers 2^8 additions in a row at 2^-24 each
    out      one rounding to bf16 (2^-8), and 2^-24 for values near zero next to A"""
    r_out, r_lse, A, B, C = ref
    ds = (d + 8) * 2.0 ** -24 * B
    dw = (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2.0 ** -16)[..., None]
    tol = 2.0 ** -8 * (np.abs(r_out) + dw * A) + dw * A + 2.0 ** -32 * C + 1e-30
    err = np.abs(out - r_out)
    assert np.isfinite(out).all()
    assert (err <= tol).all(), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))
    if lse is not None:
        # the exponentials' sum is good to 2 ds + 2^-21 + 2^-16, and the maximum to ds
        lt = 3 * ds + 2.0 ** -16 + 2.0 ** -20 + 2.0 ** -23 * np.abs(r_lse)
        le = np.abs(lse - r_lse)
        assert (le <= lt).all(), (float((le / lt).max()), np.unravel_index((le / lt).argmax(), le.shape))


def step_table(state, slots, new, advance):
    """daa_step_table on numpy state (dict of seq_len, held, block_table, free (a list, top last)), in place."""
    qo, kp, pages, last, slot_map, pos = [0], [0], [], [], [], []
    for s, n in zip(slots, new):
        kv = int(state["seq_len"][s]) + int(n)
        need = -(-kv // P)
        for p in range(int(state["held"][s]), need):
            state["block_table"][s, p] = state["free"].pop()
        state["held"][s] = max(state["held"][s], need)
        row = state["block_table"][s, :need]
        pages += row.tolist()
        for t in range(kv - int(n), kv):
            pos.append(t)
            slot_map.append(int(row[t // P]) * P + t % P)
        last.append(kv - (need - 1) * P if need else 0)
        qo.append(qo[-1] + int(n))
        kp.append(kp[-1] + need)
        if advance:
            state["seq_len"][s] = kv
    return {"qo_indptr": qo, "kv_indptr": kp, "page_indices": pages, "last_page_len": last, "slot_map": slot_map,
            "positions": pos}
