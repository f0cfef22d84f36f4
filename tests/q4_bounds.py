"""Bounds of attention over the 4-bit cache that see wrong V data.  q4_support's
check_attention allows the softmax weights the rounding of bf16 on every path, and in a
long context that is more than a page of V; here the rounding is an argument, and V is
zero but for one page at a time, so that the bounds are relative to that page alone."""
import numpy as np
import torch

import q4_support as ref

FP16, BF16 = 2.0 ** -11, 2.0 ** -8  # half a step of the softmax weights, relative
P = 16


def by_page(q, pool, t, r, d, scale, causal=True):
    """Request r against its V pages one at a time, float64: (out, A, C), [pages, tokens, Hq, d] each.  out[p] is the
    attention with V zero outside page p; A the same of |v|, and C the sum of |v| over the page's visible keys."""
    hkv = pool.shape[1]
    a0, a1, p0, p1 = t["qo_indptr"][r], t["qo_indptr"][r + 1], t["kv_indptr"][r], t["kv_indptr"][r + 1]
    n, m = a1 - a0, p1 - p0
    kvlen = (m - 1) * P + t["last_page_len"][r]
    pages = torch.from_numpy(ref.decode_pages(pool[t["page_indices"][p0:p1]], d, None))  # [m, 2, Hkv, 16, d]
    k, v = (pages[:, i].transpose(1, 2).reshape(m * P, hkv, d) for i in (0, 1))
    s = torch.einsum("thgd,khd->thgk", torch.from_numpy(q[a0:a1]).reshape(n, hkv, -1, d), k) * scale
    last = kvlen - n + torch.arange(n) if causal else torch.full((n,), kvlen - 1)
    seen = torch.arange(m * P) <= last[:, None]
    s = s.masked_fill(~seen[:, None, None], -torch.inf)
    w = torch.softmax(s, -1)
    see = seen[:, None, None].double().expand_as(w)
    v = torch.where(torch.arange(m * P)[:, None, None] < kvlen, v, torch.zeros_like(v))
    split = lambda x: x.reshape(*x.shape[:-1], m, P)  # noqa: E731
    out, A, C = (torch.einsum("thgpk,pkhd->pthgd", split(a), b.reshape(m, P, hkv, d)).reshape(m, n, -1, d).numpy()
                 for a, b in ((w, v), (w, v.abs()), (see, v.abs())))
    return out, A, C


def check_by_page(got, want, B, d, weight):
    """got [..., d] against by_page's values, with scores whose sum of |q k| times the scale is at most B:
    scores   fp32 sums of d products and a scaling, ds = (d + 8) 2^-24 B; on both sides of the quotient, each with the
             row's maximum
    weights  rounded by `weight` at most; exponentials 2^-22 on both sides; fp16's steps end at 2^-24, and weights are
             held times 2^7 over a maximum that is at most the row's: 2^-32 C
    sums     fp32, split and joined: 2^-16
    out      one rounding to bf16, 2^-8"""
    out, A, C = want
    ds = (d + 8) * 2.0 ** -24 * B
    dw = (weight + 4 * ds + 2.0 ** -21 + 2.0 ** -16) * A + 2.0 ** -32 * C
    tol = 2.0 ** -8 * (np.abs(out) + dw) + dw + 1e-30
    err = np.abs(got - out)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))
