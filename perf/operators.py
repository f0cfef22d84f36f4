"""What is measured of the 4-bit KV cache and of the step tables that feed it.

Operators (public entry points of ``decode_attention_append_gb300``):

* ``PagePool.build``       -- a step's page table, slot map and positions from the
                              requests' lengths, with the pages it needs taken
                              from the free list;
* ``kv_append_q4``         -- new K/V rows quantised to 4 bits and written into
                              their page slots;
* ``kv_dequant_q4``        -- pages of the 4-bit cache as bf16 pages;
* ``BatchAttentionQ4.run`` -- mixed-batch attention that reads the 4-bit cache.

The 4-bit cache: uint8 ``[num_pages, Hkv, 2 (K, V), 9 * d]``.  A slice holds 16
token rows of d/2 bytes (dim 2i in the low nibble of byte i, dim 2i + 1 in the
high one; e2m1: sign, two exponent bits, one mantissa bit), then the e4m3 scales
of every 16 dims of a token: K's as [16 tokens][d/16], V's as [d/16][16 tokens].
A value is e2m1 * e4m3 * 2^kv_exp[K or V][head].
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a serving loop: the page table of 64 requests, one new token each
        {"name": "table_decode", "op": "table", "batch": 64, "lo": 1024, "hi": 4096, "new_lo": 1, "new_hi": 1, "spare": 16},
        # a large fleet of long conversations: 512 requests of up to 128k cached tokens, short chunks arriving
        {"name": "table_long", "op": "table", "batch": 512, "lo": 4096, "hi": 131072, "new_lo": 1, "new_hi": 61, "spare": 128},
        # one new token of 128 decode requests (GQA, 8 kv heads): latency
        {"name": "append_decode", "op": "append", "batch": 128, "new_lo": 1, "new_hi": 1, "cached_hi": 4096, "hkv": 8, "d": 128, "exps": False},
        # prompts of ragged lengths prefilled in one step, with per-head exponents
        {"name": "append_prompts", "op": "append", "batch": 7, "new_lo": 1001, "new_hi": 8192, "cached_hi": 777, "hkv": 8, "d": 128, "exps": True},
        # a few pages of a request handed to a bf16 reader, head_dim 64, an odd number of heads
        {"name": "pages_few", "op": "dequant", "pages": 129, "hkv": 5, "d": 64, "exps": True},
        # the cache of a long prompt (one layer), 8 kv heads
        {"name": "pages_many", "op": "dequant", "pages": 8192, "hkv": 8, "d": 128, "exps": False},
        # the smallest step: a 16-token chunk of a 64-token prompt and two decodes, head_dim 64
        {"name": "attn_tiny", "op": "attention", "hq": 4, "hkv": 2, "d": 64, "chunks": 1, "chunk": 16, "chunk_cached": 48, "reqs": 2, "new": 1, "kv_lo": 40, "kv_hi": 73, "exps": False},
        # decode of a 7B-class model: every query head has its own kv head
        {"name": "attn_decode_mha", "op": "attention", "hq": 32, "hkv": 32, "d": 128, "chunks": 0, "chunk": 0, "chunk_cached": 0, "reqs": 32, "new": 1, "kv_lo": 512, "kv_hi": 4096, "exps": False},
        # decode shard of a large GQA model: 12 query heads on one kv head, long conversations
        {"name": "attn_decode_gqa", "op": "attention", "hq": 12, "hkv": 1, "d": 128, "chunks": 0, "chunk": 0, "chunk_cached": 0, "reqs": 128, "new": 1, "kv_lo": 1024, "kv_hi": 32768, "exps": True},
        # a speculative-decoding verify step: 5 new tokens a request, head_dim 128, GQA 4:1
        {"name": "attn_verify", "op": "attention", "hq": 32, "hkv": 8, "d": 128, "chunks": 0, "chunk": 0, "chunk_cached": 0, "reqs": 32, "new": 5, "kv_lo": 1024, "kv_hi": 4096, "exps": False},
        # a continuous batch: one 512-token chunk over 1536 cached tokens beside 32 decodes, GQA 4:1
        {"name": "attn_mixed", "op": "attention", "hq": 32, "hkv": 8, "d": 128, "chunks": 1, "chunk": 512, "chunk_cached": 1536, "reqs": 32, "new": 1, "kv_lo": 1024, "kv_hi": 4096, "exps": False},
        # long-prompt prefill: two 8192-token chunks over 8192 cached tokens beside 32 decodes, GQA 8:1
        {"name": "attn_prefill", "op": "attention", "hq": 64, "hkv": 8, "d": 128, "chunks": 2, "chunk": 8192, "chunk_cached": 8192, "reqs": 32, "new": 1, "kv_lo": 2048, "kv_hi": 16384, "exps": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["table", "append", "dequant", "attention", "attention", "attention"])
    d = rng.choice([64, 128, 128])
    exps = rng.random() < 0.5
    if op == "table":
        hi = _log_int(rng, 64, 131072)
        return {"op": op, "batch": _log_int(rng, 1, 512), "lo": _log_int(rng, 1, hi), "hi": hi, "new_lo": rng.choice([0, 1]), "new_hi": _log_int(rng, 1, 700), "spare": rng.randint(0, 100)}
    if op == "append":
        new_hi = _log_int(rng, 1, 8192)
        batch = _log_int(rng, 1, max(1, min(500, 40000 // new_hi)))
        return {"op": op, "batch": batch, "new_lo": rng.choice([0 if batch > 8 else 1, 1, 1 + new_hi // 3]), "new_hi": new_hi, "cached_hi": _log_int(rng, 1, 2000), "hkv": rng.randint(1, 8), "d": d, "exps": exps}
    if op == "dequant":
        return {"op": op, "pages": _log_int(rng, 1, 8192), "hkv": rng.randint(1, 8), "d": d, "exps": exps}
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    hkv = rng.randint(1, 8) if g > 1 else rng.randint(1, 32)
    reqs = _log_int(rng, 1, 128)
    kv_hi = _log_int(rng, 16, max(16, min(32768, (1 << 21) // (reqs * hkv))))
    new = rng.choice([1, 1, 1, 2, 3, 4, 6, 8, 13])
    kind = rng.choice(["decode", "decode", "mixed"])
    chunks = rng.randint(1, 2) if kind == "mixed" else 0
    return {"op": op, "hq": g * hkv, "hkv": hkv, "d": d, "chunks": chunks, "chunk": _log_int(rng, 17, 4096) if chunks else 0, "chunk_cached": rng.randint(0, 4096) if chunks else 0,
            "reqs": reqs, "new": new, "kv_lo": max(new, _log_int(rng, 1, kv_hi)), "kv_hi": max(new, kv_hi), "exps": exps}


# -------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator()
    g.manual_seed(1_000_003 * int(seed) + salt)
    return g


def _lengths(n, lo, hi, g):
    """n lengths of [lo, hi], even over their logarithm where that spans more than a factor of ten."""
    u = torch.rand(n, generator=g, dtype=torch.float64)
    if lo > 0 and hi > 10 * lo:
        x = torch.exp(math.log(lo) + u * (math.log(hi + 1) - math.log(lo)))
    else:
        x = lo + u * (hi + 1 - lo)
    return x.floor().long().clamp(lo, hi)


def _lengths_of(case, seed):
    """(cached, new) of every request, host int64: a case's lengths are the same for every seed, and the seed orders the requests."""
    g = _gen(0, sum((i + 1) * v for i, v in enumerate(v for v in case.values() if isinstance(v, int))))
    if case["op"] == "table":
        cached, new = _lengths(case["batch"], case["lo"], case["hi"], g), _lengths(case["batch"], case["new_lo"], case["new_hi"], g)
    elif case["op"] == "append":
        cached, new = _lengths(case["batch"], 0, case["cached_hi"], g), _lengths(case["batch"], case["new_lo"], case["new_hi"], g)
    else:
        kv = _lengths(case["reqs"], case["kv_lo"], case["kv_hi"], g)
        cached, new = kv - case["new"], torch.full((case["reqs"],), case["new"])
    order = torch.randperm(len(new), generator=_gen(seed, 1))
    cached, new = cached[order], new[order]
    if case["op"] != "attention":
        return cached, new
    chunks = torch.full((case["chunks"],), case["chunk"])
    return torch.cat([torch.full((case["chunks"],), case["chunk_cached"]), cached]), torch.cat([chunks, new])


def _csr(n):
    return torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])


def _tables(cached, new, g, spare=7):
    """The batch's page table (host int32) over a random permutation of the pool's pages."""
    kv = cached + new
    np_ = (kv + PAGE - 1) // PAGE
    total = int(np_.sum())
    pool = total + spare
    return {"qo_indptr": _csr(new).int(), "kv_indptr": _csr(np_).int(), "page_indices": torch.randperm(pool, generator=g)[:total].int(),
            "last_page_len": torch.where(np_ > 0, kv - (np_ - 1) * PAGE, 0).int(), "num_pages": pool}


def _exps(case, g):
    e = torch.randint(-3, 4, (2, case["hkv"]), generator=g, dtype=torch.int32)
    return e.to(DEV) if case["exps"] else None


def _normal(shape, g, spread=None):
    """bf16 values as K and V have them: N(0, 1), and with `spread` a few dims of a head eight times as large."""
    dg = torch.Generator(device=DEV)
    dg.manual_seed(int(torch.randint(1 << 40, (1,), generator=g)))
    x = torch.randn(shape, generator=dg, device=DEV)
    if spread is not None:
        x[..., spread::37] *= 8
    return x.bfloat16()


def _pool(case, pages, g, exps):
    """A 4-bit pool whose every slot holds quantised values (as reused pages do)."""
    hkv, d = case["hkv"], case["d"]
    pool = torch.empty(pages, hkv, 2, 9 * d, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (hkv * 2 * PAGE * d))
    for p in range(0, pages, step):  # a part of the pages at a time, for room
        n = min(step, pages - p)
        k, v = _normal((n, hkv, PAGE, d), g, 5), _normal((n, hkv, PAGE, d), g)
        pool[p:p + n] = _pack_pages(k, v, exps)
    return pool


def prepare(case, seed):
    s = {"case": case}
    g = _gen(seed, 2)
    if case["op"] == "dequant":
        s["exps"] = _exps(case, g)
        s["pool"] = _pool(case, case["pages"] + 9, g, s["exps"])
        s["ids"] = torch.randperm(case["pages"] + 9, generator=g)[:case["pages"]].int().to(DEV)
        s["out"] = torch.empty(case["pages"], 2, case["hkv"], PAGE, case["d"], dtype=torch.bfloat16, device=DEV)
        return s
    cached, new = _lengths_of(case, seed)
    if case["op"] == "table":
        # a fleet of slots: the batch's requests sit in some of them and hold their cached pages
        n, slots = case["batch"], case["batch"] + case["spare"]
        held = (cached + PAGE - 1) // PAGE
        total = (cached + new + PAGE - 1) // PAGE
        num_pages = int(total.sum()) + 11 * slots
        perm = torch.randperm(num_pages, generator=g)
        at = torch.randperm(slots, generator=g)[:n]
        width = int(total.max()) + 3
        table = torch.full((slots, width), -1, dtype=torch.int32)
        used = torch.arange(width)[None, :] < held[:, None]
        rows = torch.full((n, width), -1, dtype=torch.int32)
        rows[used] = perm[:int(held.sum())].int()
        table[at] = rows
        free = perm[int(held.sum()):]
        seq, hold = torch.zeros(slots, dtype=torch.int32), torch.zeros(slots, dtype=torch.int32)
        seq[at], hold[at] = cached.int(), held.int()
        stack = torch.full((num_pages,), -1, dtype=torch.int32)
        stack[:len(free)] = free.int()
        s.update(slots=at.int().to(DEV), new=new.int().to(DEV), seq_len=seq.to(DEV), held=hold.to(DEV), block_table=table.to(DEV), free_pages=stack.to(DEV),
                 counters=torch.tensor([len(free), 0], dtype=torch.int32, device=DEV), num_pages=num_pages, n_pages=int(total.sum()), n_rows=int(new.sum()))
        i32 = dict(dtype=torch.int32, device=DEV)
        s["out"] = {"qo_indptr": torch.empty(n + 1, **i32), "kv_indptr": torch.empty(n + 1, **i32), "page_indices": torch.empty(s["n_pages"], **i32), "last_page_len": torch.empty(n, **i32),
                    "slot_map": torch.empty(s["n_rows"], dtype=torch.int64, device=DEV), "positions": torch.empty(s["n_rows"], **i32)}
        if own:
            import decode_attention_append_gb300 as daa
            s["pages"] = daa.PagePool.from_tensors(s["seq_len"], s["held"], s["block_table"], s["free_pages"], s["counters"])
        return s
    t = _tables(cached, new, g)
    s["exps"] = _exps(case, g)
    s["pool"] = _pool(case, t.pop("num_pages"), g, s["exps"])
    s["t"] = {k: v.to(DEV) for k, v in t.items()}
    rows = int(new.sum())
    if case["op"] == "append":
        s["k"] = _normal((rows, case["hkv"], case["d"]), g, 5)
        s["v"] = _normal((rows, case["hkv"], case["d"]), g)
        # the pages that the step writes, for reading them back
        kv, np_ = cached + new, t["kv_indptr"].long()
        first = cached // PAGE
        count = torch.where(new > 0, np_[1:] - np_[:-1] - first, 0)
        base = torch.repeat_interleave(np_[:-1] + first - (_csr(count)[:-1]), count)
        s["written"] = t["page_indices"][base + torch.arange(int(count.sum()))].to(DEV)
        s["out"] = torch.empty(len(s["written"]), 2, case["hkv"], PAGE, case["d"], dtype=torch.bfloat16, device=DEV)
        return s
    s["lens"] = (cached, new)
    s["q"] = _normal((rows, case["hq"], case["d"]), g)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(rows, case["hq"], dtype=torch.float32, device=DEV)
    # short requests (as many new tokens as a verify step has) as one padded batch
    kv = cached + new
    short = torch.nonzero(new <= PAGE).flatten()
    s["long"] = [int(r) for r in torch.nonzero(new > PAGE).flatten()]
    s["short"], s["kv_len"], s["new"] = short.to(DEV), kv.to(DEV), new.to(DEV)
    s["max_new"], s["max_pages"] = (int(new[short].max()), int((kv[short].max() + PAGE - 1) // PAGE)) if len(short) else (0, 0)
    if own:
        import decode_attention_append_gb300 as daa
        table = daa.PageTable.from_host(t["qo_indptr"], t["kv_indptr"], t["page_indices"], t["last_page_len"], DEV)
        s["attn"] = daa.BatchAttentionQ4(table, case["hq"], s["pool"], kv_exp=s["exps"])
        s["attn"].plan()
    return s


# ---------------------------------------------------------------- plain form
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x, e):
    """Codes (uint8, one a value) and e4m3 scales (uint8, one each 16 dims) of x [..., d]; e: its exponents, broadcast over x, or None."""
    y = x.float().nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf)
    if e is not None:
        y = y * torch.exp2(-e.float())
    y = y.unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=x.device)  # a division: by a Python number torch multiplies by its reciprocal
    scale = (y.abs().amax(-1) / six).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    t = (y / scale.float()[..., None]).abs()
    # nearest value, ties to the even code: a tie goes up only where the upper code is even
    code = ((t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte() + (t > 2.5).byte() + (t >= 3.5).byte() + (t > 5.0).byte())
    code = code + 8 * torch.signbit(y).byte()
    return code.flatten(-2), scale.view(torch.uint8)


def _pack_rows(x, e):
    code, scale = _quantise(x, e)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _pack_pages(k, v, exps):
    """bf16 pages [n, Hkv, 16, d] of K and V as 4-bit slices [n, Hkv, 2, 9 * d]."""
    ek, ev = (None, None) if exps is None else (exps[0][:, None, None], exps[1][:, None, None])
    (ck, sk), (cv, sv) = _pack_rows(k, ek), _pack_rows(v, ev)
    return torch.stack([torch.cat([ck.flatten(2), sk.flatten(2)], -1), torch.cat([cv.flatten(2), sv.transpose(2, 3).flatten(2)], -1)], 2)


def _dequantise(slices, d, exps):
    """fp32 (K, V) [..., Hkv, 16, d] of slices [..., Hkv, 2, 9 * d]."""
    lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=slices.device)
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)  # [byte] -> (low, high)
    vals = pairs.index_select(0, slices[..., :8 * d].flatten().int()).view(*slices.shape[:-1], PAGE, d)
    sc = slices[..., 8 * d:].view(torch.float8_e4m3fn).float()
    sk = sc[..., 0, :].unflatten(-1, (PAGE, d // 16))
    sv = sc[..., 1, :].unflatten(-1, (d // 16, PAGE)).transpose(-1, -2)
    if exps is not None:
        e = torch.exp2(exps.float())[:, :, None, None]
        sk, sv = sk * e[0], sv * e[1]
    k = (vals[..., 0, :, :].unflatten(-1, (d // 16, 16)) * sk[..., None]).flatten(-2)
    v = (vals[..., 1, :, :].unflatten(-1, (d // 16, 16)) * sv[..., None]).flatten(-2)
    return k, v


def _plain_dequant(s, ids):
    k, v = _dequantise(s["pool"][ids.long()], s["case"]["d"], s["exps"])
    return torch.stack([k, v], 1).bfloat16()


def _plain_table(s):
    slots, new = s["slots"].long(), s["new"].long()
    seq, held = s["seq_len"][slots].long(), s["held"][slots].long()
    kv = seq + new
    pages = (kv + PAGE - 1) // PAGE
    take = (pages - held).clamp(min=0)
    zero = torch.zeros(1, dtype=torch.long, device=slots.device)
    qo, kp, tp = (torch.cat([zero, x.cumsum(0)]) for x in (new, pages, take))
    n = len(slots)
    free = s["counters"][0].long()
    req = torch.repeat_interleave(torch.arange(n, device=slots.device), pages, output_size=s["n_pages"])
    p = torch.arange(s["n_pages"], device=slots.device) - kp[req]
    fresh = p >= held[req]
    j = torch.where(fresh, free - 1 - (tp[req] + p - held[req]), 0)
    ids = torch.where(fresh, s["free_pages"][j], s["block_table"][slots[req], p])
    s["block_table"][slots[req], p] = ids
    row = torch.repeat_interleave(torch.arange(n, device=slots.device), new, output_size=s["n_rows"])
    pos = seq[row] + torch.arange(s["n_rows"], device=slots.device) - qo[row]
    slot_map = ids[kp[row] + pos // PAGE].long() * PAGE + pos % PAGE
    s["held"][slots] = torch.maximum(held, pages).int()
    s["counters"][0] = (free - tp[n]).int()
    last = torch.where(pages > 0, kv - (pages - 1) * PAGE, 0)
    return {"qo_indptr": qo.int(), "kv_indptr": kp.int(), "page_indices": ids, "last_page_len": last.int(), "slot_map": slot_map, "positions": pos.int()}


def _plain_append(s):
    t, d = s["t"], s["case"]["d"]
    qo, kp = t["qo_indptr"].long(), t["kv_indptr"].long()
    new, np_ = qo[1:] - qo[:-1], kp[1:] - kp[:-1]
    kv = torch.where(np_ > 0, (np_ - 1) * PAGE + t["last_page_len"], 0)
    rows = s["k"].shape[0]
    req = torch.repeat_interleave(torch.arange(len(new), device=qo.device), new, output_size=rows)
    pos = (kv - new)[req] + torch.arange(rows, device=qo.device) - qo[req]
    page, slot = t["page_indices"][kp[req] + pos // PAGE].long(), pos % PAGE
    ek, ev = (None, None) if s["exps"] is None else (s["exps"][0][:, None], s["exps"][1][:, None])
    (ck, sk), (cv, sv) = _pack_rows(s["k"], ek), _pack_rows(s["v"], ev)
    codes = s["pool"][..., :8 * d].unflatten(-1, (PAGE, d // 2))
    scale = s["pool"][..., 8 * d:]
    codes[page, :, 0, slot], codes[page, :, 1, slot] = ck, cv
    scale.unflatten(-1, (PAGE, d // 16))[page, :, 0, slot] = sk
    scale.unflatten(-1, (d // 16, PAGE))[page, :, 1, :, slot] = sv


def _attend(q, k, v, see, scale):
    """q [..., rows, d], k, v [..., keys, d], see [..., rows, keys]: (out, natural-log lse), fp32."""
    x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    return (p @ v) / z, (m + z.log())[..., 0]


def _plain_attention(s):
    c, t = s["case"], s["t"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, scale = hq // hkv, 1.0 / math.sqrt(d)
    qo, kp = t["qo_indptr"].long(), t["kv_indptr"].long()
    q = s["q"]
    if s["max_new"]:
        r, mq, mp = s["short"], s["max_new"], s["max_pages"]
        kv, new = s["kv_len"][r], s["new"][r]
        at = (kp[r][:, None] + torch.arange(mp, device=DEV)).clamp(max=len(t["page_indices"]) - 1)
        key = torch.arange(mp * PAGE, device=DEV)
        k, v = _dequantise(s["pool"][t["page_indices"].long()[at]], d, s["exps"])
        k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))  # [R, Hkv, keys, d]
        tok = torch.arange(mq, device=DEV)
        row = (qo[r][:, None] + tok).clamp(max=len(q) - 1)
        x = q.float()[row].view(len(r), mq, hkv, g, d).transpose(1, 2).reshape(len(r), hkv, mq * g, d)
        pos = (kv - new)[:, None] + tok
        see = (key <= pos[..., None]) & (key < kv[:, None, None])  # [R, tokens, keys]
        see = see.repeat_interleave(g, 1)[:, None]
        o, lse = _attend(x, k, v, see, scale)
        o = o.view(len(r), hkv, mq, g, d).transpose(1, 2).reshape(len(r), mq, hq, d)
        lse = lse.view(len(r), hkv, mq, g).transpose(1, 2).reshape(len(r), mq, hq)
        real = tok < new[:, None]
        s["out"][row[real]], s["lse"][row[real]] = o[real].bfloat16(), lse[real]
        del k, v, o
    cached, new = s["lens"]
    for r in s["long"]:  # a prompt's chunk: large products, one kv head at a time for room
        n, kv = int(new[r]), int(cached[r] + new[r])
        rows = slice(int(new[:r].sum()), int(new[:r].sum()) + n)
        first = int(((cached[:r] + new[:r] + PAGE - 1) // PAGE).sum())
        ids = t["page_indices"][first:first + (kv + PAGE - 1) // PAGE].long()
        k, v = (x.transpose(0, 1).flatten(1, 2)[:, :kv] for x in _dequantise(s["pool"][ids], d, s["exps"]))
        see = torch.arange(kv, device=DEV) <= (kv - n + torch.arange(n, device=DEV))[:, None]
        for h in range(hkv):
            o, lse = _attend(q[rows, h * g:(h + 1) * g].float().transpose(0, 1), k[h], v[h], see, scale)
            s["out"][rows, h * g:(h + 1) * g] = o.transpose(0, 1).bfloat16()
            s["lse"][rows, h * g:(h + 1) * g] = lse.T
    return s["out"], s["lse"]


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op == "table":
        # the step's tables for the pending tokens; the lengths advance once they are accepted, so a pass can be made again
        if own:
            s["pages"].build(s["slots"], s["new"], advance=False, **s["out"])
            got = s["out"]
        else:
            got = _plain_table(s)
        return {**got, "held": s["held"], "block_table": s["block_table"], "free": s["counters"][:1]}
    if op == "append":
        if own:
            import decode_attention_append_gb300 as daa
            t = s["t"]
            daa.kv_append_q4(s["k"], s["v"], s["pool"], t["qo_indptr"], t["page_indices"], t["kv_indptr"], t["last_page_len"], kv_exp=s["exps"])
            return daa.kv_dequant_q4(s["pool"], s["written"], kv_exp=s["exps"], out=s["out"])
        _plain_append(s)
        return _plain_dequant(s, s["written"])
    if op == "dequant":
        if own:
            import decode_attention_append_gb300 as daa
            return daa.kv_dequant_q4(s["pool"], s["ids"], kv_exp=s["exps"], out=s["out"])
        return _plain_dequant(s, s["ids"])
    if own:
        return s["attn"].run(s["q"], out=s["out"], lse=s["lse"]), s["lse"]
    return _plain_attention(s)


# ---------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass."""
    if case["op"] == "dequant":
        values = case["pages"] * case["hkv"] * 2 * PAGE * case["d"]
        return {"bytes": values * (9 / 16 + 2), "flops": values}
    cached, new = _lengths_of(case, 0)
    kv = cached + new
    if case["op"] == "table":
        pages = int(((kv + PAGE - 1) // PAGE).sum())
        return {"bytes": 8 * pages + 12 * int(new.sum()) + 32 * case["batch"], "flops": 4 * pages + 4 * int(new.sum())}
    d = case["d"]
    if case["op"] == "append":
        values = int(new.sum()) * case["hkv"] * 2 * d
        back = int(((kv + PAGE - 1) // PAGE - cached // PAGE)[new > 0].sum()) * case["hkv"] * 2 * PAGE * d
        return {"bytes": values * (2 + 9 / 16) + back * (9 / 16 + 2), "flops": 4 * values + back}
    pairs = int((new * cached + new * (new + 1) // 2).sum())
    return {"bytes": int(kv.sum()) * case["hkv"] * 2 * d * 9 // 16 + int(new.sum()) * case["hq"] * (4 * d + 4), "flops": 4 * d * case["hq"] * pairs}


# --------------------------------------------------------------------- exact
def _two_to(n):
    """2^n of whole numbers -64 .. 63 in float64, from a table made on the host (a GPU's pow is not exact)."""
    return torch.tensor([2.0 ** i for i in range(-64, 64)], dtype=torch.float64).to(n.device)[n.long() + 64]


def _exact_values(x, e):
    """float64 values that the cache holds for x [..., d] (float64), e broadcast over it: the definition, by nearest neighbours."""
    y = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf) * _two_to(-e)
    y = y.reshape(*y.shape[:-1], -1, 16)
    # every positive e4m3 number in the order of its code, 2^-9 to 448
    m = torch.arange(1, 127, device=x.device, dtype=torch.float64)
    ex, fr = torch.div(m, 8, rounding_mode="floor"), m % 8
    grid = torch.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * _two_to(ex - 10))

    def nearest(v, grid, first):
        mid = (grid[1:] + grid[:-1]) / 2
        i = torch.searchsorted(mid, v)  # ties to the lower code
        tie = v == mid[i.clamp(max=len(mid) - 1)]
        return i + (tie & ((i + first) % 2 == 1)).long()  # and to the even one

    s = grid[nearest(y.abs().amax(-1).clamp(max=1e9), 6 * grid, 1)].unsqueeze(-1)  # nearest to a sixth
    e2m1 = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device=x.device, dtype=torch.float64) / 2
    q = e2m1[nearest((y.abs() / s).clamp(max=1e9), e2m1, 0)]
    return (torch.copysign(q, y) * s).reshape(x.shape) * _two_to(e)


def _exact_pages(pool, d, exps):
    """float64 [n, 2, Hkv, 16, d]: the nibbles and scales taken apart bit by bit."""
    n, hkv = pool.shape[:2]
    body = pool[..., :8 * d].long().view(n, hkv, 2, PAGE, d // 2, 1)
    code = torch.cat([body % 16, body // 16], -1).view(n, hkv, 2, PAGE, d)
    ex, fr = (code // 2) % 4, code % 2
    val = torch.where(ex == 0, fr * 0.5, (1 + fr * 0.5) * _two_to(ex - 1))
    val = torch.where(code >= 8, -val, val)
    b = pool[..., 8 * d:].long()
    ex, fr = (b // 8) % 16, b % 8
    sc = torch.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * _two_to(ex - 10))
    sc = torch.stack([sc[:, :, 0].view(n, hkv, PAGE, d // 16), sc[:, :, 1].view(n, hkv, d // 16, PAGE).transpose(2, 3)], 2)
    if exps is not None:
        sc = sc * _two_to(exps).T[None, :, :, None, None]
    return (val.view(n, hkv, 2, PAGE, d // 16, 16) * sc[..., None]).view(n, hkv, 2, PAGE, d).transpose(1, 2)


def exact(case, seed):
    if case["op"] == "table":
        return None  # whole numbers
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "dequant":
        return _exact_pages(s["pool"][s["ids"].long()], d, s["exps"])
    if case["op"] == "append":
        out = _exact_pages(s["pool"][s["written"].long()], d, s["exps"])
        where = {int(p): i for i, p in enumerate(s["written"].tolist())}
        e = s["exps"] if s["exps"] is not None else torch.zeros(2, case["hkv"], dtype=torch.int32, device=DEV)
        t = {k: v.tolist() for k, v in s["t"].items()}
        at_page, at_slot = [], []
        for r in range(len(t["last_page_len"])):
            n, p0, p1 = t["qo_indptr"][r + 1] - t["qo_indptr"][r], t["kv_indptr"][r], t["kv_indptr"][r + 1]
            kv = (p1 - p0 - 1) * PAGE + t["last_page_len"][r] if p1 > p0 else 0
            for pos in range(kv - n, kv):
                at_page.append(where[t["page_indices"][p0 + pos // PAGE]])
                at_slot.append(pos % PAGE)
        at_page, at_slot = torch.tensor(at_page, device=DEV), torch.tensor(at_slot, device=DEV)
        for i, x in enumerate((s["k"], s["v"])):
            out[at_page, i, :, at_slot] = _exact_values(x.double(), e[i][:, None])
        return out
    cached, new = s["lens"]
    if float((new * (cached + new)).sum()) * case["hq"] * d * 4 > 1.2e13:
        return None
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    row = page = 0
    for c, n in zip(cached.tolist(), new.tolist()):
        np_ = -(-(c + n) // PAGE)
        kv = _exact_pages(s["pool"][s["t"]["page_indices"][page:page + np_].long()], d, s["exps"])
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, np_ * PAGE, d)[:, :, :c + n]
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            q = s["q"][row + a:row + b].double().view(b - a, hkv, g, d)
            x = torch.einsum("thgd,hkd->thgk", q, kv[0]) / math.sqrt(d)
            later = torch.arange(c + n, device=DEV) > (c + torch.arange(a, b, device=DEV))[:, None]
            x.masked_fill_(later[:, None, None], -math.inf)
            z = torch.logsumexp(x, -1)
            out[row + a:row + b] = torch.einsum("thgk,hkd->thgd", (x - z[..., None]).exp_(), kv[1]).reshape(b - a, -1, d)
            lse[row + a:row + b] = z.reshape(b - a, -1)
        row, page = row + n, page + np_
    return out, lse
