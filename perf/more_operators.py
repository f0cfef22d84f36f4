"""What is measured of the rotary positions and of the appends that apply them.

Operators (public entry points of ``decode_attention_append_gb300``):

* ``apply_rope``      -- query and key rows rotated by their tokens' positions;
* ``append_rope``     -- a step's queries rotated, its keys rotated and written
                         with its values into bf16 pages;
* ``append_rope_q4``  -- the same into a 4-bit pool.

A head's first ``rot`` dims form pairs -- (i, i + rot/2), or (2i, 2i + 1) when
interleaved -- and pair i of a token at position p turns by p * f[i] and grows by
the magnitude m; the other dims stay.  f[i] = base^(-2i/rot), changed for long
contexts by one of the scalings.  With norm weights each head is first divided by
its root mean square over the head's dims and multiplied by the weights.
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"
EPS = 1e-6
BASE = 10000.0
# what a context of ORIGINAL tokens is scaled by, and the bounds of the two scalings that treat pairs by their wavelength
FACTOR, ORIGINAL = 8.0, 4096
YARN = (32.0, 1.0)
WAVELENGTH = (1.0, 4.0)


# --------------------------------------------------------------------- cases
def _case(op, hq, hkv, d, rot, interleaved=False, scaling="none", norm=False, fused=True, prompts=0, p_lo=0, p_hi=0, p_cached=0, reqs=0, new=0, cached_lo=0, cached_hi=0, tree=False):
    """A step: `prompts` chunks of p_lo .. p_hi new tokens behind p_cached cached ones, and `reqs` requests of `new` tokens behind cached_lo .. cached_hi.
    fused: q, k and v are views of one projection's rows.  tree: the new tokens are nodes of draft trees, at the positions of their depths."""
    return {"op": op, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "interleaved": interleaved, "scaling": scaling, "norm": norm, "fused": fused, "prompts": prompts, "p_lo": p_lo, "p_hi": p_hi,
            "p_cached": p_cached, "reqs": reqs, "new": new, "cached_lo": cached_lo, "cached_hi": cached_hi, "tree": tree}


def listed():
    return [
        # the smallest step: a 16-token chunk behind 48 cached tokens and two decodes, head_dim 64; contiguous q and k
        {"name": "rope_tiny", **_case("rope", 4, 2, 64, 64, fused=False, prompts=1, p_lo=16, p_hi=16, p_cached=48, reqs=2, new=1, cached_lo=39, cached_hi=72)},
        # one decode step of a 7B-class model, every query head with its own kv head
        {"name": "rope_decode", **_case("rope", 32, 32, 128, 128, reqs=32, new=1, cached_lo=511, cached_hi=4095)},
        # ragged prompts of a model that turns half of a 64-dim head, neighbouring dims paired
        {"name": "rope_partial", **_case("rope", 20, 4, 64, 32, interleaved=True, scaling="linear", prompts=3, p_lo=301, p_hi=2001, p_cached=0)},
        # a long prompt's second half, two requests, beside 32 decodes, GQA 8:1, at positions past the trained context
        {"name": "rope_prompts", **_case("rope", 64, 8, 128, 128, scaling="yarn", prompts=2, p_lo=8192, p_hi=8192, p_cached=8192, reqs=32, new=1, cached_lo=2048, cached_hi=16383)},
        # the smallest step, appended
        {"name": "append_tiny", **_case("append", 4, 2, 64, 64, fused=False, prompts=1, p_lo=16, p_hi=16, p_cached=48, reqs=2, new=1, cached_lo=39, cached_hi=72)},
        # decode shard of a large GQA model, long conversations: latency
        {"name": "append_decode", **_case("append", 12, 1, 128, 128, scaling="wavelength", reqs=128, new=1, cached_lo=1023, cached_hi=32767)},
        # a verify step of small draft trees, heads normalised, GQA 4:1
        {"name": "append_verify", **_case("append", 32, 8, 128, 128, norm=True, reqs=32, new=5, cached_lo=1024, cached_hi=4096, tree=True)},
        # a continuous batch: one 512-token chunk behind 1536 cached tokens beside 32 decodes
        {"name": "append_mixed", **_case("append", 32, 8, 128, 128, scaling="ntk", prompts=1, p_lo=512, p_hi=512, p_cached=1536, reqs=32, new=1, cached_lo=1023, cached_hi=4095)},
        # long-prompt prefill: four 8192-token chunks behind 8192 cached tokens beside 64 decodes, GQA 8:1
        {"name": "append_prefill", **_case("append", 64, 8, 128, 128, scaling="yarn", prompts=4, p_lo=8192, p_hi=8192, p_cached=8192, reqs=64, new=1, cached_lo=2047, cached_hi=16383)},
        # one decode step into the 4-bit cache, GQA 4:1 (and the step's pages read back)
        {"name": "q4_decode", **_case("append_q4", 32, 8, 128, 128, reqs=128, new=1, cached_lo=1, cached_hi=4096)},
        # short ragged chunks of a model with odd head counts that turns a quarter of a 64-dim head
        {"name": "q4_partial", **_case("append_q4", 15, 5, 64, 16, scaling="linear", norm=True, fused=False, prompts=3, p_lo=17, p_hi=333, p_cached=777, reqs=9, new=3, cached_lo=5, cached_hi=3000)},
        # prompts of ragged lengths into the 4-bit cache
        {"name": "q4_prompts", **_case("append_q4", 32, 8, 128, 128, scaling="wavelength", prompts=7, p_lo=1001, p_hi=8192, p_cached=777)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "append_q4"])
    d = rng.choice([64, 128, 128])
    rot = rng.choice([d, d, d, d // 2, d // 4, d - 16])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    hkv = rng.randint(1, 8) if g > 1 else rng.randint(1, 32)
    heads = (g + 2) * hkv
    kind = rng.choice(["decode", "verify", "mixed", "prompts"])
    most = 2_000_000 // heads  # rows, so that no case costs more than the largest listed one
    c = dict(interleaved=rng.random() < 0.3, scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]), norm=rng.random() < 0.3, fused=rng.random() < 0.6)
    if kind in ("mixed", "prompts"):
        hi = _log_int(rng, 2, 8192)
        c.update(prompts=_log_int(rng, 1, max(1, min(32, most // (hi + 200)))), p_lo=_log_int(rng, 1, hi), p_hi=hi, p_cached=rng.randint(0, 20000))
    if kind != "prompts":
        hi = _log_int(rng, 17, 131071)
        new = rng.randint(2, 16) if kind == "verify" else 1
        c.update(reqs=_log_int(rng, 1, 512 // new), new=new, cached_lo=_log_int(rng, 1, hi), cached_hi=hi, tree=kind == "verify" and rng.random() < 0.5)
    return _case(op, g * hkv, hkv, d, rot, **c)


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


def _lengths_of(c, seed):
    """(cached, new) of every request, host int64: a case's lengths are the same for every seed, and the seed orders the requests."""
    g = _gen(0, sum((i + 1) * v for i, v in enumerate(v for v in c.values() if isinstance(v, int))))
    new = torch.cat([_lengths(c["prompts"], c["p_lo"], c["p_hi"], g), torch.full((c["reqs"],), c["new"])])
    cached = torch.cat([torch.full((c["prompts"],), c["p_cached"]), _lengths(c["reqs"], c["cached_lo"], c["cached_hi"], g)])
    order = torch.randperm(len(new), generator=_gen(seed, 1))
    return cached[order], new[order]


def _csr(n):
    return torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])


def _normal(shape, g, spread=None):
    """bf16 values as projections give them: N(0, 1), and with `spread` a few dims eight times as large."""
    dg = torch.Generator(device=DEV)
    dg.manual_seed(int(torch.randint(1 << 40, (1,), generator=g)))
    x = torch.randn(shape, generator=dg, device=DEV, dtype=torch.bfloat16)
    if spread is not None:
        x[..., spread::37] *= 8
    return x


def prepare(case, seed):
    c, g = case, _gen(seed, 2)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    cached, new = _lengths_of(c, seed)
    rows = int(new.sum())
    s = {"case": c}
    first = torch.repeat_interleave(_csr(new)[:-1], new)
    at = torch.arange(rows) - first  # a row's token among its request's new ones
    if c["tree"]:  # nodes numbered parents first, two children each
        at = torch.tensor([(i + 1).bit_length() - 1 for i in range(c["new"] + 1)])[at.clamp(max=c["new"])]
    pos = (torch.repeat_interleave(cached, new) + at).int().to(DEV)
    s["positions"] = pos if c["op"] == "rope" or c["tree"] else None
    if c["fused"]:
        x = _normal((rows, hq + 2 * hkv, d), g, 5)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = _normal((rows, hq, d), g, 5), _normal((rows, hkv, d), g, 5), _normal((rows, hkv, d), g)
    s["q_norm"], s["k_norm"] = ((1 + 0.2 * _normal((d,), g).float()).bfloat16() for _ in range(2)) if c["norm"] else (None, None)
    s["q_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
    if own:
        import decode_attention_append_gb300 as daa
        scaling = {"none": None, "linear": {"type": "linear", "factor": FACTOR}, "ntk": {"type": "ntk", "factor": FACTOR},
                   "yarn": {"type": "yarn", "factor": FACTOR, "original": ORIGINAL, "beta_fast": YARN[0], "beta_slow": YARN[1]},
                   "wavelength": {"type": "wavelength", "factor": FACTOR, "original": ORIGINAL, "low": WAVELENGTH[0], "high": WAVELENGTH[1]}}[c["scaling"]]
        s["rope"] = daa.Rope(d, base=BASE, rotary_dim=c["rot"], interleaved=c["interleaved"], scaling=scaling)
    else:
        s["freq"], s["m"] = _frequencies(c)
    if c["op"] == "rope":
        s["k_out"] = torch.empty(rows, hkv, d, dtype=torch.bfloat16, device=DEV)
        return s
    # pages that receive new tokens are a request's own; those before them hold a prefix that requests share
    kv = cached + new
    np_, whole = (kv + PAGE - 1) // PAGE, cached // PAGE
    kp, mine = _csr(np_), np_ - whole
    num_pages = int(mine.sum()) + 64
    perm = torch.randperm(num_pages, generator=g)
    ids = perm[torch.randint(64, (int(kp[-1]),), generator=g)]
    base = torch.repeat_interleave(kp[:-1] + whole - _csr(mine)[:-1], mine)
    own_at = base + torch.arange(int(mine.sum()))
    ids[own_at] = perm[64:]
    s["t"] = {k: v.int().to(DEV) for k, v in (("qo_indptr", _csr(new)), ("kv_indptr", kp), ("page_indices", ids), ("last_page_len", torch.where(np_ > 0, kv - (np_ - 1) * PAGE, 0)))}
    if c["op"] == "append":
        s["pool"] = _normal((num_pages, 2, hkv, PAGE, d), g)
        return s
    bytes_ = torch.Generator(device=DEV)
    bytes_.manual_seed(int(torch.randint(1 << 40, (1,), generator=g)))
    s["pool"] = torch.randint(256, (num_pages, hkv, 2, 9 * d), generator=bytes_, device=DEV, dtype=torch.uint8)
    s["pool"][..., 8 * d:] = s["pool"][..., 8 * d:] % 24 + 40  # scales from 1/4 to 2
    s["exps"] = torch.randint(-2, 3, (2, hkv), generator=g, dtype=torch.int32).to(DEV)
    s["written"] = ids[own_at].int().to(DEV)
    s["out"] = torch.empty(len(own_at), 2, hkv, PAGE, d, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain form
def _frequencies(c):
    """(f [rot / 2] float64 on the GPU, magnitude) of a case."""
    rot, L = c["rot"], ORIGINAL
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = BASE * FACTOR ** (rot / (rot - 2)) if c["scaling"] == "ntk" else BASE
    f, m = base ** (-2 * i / rot), 1.0
    if c["scaling"] == "linear":
        f = f / FACTOR
    elif c["scaling"] == "yarn":  # pairs that turn often in the original context stay, slow ones are interpolated
        at = lambda turns: rot * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(YARN[0])), 0), min(math.ceil(at(YARN[1])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / FACTOR * ramp + f * (1 - ramp)
        m = 0.1 * math.log(FACTOR) + 1
    elif c["scaling"] == "wavelength":
        low, high = WAVELENGTH
        keep = ((L * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / FACTOR * (1 - keep)
    return f.to(DEV), m


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _turned(s, x, weight, pos, type_):
    """bf16 rows x [rows, heads, d], normalised where there are weights, and rotated; computed in `type_`."""
    c, rot = s["case"], s["case"]["rot"]
    x = x.to(type_)
    if weight is not None:
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * weight.to(type_)
    angle = pos.double()[:, None, None] * s["freq"]
    cos, sin = (angle.cos() * s["m"]).to(type_), (angle.sin() * s["m"]).to(type_)
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _places(s):
    """(page, slot, position) of every new row."""
    t, rows = s["t"], s["q"].shape[0]
    qo, kp = t["qo_indptr"].long(), t["kv_indptr"].long()
    new, np_ = qo[1:] - qo[:-1], kp[1:] - kp[:-1]
    kv = torch.where(np_ > 0, (np_ - 1) * PAGE + t["last_page_len"], 0)
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), new, output_size=rows)
    at = (kv - new)[req] + torch.arange(rows, device=DEV) - qo[req]
    return t["page_indices"][kp[req] + at // PAGE].long(), at % PAGE, at


def _quantise(x, e):
    """Codes (uint8, one a value) and e4m3 scales (uint8, one each 16 dims) of bf16 x [rows, Hkv, d] under exponents e [Hkv]."""
    y = (x.float() * torch.exp2(-e.float())[:, None]).unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=x.device)  # a division: by a Python number torch multiplies by its reciprocal
    scale = (y.abs().amax(-1) / six).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    t = (y / scale.float()[..., None]).abs()
    # nearest value, ties to the even code: a tie goes up only where the upper code is even
    code = ((t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte() + (t > 2.5).byte() + (t >= 3.5).byte() + (t > 5.0).byte())
    code = (code + 8 * torch.signbit(y).byte()).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _dequantised(s):
    """The written pages as bf16 pages."""
    d, x = s["case"]["d"], s["pool"][s["written"].long()]
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=DEV)
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)  # [byte] -> (low, high)
    vals = pairs.index_select(0, x[..., :8 * d].flatten().int()).view(*x.shape[:-1], PAGE, d // 16, 16)
    sc = x[..., 8 * d:].contiguous().view(torch.float8_e4m3fn).float()
    sc = torch.stack([sc[..., 0, :].unflatten(-1, (PAGE, d // 16)), sc[..., 1, :].unflatten(-1, (d // 16, PAGE)).transpose(-1, -2)], 2)
    sc = sc * torch.exp2(s["exps"].float()).T[:, :, None, None]
    return (vals * sc[..., None]).flatten(-2).transpose(1, 2).bfloat16()


def _plain(s):
    c, d = s["case"], s["case"]["d"]
    if c["op"] == "rope":
        return _turned(s, s["q"], s["q_norm"], s["positions"], torch.float32), _turned(s, s["k"], s["k_norm"], s["positions"], torch.float32)
    page, slot, at = _places(s)
    pos = at if s["positions"] is None else s["positions"]
    q = _turned(s, s["q"], s["q_norm"], pos, torch.float32)
    if c["op"] == "append":
        s["pool"][page, 0, :, slot] = _turned(s, s["k"], s["k_norm"], pos, torch.float32)
        s["pool"][page, 1, :, slot] = s["v"]
        return q, s["pool"]
    # a key next to a border between two codes must fall on its own side: rotated in 64 bits
    (ck, sk), (cv, sv) = _quantise(_turned(s, s["k"], s["k_norm"], pos, torch.float64), s["exps"][0]), _quantise(s["v"], s["exps"][1])
    codes, scale = s["pool"][..., :8 * d].unflatten(-1, (PAGE, d // 2)), s["pool"][..., 8 * d:]
    codes[page, :, 0, slot], codes[page, :, 1, slot] = ck, cv
    scale.unflatten(-1, (PAGE, d // 16))[page, :, 0, slot] = sk
    scale.unflatten(-1, (d // 16, PAGE))[page, :, 1, :, slot] = sv
    return q, _dequantised(s)


# ----------------------------------------------------------------------- run
def run(s):
    if not own:
        return _plain(s)
    import decode_attention_append_gb300 as daa
    norms = {} if s["q_norm"] is None else {"q_norm": s["q_norm"], "k_norm": s["k_norm"], "eps": EPS}
    op = s["case"]["op"]
    if op == "rope":
        return daa.apply_rope(s["q"], s["k"], s["positions"], s["rope"], q_out=s["q_out"], k_out=s["k_out"], **norms)
    t = s["t"]
    if op == "append":
        q = daa.append_rope(s["q"], s["k"], s["v"], s["pool"], t["qo_indptr"], t["page_indices"], t["kv_indptr"], t["last_page_len"], s["rope"], positions=s["positions"], q_out=s["q_out"], **norms)
        return q, s["pool"]
    q = daa.append_rope_q4(s["q"], s["k"], s["v"], s["pool"], t["qo_indptr"], t["page_indices"], t["kv_indptr"], t["last_page_len"], s["rope"], positions=s["positions"], kv_exp=s["exps"],
                           q_out=s["q_out"], **norms)
    return q, daa.kv_dequant_q4(s["pool"], s["written"], kv_exp=s["exps"], out=s["out"])


# ---------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass."""
    c, d = case, case["d"]
    cached, new = _lengths_of(c, 0)
    rows, heads = int(new.sum()), c["hq"] + c["hkv"]
    turned = rows * heads * (3 * c["rot"] + (4 * d if c["norm"] else 0))  # two products and a sum a value; a square, a sum and two products
    if c["op"] == "rope":
        return {"bytes": rows * (heads * d * 4 + 4), "flops": turned}
    if c["op"] == "append":
        return {"bytes": rows * ((heads + c["hkv"]) * d * 4 + 4) + 16 * len(new), "flops": turned}
    values = rows * c["hkv"] * 2 * d
    back = int((((cached + new) + PAGE - 1) // PAGE - cached // PAGE).sum()) * c["hkv"] * 2 * PAGE * d
    return {"bytes": rows * (c["hq"] * d * 4 + 4) + 16 * len(new) + values * (2 + 9 / 16) + back * (9 / 16 + 2), "flops": turned + 4 * values + back}


# --------------------------------------------------------------------- exact
def _exact_turns(c):
    """Radians a token of every pair, and the magnitude: the definitions, a pair at a time."""
    rot, got = c["rot"], []
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(BASE))
        turns = ORIGINAL * f / (2 * math.pi)  # in the original context
        if c["scaling"] == "linear":
            f /= FACTOR
        elif c["scaling"] == "ntk":  # the first pair as it was, the last one slower by the factor
            f *= FACTOR ** (-2 * i / (rot - 2))
        elif c["scaling"] == "yarn":
            bounds = [rot / 2 * math.log(ORIGINAL / (2 * math.pi * b)) / math.log(BASE) for b in YARN]
            lo, hi = max(math.floor(bounds[0]), 0), min(math.ceil(bounds[1]), rot - 1)
            share = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - share + share / FACTOR)
        elif c["scaling"] == "wavelength" and turns < WAVELENGTH[1]:
            share = max(0.0, (turns - WAVELENGTH[0]) / (WAVELENGTH[1] - WAVELENGTH[0]))
            f = share * f + (1 - share) * f / FACTOR
        got.append(f)
    return torch.tensor(got, dtype=torch.float64, device=DEV), 1 + 0.1 * math.log(FACTOR) if c["scaling"] == "yarn" else 1.0


def _exact_rows(c, x, weight, pos):
    """float64: pairs as complex numbers times m e^(i p f)."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    f, m = _exact_turns(c)
    turn = torch.polar(torch.full((), m, dtype=torch.float64, device=DEV).expand(len(pos), len(f)).contiguous(), pos.double()[:, None] * f)[:, None]
    rot = c["rot"]
    head = x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2) if c["interleaved"] else x[..., :rot].reshape(*x.shape[:-1], 2, rot // 2).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    out = x.clone()
    out[..., :rot] = (z if c["interleaved"] else z.transpose(-1, -2)).reshape(*x.shape[:-1], rot)
    return out


def _two_to(n):
    """2^n of whole numbers -64 .. 63 in float64, from a table made on the host (a GPU's pow is not exact)."""
    return torch.tensor([2.0 ** i for i in range(-64, 64)], dtype=torch.float64).to(n.device)[n.long() + 64]


def _exact_values(x, e):
    """float64 values that the 4-bit cache holds for x [rows, Hkv, d] under exponents e [Hkv]: the definition, by nearest neighbours."""
    two = _two_to(e)[:, None, None]
    y = x.bfloat16().double().reshape(*x.shape[:-1], -1, 16) / two
    m = torch.arange(1, 127, device=DEV, dtype=torch.float64)  # every positive e4m3 number in the order of its code, 2^-9 to 448
    ex, fr = torch.div(m, 8, rounding_mode="floor"), m % 8
    grid = torch.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * _two_to(ex - 10))

    def nearest(v, grid, first):
        mid = (grid[1:] + grid[:-1]) / 2
        i = torch.searchsorted(mid, v.contiguous())  # ties to the lower code
        tie = v == mid[i.clamp(max=len(mid) - 1)]
        return i + (tie & ((i + first) % 2 == 1)).long()  # and to the even one

    sc = grid[nearest(y.abs().amax(-1), 6 * grid, 1)].unsqueeze(-1)  # nearest to a sixth
    e2m1 = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device=DEV, dtype=torch.float64) / 2
    return (torch.copysign(e2m1[nearest(y.abs() / sc, e2m1, 0)], y) * sc * two).reshape(x.shape)


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
    sc = sc * _two_to(exps).T[None, :, :, None, None]
    return (val.view(n, hkv, 2, PAGE, d // 16, 16) * sc[..., None]).view(n, hkv, 2, PAGE, d).transpose(1, 2)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        return _exact_rows(c, s["q"], s["q_norm"], s["positions"]), _exact_rows(c, s["k"], s["k_norm"], s["positions"])
    # every row's place, request by request
    cached, new = _lengths_of(c, seed)
    first_page, at, ids = s["t"]["kv_indptr"].tolist(), [], s["t"]["page_indices"].cpu()
    places = [torch.arange(a, a + n) for a, n in zip(cached.tolist(), new.tolist())]
    page = torch.cat([ids[p0 + x // PAGE] for p0, x in zip(first_page, places)]).long().to(DEV)
    at = torch.cat(places).to(DEV)
    pos = at if s["positions"] is None else s["positions"]
    q, k = _exact_rows(c, s["q"], s["q_norm"], pos), _exact_rows(c, s["k"], s["k_norm"], pos)
    if c["op"] == "append":
        pool = s["pool"].double()
        pool[page, 0, :, at % PAGE], pool[page, 1, :, at % PAGE] = k, s["v"].double()
        return q, pool
    out = _exact_pages(s["pool"][s["written"].long()], c["d"], s["exps"])
    where = torch.full((s["pool"].shape[0],), -1, dtype=torch.long, device=DEV)
    where[s["written"].long()] = torch.arange(len(s["written"]), device=DEV)
    out[where[page], 0, :, at % PAGE] = _exact_values(k, s["exps"][0])
    out[where[page], 1, :, at % PAGE] = _exact_values(s["v"].double(), s["exps"][1])
    return q, out
