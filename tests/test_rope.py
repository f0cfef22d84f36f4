"""Host side of the rotary positions: frequencies and their scalings, the rotation's record, and refusals
(found before anything is enqueued).  No GPU."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import rope_support as ref

OK, INVALID, SHAPE, UNSUPPORTED, ALIGNMENT = 0, -1, -2, -4, -7
A = 0x100000  # an address that passes a null and alignment check and is never read


_rec = struct.Struct("@PqqPqqPqqPqqPqqiPPPf0P").pack  # daa_rope_rows


@pytest.fixture(scope="module")
def daa():
    from decode_attention_append_gb300 import build
    build.build()
    import decode_attention_append_gb300 as m
    m.load_library()
    return m


SCALINGS = [None, dict(type="linear", factor=4.0), dict(type="ntk", factor=8.0), dict(type="yarn", factor=16.0, original=4096),
            dict(type="yarn", factor=2.5, original=100, beta_fast=4.0, beta_slow=2.0),
            dict(type="wavelength", factor=8.0, original=8192), dict(type="wavelength", factor=3.0, original=77, low=0.5, high=1.5)]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("n,base", [(16, 10000.0), (64, 500000.0), (96, 10000.0), (128, 1e6)])
def test_frequencies(daa, scaling, n, base):
    f, m = daa.rope_frequencies(n, base, scaling)
    o = dict(scaling or {})
    kind = o.pop("type", None)
    names = {"factor": "s", "original": "original", "beta_fast": "fast", "beta_slow": "slow", "low": "low", "high": "high"}
    want = ref.frequencies(n, base, kind, **{names[k]: v for k, v in o.items()})
    # powers and mixtures in 64 bits: some tens of roundings of 2^-53, those of an exponent up to 14 times as large
    assert np.allclose(f, want, rtol=1e-13, atol=0)
    assert m == (pytest.approx(0.1 * math.log(o["factor"]) + 1, rel=1e-15) if kind == "yarn" else 1.0)
    r = daa.Rope(128 if n > 64 else 64, base, n, scaling=scaling)
    assert np.array_equal(r.frequencies, f) and r.magnitude == m and r._rope.magnitude == m


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=15), dict(rotary_dim=0), dict(base=0.0), dict(base=float("nan")), dict(scaling=dict(type="other", factor=2)),
    dict(scaling=dict(factor=2)), dict(scaling=dict(type="linear")), dict(scaling=dict(type="linear", factor=0.5)),
    dict(scaling=dict(type="linear", factor=2, original=4)), dict(scaling=dict(type="ntk", factor=float("inf"))),
    dict(scaling=dict(type="yarn", factor=2)), dict(scaling=dict(type="yarn", factor=2, original=0)),
    dict(scaling=dict(type="yarn", factor=2, original=64, beta_fast=1, beta_slow=2)), dict(scaling=dict(type="yarn", factor=2, original=64), base=1.0),
    dict(scaling=dict(type="wavelength", factor=2, original=64, low=4, high=4)), dict(scaling=dict(type="ntk", factor=2), rotary_dim=2),
])
def test_frequency_refusals(daa, bad):
    with pytest.raises(ValueError):
        daa.rope_frequencies(**{"rotary_dim": 64, **bad})


def test_turns_are_exact(daa):
    """A pair's turns a token, as 2^-64 of a turn: within one unit of the value by whole numbers."""
    f = np.array([0.0, 1.0, 2 * math.pi, math.pi, 1e-9, -1e-9, -1.0, 0.3, 123456.789, -1048576.0, 1048576.0, 5e-324, 1e-20, 2.5, 1e-4, 0.7])
    r = daa.Rope(64, rotary_dim=32, frequencies=f)
    for x, got in zip(f, r._rope.turns):
        n, d = float(x).as_integer_ratio()
        want = n * 10 ** 60 * 2 ** 63 // (d * ref._PI)  # x / 2 pi in units of 2^-64
        off = (got - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, (x, got, want)


def test_angles_of_far_positions(daa):
    """p times a pair's turns, modulo one, is off by p 2^-65 turns at most: 2^-41 of a turn at 2^24, 2^-34 at the last position."""
    f = ref.frequencies(128, 500000.0)
    r = daa.Rope(128, frequencies=f)
    for p in (1, 131_071, 2 ** 24, -2 ** 24, 2 ** 31 - 1, -2 ** 31):
        for x, turns in zip(f, r._rope.turns):
            n, d = float(x).as_integer_ratio()
            want = p * n * 10 ** 60 * 2 ** 79 // (d * ref._PI)  # p x / 2 pi in units of 2^-80
            off = ((p * turns << 16) - want) % 2 ** 80
            assert min(off, 2 ** 80 - off) <= abs(p) * (2 ** 15 + 1) + 1, (p, x)


@pytest.mark.parametrize("change,expect", [
    (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=80), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED),
    (dict(inter=2), INVALID), (dict(m=0.0), INVALID), (dict(m=-1.0), INVALID), (dict(m=float("nan")), INVALID), (dict(m=1e300), INVALID),
    (dict(m=1e-60), INVALID), (dict(f=float("inf")), INVALID), (dict(f=float("nan")), INVALID), (dict(f=1048577.0), INVALID), (dict(f=None), INVALID), (dict(out=False), INVALID), ({}, OK),
])
def test_rope_init_refusals(daa, change, expect):
    c = dict(d=64, rot=64, inter=0, m=1.0, f=0.5, out=True)
    c.update(change)
    f = np.full(64, 0.25 if c["f"] is None else c["f"])
    r = daa._Rope()
    r.magnitude = 77.0
    st = daa.load_library().daa_rope_init(ctypes.byref(r) if c["out"] else None, c["d"], c["rot"], c["inter"],
                                          None if c["f"] is None else f.ctypes.data_as(ctypes.c_void_p), c["m"])
    assert st == expect
    assert (r.magnitude == 77.0) == (expect != OK)  # refused: left as it was


def test_python_refusals(daa):
    for kw in (dict(frequencies=[1.0]), dict(frequencies=[float("nan")] * 32), dict(frequencies=[1.0] * 32, scaling=dict(type="linear", factor=2))):
        with pytest.raises(ValueError):
            daa.Rope(64, **kw)
    for kw in (dict(rotary_dim=40), dict(magnitude=0.0)):
        with pytest.raises(daa.DaaError):
            daa.Rope(64, **kw)
    x, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    rope = daa.Rope(64)
    with pytest.raises(TypeError):
        daa.apply_rope(x, x, pos, rope)
    with pytest.raises(TypeError):
        daa.append_rope(x, x, x, torch.zeros(4, 2, 2, 16, 64, dtype=torch.bfloat16), pos, pos, pos, pos, rope)
    with pytest.raises(TypeError):
        daa.append_rope_q4(x, x, x, torch.zeros(4, 2, 2, 9 * 64, dtype=torch.uint8), pos, pos, pos, pos, rope)


def test_copies_of_a_rope_stand_alone(daa):
    import copy
    import gc
    import pickle
    r = daa.Rope(128, rotary_dim=64, interleaved=True, scaling=dict(type="yarn", factor=4.0, original=512))
    want = bytes(r._rope)
    others = [copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))]
    f = r.frequencies
    f[:] = 0  # a copy
    assert r.frequencies.all()
    del r
    gc.collect()
    for o in others:
        assert daa._rope_addr(o) == ctypes.addressof(o._rope) and bytes(o._rope) == want
        assert o.magnitude == others[0].magnitude and np.array_equal(o.frequencies, others[0].frequencies)


def _append(daa, q4=False, batch=0, rope=None, pool=0x70000000, table=A, dims=(4, 2, 64, 16, 64), rows=8, **change):
    """An append of 8 rows that cannot launch: with batch 0 it is refused as SHAPE once its rows are accepted."""
    T = 512  # elements of a projection's row: q, k, v
    io = dict(q=(A, T, 64), k=(A + 512, T, 64), v=(A + 768, T, 64), q_out=(0x900000, 256, 64), k_out=(0, 0, 0), pos=0, qn=0, kn=0, eps=1e-6)
    io.update(change)
    rec = _rec(*io["q"], *io["k"], *io["v"], *io["q_out"], *io["k_out"], rows, io["pos"], io["qn"], io["kn"], io["eps"])
    rope = daa.Rope(64) if rope is None else rope
    lib = daa.load_library()
    tab = [table, A, A, A]
    if q4:
        return lib.daa_append_rope_q4(ctypes.addressof(rope._rope), rec, pool, None, *tab, batch, daa._Dims(*dims), None)
    return lib.daa_append_rope(ctypes.addressof(rope._rope), rec, pool, *tab, batch, daa._Dims(*dims), None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("change,expect", [
    (dict(), SHAPE), (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(batch=-1), INVALID), (dict(dims=(4, 2, 128, 16, 64)), INVALID),
    (dict(dims=(4, 2, 96, 16, 64)), UNSUPPORTED), (dict(dims=(4, 2, 64, 32, 64)), UNSUPPORTED), (dict(dims=(3, 2, 64, 16, 64)), INVALID),
    (dict(batch=2, pool=None), INVALID), (dict(batch=2, table=None), INVALID), (dict(batch=2, pool=0x70000008), ALIGNMENT), (dict(batch=2, table=A + 2), ALIGNMENT),
    (dict(k=(0, 512, 64)), INVALID), (dict(v=(0, 512, 64)), INVALID), (dict(q_out=(0, 256, 64)), INVALID),
    (dict(q=(0, 0, 0)), INVALID), (dict(q=(0, 0, 0), q_out=(0, 0, 0)), SHAPE),
    (dict(q=(A + 8, 512, 64)), ALIGNMENT), (dict(k=(A + 512, 508, 64)), ALIGNMENT), (dict(v=(0x50000, 512, 68)), ALIGNMENT),
    (dict(k=(A + 512, -512, 64)), INVALID), (dict(k=(A + 512, 1 << 41, 64)), INVALID), (dict(pos=A + 2), ALIGNMENT), (dict(kn=A + 1), ALIGNMENT),
    (dict(kn=A, eps=-1.0), INVALID), (dict(qn=A, eps=float("nan")), INVALID), (dict(eps=float("nan")), SHAPE),
    (dict(rows=2 ** 31 - 1), UNSUPPORTED),
    # inputs may be broadcast, outputs may not
    (dict(v=(0x50000, 0, 0)), SHAPE), (dict(q_out=(0x900000, 0, 64)), INVALID), (dict(q_out=(0x900000, 256, 0)), INVALID), (dict(q_out=(0x900000, 248, 64)), INVALID),
    (dict(q_out=(0x900000, 64, 512)), SHAPE), (dict(q_out=(0x900000, 64, 504)), INVALID), (dict(rows=1, q_out=(0x900000, 3, 64)), SHAPE), (dict(rows=1, q_out=(0x900000, 3, 56)), INVALID),
    # in place, beside one another, and across
    (dict(q_out=(A, 512, 64)), SHAPE), (dict(q_out=(A, 256, 64)), INVALID), (dict(q_out=(A + 16, 512, 64)), INVALID), (dict(q_out=(A + 512, 512, 64)), INVALID),
    (dict(q_out=(A + 256, 512, 64)), INVALID), (dict(q=(0x50000, 512, 64), q_out=(A, 512, 64)), SHAPE), (dict(q=(0x50000, 512, 64), q_out=(A + 128, 512, 64)), INVALID),
    (dict(q=(0x50000, 512, 64), k=(0x50000 + 512, 512, 64), v=(0x50000 + 768, 512, 64), q_out=(0x50000 + 1024 * 8, 512, 64)), SHAPE),
    (dict(q=(0x50000, 512, 64), k=(0x50000 + 512, 512, 64), v=(0x50000 + 768, 512, 64), q_out=(0x50000 + 1024 * 7, 512, 64)), INVALID),
    # strides of one row or head are not looked at
    (dict(rows=1, k=(A + 512, -8, 64)), SHAPE), (dict(rows=1, dims=(2, 1, 64, 16, 64), k=(A + 512, 1 << 50, -3)), SHAPE), (dict(rows=2, dims=(2, 1, 64, 16, 64), k=(A + 512, 512, 1)), SHAPE),
    # positions and weights under an output
    (dict(pos=0x900000 + 4092), INVALID), (dict(pos=0x900000 + 4096), SHAPE), (dict(pos=0x900000 - 28), INVALID), (dict(pos=0x900000 - 32), SHAPE),
    (dict(qn=0x900000), INVALID), (dict(kn=0x900000 - 126), INVALID), (dict(kn=0x900000 - 128), SHAPE),
    # heads of q, k and v between one another: [rows][heads][q, k, v][64]
    (dict(q=(A, 768, 192), k=(A + 128, 768, 192), v=(A + 256, 768, 192), q_out=(A, 768, 192)), SHAPE),
    (dict(q=(A, 768, 192), k=(A + 128, 768, 192), v=(A + 192, 768, 192), q_out=(A + 128, 768, 192)), INVALID),
])
def test_append_refusals(daa, change, expect, q4):
    assert _append(daa, q4, **change) == expect


@pytest.mark.parametrize("name", ["q", "k", "v", "q_out"])
def test_rows_within_the_pool_are_refused(daa, name):
    """The pool's 64 pages of 2 x 2 x 16 x 64 values at 0x70000000: 524,288 bytes."""
    end = 0x70000000 + 64 * 2 * 2 * 16 * 64 * 2
    for at, expect in ((0x70000000, INVALID), (end - 16, INVALID), (end, SHAPE)):
        # with a batch, so that the pool is looked at: a misaligned table ends what is accepted
        got = _append(daa, batch=0 if expect == SHAPE else 2, **{name: (at, 1024, 64)})
        assert got == expect, (name, hex(at))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("name,size", [("append_indptr", 12), ("page_indices", 4), ("kv_indptr", 12), ("last_page_len", 8), ("kv_exp", 16), ("pos", 32), ("qn", 128), ("kn", 128)])
def test_tables_under_what_is_written_are_refused(daa, q4, name, size):
    """A table, positions or weights in the pool (64 pages) or under the rotated queries.  Found once everything else is in
    order: not on a machine where a call that is not refused would launch."""
    if torch.cuda.is_available():
        pytest.skip("addresses that are none")
    if name == "kv_exp" and not q4:
        pytest.skip("bf16 pages have no exponents")
    pool = 0x70000000
    pool_end = pool + 64 * 2 * 2 * (9 * 64 if q4 else 2 * 16 * 64)
    q_out, q_end = 0x900000, 0x900000 + 8 * 256 * 2
    lib, rope = daa.load_library(), daa.Rope(64)
    for at in (pool, pool_end - 4, pool - size + 4, q_out, q_end - 4, q_out - size + 4):
        where = dict(append_indptr=0x10000, page_indices=0x20000, kv_indptr=0x30000, last_page_len=0x40000, kv_exp=0, pos=0, qn=0, kn=0)
        where[name] = at
        rec = _rec(A, 512, 64, A + 512, 512, 64, A + 768, 512, 64, q_out, 256, 64, 0, 0, 0, 8, where["pos"], where["qn"], where["kn"], 1e-6)
        tab = [where[x] for x in ("append_indptr", "page_indices", "kv_indptr", "last_page_len")]
        args = (ctypes.addressof(rope._rope), rec, pool)
        if q4:
            st = lib.daa_append_rope_q4(*args, where["kv_exp"] or None, *tab, 2, daa._Dims(4, 2, 64, 16, 64), None)
        else:
            st = lib.daa_append_rope(*args, *tab, 2, daa._Dims(4, 2, 64, 16, 64), None)
        assert st == INVALID, hex(at)


def test_bad_records_are_refused(daa):
    lib = daa.load_library()
    rope = daa.Rope(64)
    rec = _rec(A, 64, 64, 0, 0, 0, 0, 0, 0, 0x900000, 64, 64, 0, 0, 0, 8, A, 0, 0, 0.0)
    assert lib.daa_apply_rope(None, rec, 1, 0, None) == INVALID
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), None, 1, 0, None) == INVALID
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), rec, 0, 1, None) == INVALID
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), rec, 1, -1, None) == INVALID
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), rec, 1, 1, None) == INVALID  # no k
    none = _rec(A, 64, 64, 0, 0, 0, 0, 0, 0, 0x900000, 64, 64, 0, 0, 0, 8, 0, 0, 0, 0.0)
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), none, 1, 0, None) == INVALID  # no positions
    empty = _rec(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.0)
    assert lib.daa_apply_rope(ctypes.addressof(rope._rope), empty, 1, 1, None) == OK
    other = daa._Rope.from_buffer_copy(bytes(rope._rope))
    for field, value, expect in (("rotary_dim", 72, UNSUPPORTED), ("head_dim", 32, UNSUPPORTED), ("interleaved", 7, INVALID), ("magnitude", -1.0, INVALID)):
        bad = daa._Rope.from_buffer_copy(bytes(other))
        setattr(bad, field, value)
        assert lib.daa_apply_rope(ctypes.byref(bad), rec, 1, 0, None) == expect


def test_reference_keeps_lengths_and_relative_angles():
    """A rotation keeps a pair's length (m = 1), and products of two rotated heads depend on the distance alone."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 64))
    for inter in (False, True):
        f = ref.frequencies(32)
        dots = []
        for p in ((3, 10), (1_000_003, 1_000_010), (-7, 0)):
            y, _ = ref.rotate(x, p, f, 32, inter)
            assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
            dots.append((y[0] * y[1]).sum())
        assert np.allclose(dots, dots[0], rtol=1e-12)
