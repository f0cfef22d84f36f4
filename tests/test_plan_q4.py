"""Host logic of the plan of attention over the 4-bit cache, on the CPU: every
(new token, page) of a request is in exactly one unit, or the request is one of
those that go by way of bf16 pages; ranges hold consecutive units of one class
and cost about the same; every part is merged once, in order."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, NATIVE = 16, 96


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ unavailable")
    inc = [os.path.join(ROOT, "include"), os.path.join(ROOT, "decode_attention_append_gb300", "csrc"),
           os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    exe = str(tmp_path_factory.mktemp("plan") / "plan_q4_check")
    cmd = [gxx, "-std=c++17", "-O1", *sum((["-I", i] for i in inc), []),
           os.path.join(ROOT, "tests", "plan_q4_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def _plan(exe, hq, hkv, d, sms, cached, new):
    cached, new = np.asarray(cached, int), np.asarray(new, int)
    kv = cached + new
    np_ = -(-kv // P)
    qo, kp = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(np_)])
    last = np.where(np_ > 0, kv - (np_ - 1) * P, 0)
    text = f"{hq} {hkv} {d} {P} 1000000 {sms}\n{len(new)}\n" + "\n".join(" ".join(map(str, x)) for x in (qo, kp, last)) + "\n"
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    got = {k: [] for k in "URMDXLS"}
    for ln in out.splitlines():
        f = ln.split()
        if f[0] != "E":
            got[f[0]].append(tuple(map(int, f[1:])))
    assert got["S"] == [(0,)]
    return got, qo, kp, kv


def _few(long, new, kv, g, hkv, sms):
    """Whether the long requests' 24-row units are few for the GPU (units times kv heads,
    against their longest key range)."""
    warps = hkv * sum(-(-new[r] // max(1, 24 // g)) for r in long)
    keys = max(int(kv[r]) for r in long)
    split = any(new[r] <= 2 * (128 // g) for r in long)
    if warps <= 0.6 * sms:
        return not split or warps * keys <= 150000
    return not split and warps <= 2 * sms - 160000 // keys


@pytest.mark.parametrize("hq,hkv,d,cached,new", [
    (32, 32, 128, [500] * 7 + [4000] * 5, [1] * 12), (12, 1, 128, [100, 30000, 9000, 0], [1, 1, 1, 1]),
    (32, 8, 128, [1000, 50, 0, 7], [5, 0, 1, 3]), (16, 1, 64, [400, 8000], [4, 1]),
    (8, 2, 64, [3, 0, 900], [24, 25, 1]), (4, 2, 64, [48, 39, 72], [16, 1, 1]), (3, 3, 128, [0] * 700, [1] * 700),
    (40, 8, 128, [2000, 100, 33, 64], [1, 20, 19, 300]), (1, 1, 64, [], []), (2, 1, 128, [5, 6], [0, 0]),
    (16, 16, 128, list(range(0, 3000, 37)), [1 + i % 9 for i in range(82)]), (7, 1, 128, [100000], [1]),
    (7, 1, 64, [3860, 40], [108, 1]), (4, 1, 128, [16000], [512]), (8, 2, 128, [4000, 9, 100], [128, 1, 30]),
])
@pytest.mark.parametrize("sms", [152, 3])
def test_units_cover_every_token_and_page_once(harness, hq, hkv, d, cached, new, sms):
    got, qo, kp, kv = _plan(harness, hq, hkv, d, sms, cached, new)
    g = hq // hkv
    long = [r for r in range(len(new)) if new[r] * g > NATIVE]
    if not got["X"]:  # none, or so few that the 4-bit pages are better for them, too
        assert not long or _few(long, new, kv, g, hkv, sms)
        long = []
    native = [r for r in range(len(new)) if 0 < new[r] and r not in long]
    seen = {(r, t): np.zeros(kp[r + 1] - kp[r], int) for r in native for t in range(new[r])}
    slots = {}
    owner = {int(qo[r] + t): (r, t) for r in native for t in range(new[r])}
    for u, (row, n, pos0, kvlen, base, lo, hi, part, stride) in enumerate(got["U"]):
        r, t0 = owner[row]
        assert kvlen == kv[r] and base == kp[r] and pos0 == kv[r] - new[r] + t0 and n * g <= 24
        assert lo % P == 0 and lo < hi <= kvlen and (hi % P == 0 or hi == kvlen)
        for t in range(t0, t0 + n):
            assert owner[row + t - t0] == (r, t)
            seen[r, t][lo // P:-(-hi // P)] += 1
            if part >= 0:
                slots[row + t - t0, part + (t - t0) * stride] = lo
    assert all((v == 1).all() for v in seen.values())
    # the parts of a token lie side by side, in key order, and are merged once; a token without parts has one unit
    merged = {}
    for row, begin, n in got["M"]:
        assert row not in merged and n > 1
        merged[row] = range(begin, begin + n)
        los = [slots.pop((row, s)) for s in merged[row]]
        assert los == sorted(los) and los[0] == 0
    assert not slots
    assert len({s for m in merged.values() for s in m}) == sum(map(len, merged.values())) == got["L"][0][0]
    # ranges: consecutive units, one class each, costs within a unit of each other
    at = 0
    for b, e, c in got["R"]:
        assert b == at < e
        at = e
        assert all((8 * c < u[1] * g <= 8 * c + 8) for u in got["U"][b:e])
    assert at == len(got["U"])
    for c in range(3):
        cost = [sum(-(-(u[6] - u[5]) // P) + (5, 7, 7)[c] for u in got["U"][b:e]) for b, e, k in got["R"] if k == c]
        assert len(cost) <= sms * (16 if c == 0 else 8) * (2 if long else 1)
        if len(cost) > 1 and len(cost) > 4:
            assert max(cost) <= np.mean(cost) + 8
    # the others: their pages once each, and every row in an item whose pages are theirs
    scratch = {}
    for r in long:
        scratch[r] = len(scratch) and sum(int(kp[x + 1] - kp[x]) for x in scratch)
    assert [x[0] for x in got["X"]] == [int(kp[r]) + p for r in long for p in range(kp[r + 1] - kp[r])]
    rows = {int(qo[r] + t): r for r in long for t in range(new[r])}
    covered = set()
    for row0, base, kvlen, qlen, tok0, n, lo, hi in got["D"]:
        r = rows[row0]
        assert kvlen == kv[r] and base == scratch[r] and qlen == new[r] and 0 <= lo < hi <= kvlen
        covered |= {row0 + tok0 + t for t in range(n)}
    assert covered == set(rows)
    assert got["L"][0][1] == len(got["X"])


@pytest.mark.parametrize("hq,hkv,cached,new,native", [
    (7, 1, [3860], [108], True),              # one chunk, one kv head: seven SMs' worth of tiles
    (32, 8, [1536], [512], False),            # tiles for 64 SMs, 688 units
    (32, 8, [1536, 900], [64, 1], True), (32, 8, [16000], [64], False),
    (64, 8, [8192, 8192], [8192, 8192], False), (12, 1, [16000, 5], [170, 1], True),
    (12, 1, [16000, 16000, 16000, 16000, 16000], [170] * 5, False),
])
def test_few_long_chunks_stay_on_the_4_bit_pages(harness, hq, hkv, cached, new, native):
    got, *_ = _plan(harness, hq, hkv, 128, 152, cached, new)
    assert (not got["X"]) == native and bool(got["U"]) == (native or 1 in new)
