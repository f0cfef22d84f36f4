"""Appends on page tables that do not hold: refused with the error word, nothing written for the request, and the
others as ever.  What the tables would lead to is checked on the CPU by test_place.py."""
import numpy as np
import pytest
import torch

import q4_support

pytestmark = pytest.mark.gpu
DEV = "cuda"
BIG, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.fixture(scope="module")
def daa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_append_gb300 as m
    m.device_error(reset=True)
    return m


def _i32(x):
    return torch.from_numpy(np.array(x, np.int32)).to(DEV)


def _append(daa, kind, rows, pool, qo, ids, kv, last):
    """One append of `rows` ones by the call of that kind; the rotated queries, where there are any, else None."""
    x = torch.ones(rows, 2, 64, dtype=torch.bfloat16, device=DEV)
    tab = _i32(qo), _i32(ids), _i32(kv), _i32(last)
    if kind == "plain":
        return daa.kv_append(x, x, pool, *tab)
    if kind == "q4":
        return daa.kv_append_q4(x, x, pool, *tab)
    out = torch.full((rows, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    call = daa.append_rope_q4 if kind == "rope_q4" else daa.append_rope
    call(torch.ones(rows, 4, 64, dtype=torch.bfloat16, device=DEV), x, x, pool, *tab, daa.Rope(64), q_out=out)
    return out


def _pool(kind, n=8):
    return torch.zeros(n, 2, 2, 9 * 64, dtype=torch.uint8, device=DEV) if "q4" in kind else torch.zeros(n, 2, 2, 16, 64, dtype=torch.bfloat16, device=DEV)


# a table of one request of 3 rows, or what becomes of it
BAD = [
    dict(qo=[-1, BIG]), dict(qo=[-5, 3]), dict(qo=[LOW, 3]), dict(qo=[LOW, BIG]), dict(qo=[0, BIG]), dict(qo=[0, 17]),
    dict(kv=[-1, 1]), dict(kv=[LOW, 1]), dict(kv=[LOW, BIG]), dict(kv=[0, BIG], last=[0]), dict(kv=[0, -3]), dict(kv=[1, 1]), dict(kv=[5, 4]), dict(kv=[BIG, LOW]),
    dict(last=[17]), dict(last=[0]), dict(last=[BIG]), dict(last=[LOW]),
]


@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("kind", ["plain", "q4", "rope", "rope_q4"])
def test_one_request(daa, kind, bad):
    t = {"qo": [0, 3], "kv": [0, 1], "last": [16], **bad}
    pool = _pool(kind)
    out = _append(daa, kind, 3, pool, t["qo"], [4], t["kv"], t["last"])
    assert daa.device_error(reset=True) == 3
    assert not pool.any() and (out is None or (out == 7).all())


@pytest.mark.parametrize("qo,never", [([0, 5, 2, 8], [3]), ([0, 2, BIG, 8], [3]), ([0, 2, -7, 8], [3, 6]), ([-3, 2, 5, 8], [1])])
@pytest.mark.parametrize("kind", ["plain", "q4", "rope", "rope_q4"])
def test_starts_that_fall_or_run_ahead(daa, kind, qo, never):
    """8 rows, 3 requests of one page each: rows go to their request's page or nowhere.  Where starts fall, rows 2 to 4 are
    those of two requests, and it is open which of them a search finds; else there are rows of none that fits."""
    pool = _pool(kind)
    _append(daa, kind, 8, pool, qo, [1, 3, 6], [0, 1, 2, 3], [16, 16, 16])
    assert daa.device_error(reset=True) in ((0, 3) if qo == [0, 5, 2, 8] else (3,))
    used = {int(p) for p in pool.flatten(1).any(1).nonzero().flatten()}
    assert used <= {1, 3, 6} - set(never)


@pytest.mark.parametrize("kind", ["plain", "q4", "rope", "rope_q4"])
def test_the_others_are_as_ever(daa, kind):
    """A request whose words do not fit between two that do."""
    rng = np.random.default_rng(1)
    t, n = q4_support.make_table(rng, [10, 3, 40], [4, 5, 2])
    good, bad = _pool(kind, n), _pool(kind, n)
    want = _append(daa, kind, 11, good, t["qo_indptr"], t["page_indices"], t["kv_indptr"], t["last_page_len"])
    assert daa.device_error(reset=True) == 0
    last = t["last_page_len"].copy()
    last[1] = LOW
    out = _append(daa, kind, 11, bad, t["qo_indptr"], t["page_indices"], t["kv_indptr"], last)
    assert daa.device_error(reset=True) == 3
    mine = t["page_indices"][t["kv_indptr"][1]:t["kv_indptr"][2]]
    assert not bad[mine.tolist()].any()
    good[mine.tolist()] = 0
    assert torch.equal(bad, good)
    assert out is None or (torch.equal(out[:4], want[:4]) and torch.equal(out[9:], want[9:]) and (out[4:9] == 7).all())
