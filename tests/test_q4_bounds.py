"""The bounds of q4_bounds: right values pass, and a V page that is negated, left out, counted twice
or changed for another is seen at any place of a long context (no GPU)."""
import numpy as np
import pytest
import torch

import q4_bounds
import q4_support as ref


def _case(seed, hq, hkv, d, cached, new):
    rng = np.random.default_rng(seed)
    t, n = ref.make_table(rng, cached, new)
    pool = np.concatenate([rng.integers(0, 256, (n, hkv, 2, 8 * d), dtype=np.uint8),
                           rng.integers(40, 64, (n, hkv, 2, d), dtype=np.uint8)], -1)
    q = torch.from_numpy(rng.standard_normal((int(t["qo_indptr"][-1]), hq, d))).bfloat16().double().numpy()
    return t, pool, q


def test_pages_add_up():
    t, pool, q = _case(5, 6, 2, 64, [77, 0, 40], [1, 3, 2])
    for causal in (True, False):
        want = ref.attention(q, pool, t, None, 64, 0.125, causal)
        for r in range(3):
            rows = slice(t["qo_indptr"][r], t["qo_indptr"][r + 1])
            for got, w in zip(q4_bounds.by_page(q, pool, t, r, 64, 0.125, causal), (want[0], want[2], want[4])):
                assert np.allclose(got.sum(0), w[rows], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("weight", [q4_bounds.FP16, q4_bounds.BF16])
@pytest.mark.parametrize("hq,hkv,d,cached,new", [(2, 2, 128, [5003], [1]), (4, 1, 128, [9001, 4095], [1, 1]), (16, 1, 64, [3001], [4])])
def test_a_wrong_v_page_is_seen(hq, hkv, d, cached, new, weight):
    t, pool, q = _case(3, hq, hkv, d, cached, new)
    scale = 1 / d ** 0.5
    B = ref.attention(q, pool, t, None, d, scale)[3].max()
    for r in range(len(new)):
        want = q4_bounds.by_page(q, pool, t, r, d, scale)
        right = torch.from_numpy(want[0]).bfloat16().double().numpy()
        q4_bounds.check_by_page(right, want, B, d, weight)
        for p in range(right.shape[0]):
            one = tuple(x[p] for x in want)
            for wrong in (-right[p], 0 * right[p], 2 * right[p], right[p - 1]):
                with pytest.raises(AssertionError):
                    q4_bounds.check_by_page(wrong, one, B, d, weight)
