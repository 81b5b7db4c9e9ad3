"""Attention over the 8-bit cache where scores are large: far below zero, far above, and both
sides of it in one row, against the definition in 64 bits (cache_reference).

Keys and queries are constants times powers of two, so that every product and partial sum of a
score is exact in fp32, truncated or not, and the keys of a level have one score, however it is
rounded afterwards: their weights are the same number, and O is a plain mean of values.  What is
left is, for `n` keys and mass = sum w |v|,
    O     2^-8 of itself (bf16), and 2^-11 (weights) + n 2^-22 (sums) of mass
    LSE   2^-21 of 1 + |LSE| (scale log2 e, the product with it, the reference, the logarithm, ln 2:
          each at most 2^-24 of it), and n 2^-23 (the sum)
"""
import numpy as np
import pytest
import torch

import cache_reference as ref
from test_cache_gpu import DEV, FILL, Cache, attend, fa2, i32

pytestmark = pytest.mark.gpu

ROWS = [(1, 1), (8, 1), (3, 5), (20, 1), (2, 75)]   # (group, tokens): both few-row blocks, one and two row tiles


def hold(c, G, Lq, lens, q, **kw):
    o, lse = attend(c, G, Lq, lens, q=q, check=False, **kw)
    args = (c.ks, c.vs, c.table, lens, None, True, None, c.D ** -0.5)
    want, want_lse, _, live = ref.attention(q.double().numpy(), c.k, c.v, *args)
    mass = ref.attention(q.double().numpy(), c.k, c.v & 0x7f, *args)[0]
    assert np.isfinite(want).all() and not np.isnan(live).any()
    o, lse, n = o.double().cpu().numpy(), lse.double().cpu().numpy(), max(lens)
    d = np.abs(lse - want_lse) - (2.0 ** -21 * (1 + np.abs(want_lse)) + n * 2.0 ** -23)
    assert d.max() <= 0, f"lse {d.max():.3e} over its bound"     # (False for NaN)
    d = np.abs(o - want) - (2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * (2.0 ** -11 + n * 2.0 ** -22) * mass)
    assert d.max() <= 0, f"o {d.max():.3e} over its bound"


def level_cache(D, lens, seed):
    c = Cache(len(lens), 1, D, 16, lens, seed=seed, nan_after=False)
    c.vs[:] = 120
    return c


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", ROWS)
@pytest.mark.parametrize("lens,workspace", [([300, 90], False), ([1500, 700], True)])
def test_every_score_far_below_zero(D, G, Lq, lens, workspace):
    """q 96, k -96: one score, -9216 sqrt(D), for every key; in one piece, and in parts that are merged."""
    c = level_cache(D, lens, D + G)
    c.k[:] = 0xfc                    # -384
    c.ks[:] = 125                    # 2^-2
    q = torch.full((2, G, Lq, D), 96.0, dtype=torch.bfloat16)
    hold(c, G, Lq, lens, q, workspace=workspace)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", ROWS)
@pytest.mark.parametrize("log2q,key_byte", [(6, 125), (20, 133), (60, 159)])   # k = 2^6, 2^14, 2^40
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lens,workspace", [([300, 90], False), ([1500, 700], True)])
def test_two_levels_of_large_scores(D, G, Lq, log2q, key_byte, sign, lens, workspace):
    """Pages whose scores are L beside pages at 2 L: the greater take all the weight, wherever they lie."""
    c = level_cache(D, lens, D + G + log2q)
    c.k[:] = 0x78                    # 256
    c.ks[:] = key_byte
    # the least tile, the greatest, and a mixture, at either end of a sequence
    c.ks[c.table[0, :8]] += 1
    c.ks[c.table[1, 4:6]] += 1
    c.ks[c.table[0, 17]] += 1
    q = torch.full((2, G, Lq, D), sign * 2.0 ** log2q, dtype=torch.bfloat16)
    hold(c, G, Lq, lens, q, workspace=workspace)
