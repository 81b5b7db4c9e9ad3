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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 16, 20, 200])
@pytest.mark.parametrize("apart", [12, 24, 30, 35, 40])
@pytest.mark.parametrize("workspace", [False, True])
def test_value_scales_far_apart(D, rows, apart, workspace):
    """Some pages' values are 2^apart stronger, but zero in half of the columns, where O is the weaker
    ones' alone.  A weight times its value scale is off by 2^-11 of itself, and by a part of the
    largest such product: 2^-25 of the largest in its tile of 128 keys (up to 16 rows; half a step of
    the last term, 2^-9 / 256 / 2, of weights that end between 2^7 and 2^8), 2^-31 of the row's (more;
    half a step of a small fp16, 2^-25, of weights that end at 2^6 or above)."""
    n, G = 700, rows
    c = Cache(1, 1, D, 16, [n], seed=D + rows + apart, nan_after=False)
    strong = c.table[0, [1, 9, 10, 30]]
    c.v[strong, :, :, ::2] = 0
    c.vs[:] = 110
    c.vs[strong] = 110 + apart
    q = ref.bf16(c.rng.standard_normal((1, G, 1, D)) * 0.5)
    o, lse = attend(c, G, 1, [n], q=q, workspace=workspace, check=False)
    args = (c.ks, c.vs, c.table, [n], None, True, None, D ** -0.5)
    qn = q.double().numpy()
    want, want_lse, _, lse_bound = ref.attention(qn, c.k, c.v, *args)
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= lse_bound).all()
    mass = ref.attention(qn, c.k, c.v & 0x7f, *args)[0]
    k, _ = ref.gather(c.k, c.ks, c.table[0], 0, n)
    codes, _ = ref.gather(c.v & 0x7f, np.full_like(c.vs, 127), c.table[0], 0, n)
    scale = np.repeat(ref.scale_value(c.vs[c.table[0], 0]), 16)[:n]
    tile = np.arange(n) // 128
    for r in range(rows):
        s = k @ qn[0, r, 0] * D ** -0.5
        w = np.exp(s - want_lse[0, r, 0])
        # scores' error, as cache_reference.attention derives it
        ds = (np.abs(k) @ np.abs(qn[0, r, 0])).max() * D ** -0.5 * 2 * D * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(s).max()) + \
            D ** -0.5 * (2.0 ** -21 if rows <= 16 else 2.0 ** -17) * np.abs(qn[0, r, 0]).max() * np.abs(k).sum(1).max()
        if rows <= 16:
            top = np.zeros(tile[-1] + 1)
            np.maximum.at(top, tile, w * scale)
            small = 2.0 ** -25 * top[tile] @ codes
        else:
            small = 2.0 ** -31 * (w * scale).max() * codes.sum(0)
        bound = 2.0 ** -8 * np.abs(want[0, r, 0]) + (1 + 2.0 ** -8) * ((2.0 ** -11 + 2 * ds + n * 2.0 ** -22) * mass[0, r, 0] + small)
        over = np.abs(o[0, r, 0].double().cpu().numpy() - want[0, r, 0]) - bound
        assert over.max() <= 0, f"row {r}: {over.max():.3e} over its bound"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", ROWS)
@pytest.mark.parametrize("log2", [8, 18, 24, 30, 40, 90])
@pytest.mark.parametrize("lens,workspace", [([300, 90], False), ([1500, 700], True)])
def test_large_scores_of_any_bits(D, G, Lq, log2, lens, workspace):
    """Scores of all 24 bits, some 2^log2 large: the greatest one's value is the answer wherever the
    next is further below than the scores' own error (2 D additions' and q's terms', as
    cache_reference.attention derives it) and what a weight can still show."""
    c = Cache(len(lens), 1, D, 16, lens, seed=D + G + log2, nan_after=False)
    c.ks[:] = 120
    q = ref.bf16(c.rng.standard_normal((2, G, Lq, D)) * 2.0 ** log2)
    o, lse = attend(c, G, Lq, lens, q=q, workspace=workspace, check=False)
    o, lse, qn, seen = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy(), 0
    for b, n in enumerate(lens):
        k, _ = ref.gather(c.k, c.ks, c.table[b], 0, n)
        v, _ = ref.gather(c.v, c.vs, c.table[b], 0, n)
        for g in range(G):
            for i in range(Lq):
                row, m = qn[b, g, i], n - Lq + i + 1
                s = k[:m] @ row * D ** -0.5
                first, second = s.argmax(), np.partition(s, -2)[-2]
                reach = (np.abs(k[:m]) @ np.abs(row)).max() * D ** -0.5
                ds = reach * 2 * D * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(s).max()) + \
                    D ** -0.5 * 2.0 ** (-21 if G * Lq <= 16 else -17) * np.abs(row).max() * np.abs(k[:m]).sum(1).max()
                if s[first] - second < 2 * ds + 40:      # e^-40: nothing of the next one's value
                    continue
                seen += 1
                assert abs(lse[b, g, i] - s[first]) <= ds + 2.0 ** -21 * (1 + abs(s[first]))
                # (a weight is off by 2^-11, O by 2^-8 of itself)
                d = np.abs(o[b, g, i] - v[first]) - (2.0 ** -8 + 2.0 ** -10) * np.abs(v[first])
                assert d.max() <= 2.0 ** -30, f"sequence {b}, head {g}, row {i}: {d.max():.3e} over its bound"
    assert seen >= 0.6 * len(lens) * G * Lq or log2 < 18   # (where the next is often too near)
