"""The paged 8-bit cache and attention over it, from their definitions in 64 bits (numpy,
no code of the package), and the bounds that the kernels' outputs are held to."""
import math

import numpy as np
import torch

MIN_E, MAX_E = -96, 119


def decode(codes):
    """e4m3 bytes -> the numbers they stand for (NaN for 0x7f, 0xff)."""
    c = codes.astype(np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e > 0, (8.0 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    return np.where((c & 0x7f) == 0x7f, np.nan, sign * x)


_CODES = decode(np.arange(128, dtype=np.uint8))   # magnitudes 0 .. 448, then NaN


def encode(x):
    """Numbers -> e4m3 bytes: nearest, ties to the even code, saturating at 448, NaN and infinities NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0)), 448.0)
    hi = np.clip(np.searchsorted(_CODES[:127], a), 1, 126)      # codes order as their magnitudes do
    lo = hi - 1
    d = (a - _CODES[lo]) - (_CODES[hi] - a)                     # exact: both within a step of a
    code = np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, 0x7f).astype(np.uint8)


def scale_value(byte):
    byte = np.asarray(byte).astype(np.int64)
    return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))


def write(x, codes, scale, table, starts, counts):
    """x [B, H, L, D] into codes [N, H, P, D] and scale [N, H] (uint8 arrays, changed in place)."""
    B, H, L, D = x.shape
    N, _, P, _ = codes.shape
    for b in range(B):
        lo = max(0, int(starts[b]))
        hi = min(int(starts[b]) + min(max(int(counts[b]), 0), L), table.shape[1] * P)
        while lo < hi:
            end = min(hi, (lo // P + 1) * P)
            page, slot = int(table[b, lo // P]), lo % P
            if 0 <= page < N:
                for h in range(H):
                    rows = x[b, h, lo - int(starts[b]):end - int(starts[b])].astype(np.float64)
                    finite = np.abs(rows[np.isfinite(rows)])
                    top = finite.max() if finite.size else 0.0
                    e = MIN_E
                    while e < MAX_E and top > 448 * 2.0 ** e:
                        e += 1
                    if slot:
                        before = int(scale[page, h]) - 127
                        if e > before:
                            codes[page, h, :slot] = encode(decode(codes[page, h, :slot]) * 2.0 ** (before - e))
                        e = max(e, before)
                    codes[page, h, slot:slot + end - lo] = encode(rows * 2.0 ** -e)
                    scale[page, h] = e + 127
            lo = end


def gather(codes, scale, table_row, h, n):
    """Positions 0 .. n - 1 of one sequence and head: values [n, D] and whether they have a page [n]."""
    N, _, P, D = codes.shape
    x, there = np.zeros((n, D)), np.zeros(n, dtype=bool)
    for j in range(-(-n // P)):
        page = int(table_row[j]) if j < len(table_row) else -1
        if 0 <= page < N:
            m = min(P, n - j * P)
            x[j * P:j * P + m] = decode(codes[page, h, :m]) * scale_value(scale[page, h])
            there[j * P:j * P + m] = True
    return x, there


def attention(q, kc, vc, ks, vs, table, kv_lens, q_lens, causal, window, scale):
    """(o, lse, o_bound, lse_bound), float64 [B, Hq, Lq, D] and [B, Hq, Lq]; NaN bound: row not written.

    The bounds, per row, from the kernels' arithmetic.  q is two e4m3 terms, whose products
    with codes are exact; a bf16 has no more bits than they, but an element far below its
    row's largest is off by up to half the smallest step of the last term: with that largest
    at least 128 (up to 16 rows a key/value head), and the last term's step 2^-9 / 16, 2^-21
    of it; with the largest at least 224 and a step of 2^-9 (more rows), 2^-17.  A score sums
    2 D products in fp32, each addition off by at most 2^-23 of the partial sum (a bound for
    truncating adders too).  So a score is off by at most ds =
    scale (max_j sum_d |q_d k_jd| 2 D 2^-23 + 2^-21 or 2^-17 max|q| max_j sum_d |k_jd|), plus
    2^-21 (1 + |s|) for the multiplication by the scale, the subtraction of the reference,
    the rounding of log2 e and of 2^x.  Weights are rounded to fp16, 2^-11 of themselves,
    or to three e4m3 terms, 2^-12 (far down in the types' ranges, where they are rounded
    by more, by at most 2^-26 of the largest of 128 keys each).  Sums over n keys add
    n 2^-22.  O is rounded to bf16: 2^-8 of itself.
    """
    B, Hq, Lq, D = q.shape
    H = kc.shape[1]
    o, ob = np.zeros((B, Hq, Lq, D)), np.full((B, Hq, Lq, D), np.nan)
    lse, lb = np.zeros((B, Hq, Lq)), np.full((B, Hq, Lq), np.nan)
    cap = table.shape[1] * kc.shape[2]
    for b in range(B):
        n = min(max(int(kv_lens[b]), 0), cap)
        m = Lq if q_lens is None else min(max(int(q_lens[b]), 0), Lq)
        for hk in range(H):
            k, there = gather(kc, ks, table[b], hk, n)
            v, _ = gather(vc, vs, table[b], hk, n)
            j = np.arange(n)
            for h in range(hk * (Hq // H), (hk + 1) * (Hq // H)):
                for i in range(m):
                    pos = n - m + i
                    see = there.copy()
                    if causal:
                        see &= j <= pos
                        if window is not None:
                            see &= j >= pos - window
                    if not see.any():
                        lse[b, h, i], lb[b, h, i], ob[b, h, i] = -math.inf, 0, 0
                        continue
                    kk, vv, row = k[see], v[see], q[b, h, i].astype(np.float64)
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (kk @ row)
                        top = s.max()
                        w = np.exp(s - top)
                        z = w.sum()
                        w /= z
                        lse[b, h, i] = top + math.log(z)
                        o[b, h, i] = w @ vv
                        reach = scale * (np.abs(kk) @ np.abs(row)).max()
                        small_q = scale * (2.0 ** -21 if Lq * Hq // H <= 16 else 2.0 ** -17) * np.abs(row).max() * np.abs(kk).sum(1).max()
                        ds = reach * 2 * D * 2.0 ** -23 + small_q + 2.0 ** -21 * (1 + np.abs(s).max())
                        lb[b, h, i] = ds + len(s) * 2.0 ** -23 + 2.0 ** -21 * (1 + abs(lse[b, h, i]))
                        rel = 2.0 ** -11 + 2 * ds + len(s) * 2.0 ** -22
                        mass = w @ np.abs(vv)
                        # the weight of the largest of its 128 keys, for every key
                        tile = np.zeros(-(-n // 128))
                        np.maximum.at(tile, j[see] // 128, w)
                        small = 2.0 ** -26 * (tile[j[see] // 128] @ np.ones_like(s)) * np.abs(vv).max()
                        ob[b, h, i] = 2.0 ** -8 * np.abs(o[b, h, i]) + (1 + 2.0 ** -8) * (rel * mass + small)
    return o, lse, ob, lb


def check_attention(o, lse, ref, fill=None):
    """o, lse (CPU tensors) against attention()'s answer; rows it does not write hold `fill`."""
    ro, rl, bo, bl = ref
    o, lse = o.double().numpy(), lse.double().numpy()
    written = ~np.isnan(bl) | np.isnan(rl)
    for got, want, bound, name in ((lse, rl, bl, "lse"), (o, ro, bo, "o")):
        live = written if got.ndim == 3 else np.broadcast_to(written[..., None], got.shape)
        if fill is not None:
            assert np.all(got[~live] == fill), f"{name}: a row that is not the sequence's was written"
        nan = np.isnan(want) & live
        assert np.array_equal(np.isnan(got) & live, nan), f"{name}: NaN in other places"
        ok = live & ~nan
        inf = np.isinf(want) & ok
        assert np.array_equal(got[inf], want[inf]), name
        ok &= ~inf & ~np.isnan(bound)
        over = np.abs(got[ok] - want[ok]) - bound[ok]
        assert not over.size or over.max() <= 0, \
            f"{name}: {over.max():.3e} over its bound, at {np.argwhere(ok)[over.argmax()]}"


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def check_beside_nan(o, lse, q, kc, vc, ks, vs, table, kv_lens, q_lens, causal, window, scale):
    """As check_attention, where values hold NaN: a column of O is no other column's, so those that
    no NaN reaches are held to the answer, and its bound, of the cache with numbers in their places
    (attention()'s own bound takes the largest value of all columns and is NaN there)."""
    rest = (q, kc, vc, ks, vs, table, kv_lens, q_lens, causal, window, scale)
    ro, rl, _, _ = attention(*rest)
    clean = (q, kc, np.where((vc & 0x7f) == 0x7f, 0, vc), ks, np.where(vs == 255, 127, vs), *rest[5:])
    co, cl, bo, bl = attention(*clean)
    o, lse = o.double().numpy(), lse.double().numpy()
    written = ~np.isnan(bl) | np.isnan(cl)
    for got, nan_of, want, bound, name in ((lse, rl, cl, bl, "lse"), (o, ro, co, bo, "o")):
        live = written if got.ndim == 3 else np.broadcast_to(written[..., None], got.shape)
        nan = np.isnan(nan_of) & live
        assert np.array_equal(np.isnan(got) & live, nan), f"{name}: NaN in other places"
        ok = live & ~nan & ~np.isinf(want)
        assert np.isfinite(bound[ok]).all() and np.array_equal(got[live & np.isinf(want)], want[live & np.isinf(want)]), name
        over = np.abs(got[ok] - want[ok]) - bound[ok]
        assert not over.size or over.max() <= 0, \
            f"{name}: {over.max():.3e} over its bound, at {np.argwhere(ok)[over.argmax()]}"
