"""Attention over the paged 16-bit cache in 64 bits, with bounds as narrow as include/fa2_paged.h promises
for the weights of each form, and the same sums with weights rounded as a kernel may round them, so that
a test on the CPU can show what a bound lets through.

(paged_reference's bounds take one term for all but 16 rows, and 2^-24 of the largest value a key for small
fp16 weights, where the header says 32 rows and 2^-31.)"""
import math

import torch

from paged_reference import HALF, TINY


def two_terms(D, rows, dtype):
    """Whether a weight goes into the product with V as two terms: `rows` query rows a key/value head."""
    return rows <= (16 if D == 256 else 32) or (D == 256 and dtype == torch.bfloat16)


def _heads(q, c, kv_lens, q_lens, causal, scale):
    """For each sequence and query head with rows: b, h, m, scores [m, n] in 64 bits (-inf where not seen), the
    sums of their terms' magnitudes, values.  All that is seen is finite and has a page."""
    B, Hq, Lq, D = q.shape
    for b in range(B):
        n = int(kv_lens[b])
        m = Lq if q_lens is None else int(q_lens[b])
        if m == 0:
            continue
        see = torch.arange(n)[None] <= (n - m + torch.arange(m) if causal else torch.full((m,), n))[:, None]
        for h in range(Hq):
            k, v, there = c.gather(b, h // (Hq // c.H), n)
            assert bool(there.all()) and bool(see.any(1).all())
            x = q[b, h, :m].double()
            yield b, h, m, torch.where(see, (x @ k.T) * scale, -math.inf), scale * (x.abs() @ k.abs().T) * see, v


def attention(q, c, kv_lens, q_lens=None, causal=True, scale=1.0, terms=None):
    """O, LSE and how far each may be off, as paged_reference.attention has them (whose terms for scores,
    exponents, sums and O's rounding these are), but narrower for weights: two terms are off by half a step of half a
    step; one by half a step of |v| + |O|; either by half a step of the type's least number, 2^-25 for fp16,
    beside weights of which the row's largest is at least 2^6, so 2^-31 of it.  bf16 weights end at 2^-126
    where the largest is at least 2^-12: 2^-114 of it.  Products and sums keep 2^-149 and what it makes
    beside those 2^-12, 2^-137: for every key, and twice for every part put together."""
    B, Hq, Lq, D = q.shape
    if terms is None:
        terms = 2 if two_terms(D, Lq * (Hq // c.H), q.dtype) else 1
    half, tiny = HALF[q.dtype], TINY[q.dtype]
    o, ob = torch.zeros(B, Hq, Lq, D, dtype=torch.float64), torch.full((B, Hq, Lq, D), math.nan, dtype=torch.float64)
    lse, lb = torch.zeros(B, Hq, Lq, dtype=torch.float64), torch.full((B, Hq, Lq), math.nan, dtype=torch.float64)
    for b, h, m, s, size, v in _heads(q, c, kv_lens, q_lens, causal, scale):
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - top)
        z, n = w.sum(1, keepdim=True), (s > -math.inf).sum(1, keepdim=True).double()
        w = w / z
        o[b, h, :m], lse[b, h, :m] = w @ v, (top + torch.log(z))[:, 0]
        out, mass = o[b, h, :m].abs(), w @ v.abs()
        # (a sum's zeros add nothing to what it is off by; a score counts by its key's weight)
        ds = size * 2 * (q[b, h, :m] != 0).sum(1, keepdim=True) * 2.0 ** -24
        ds = w * (ds + 2.0 ** -21 * (1 + torch.where(s > -math.inf, top - s, 0.0)))
        lb[b, h, :m] = ds.sum(1) + n[:, 0] * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[b, h, :m].abs())
        off = ds @ v.abs() + ds.sum(1, keepdim=True) * out + (n * 2.0 ** -23 + 2.0 ** -20) * mass
        off = off + (2 * half * half * mass if terms == 2 else half * (mass + out))
        least = 2.0 ** -31 if q.dtype == torch.float16 else 2.0 ** -114
        off = off + n / z * least * v.abs().amax(0, keepdim=True) + (n + 600) * 2.0 ** -137
        ob[b, h, :m] = half * out + tiny + (1 + half) * off
    return o, lse, ob, lb


def rounded(q, c, kv_lens, q_lens=None, causal=True, scale=1.0, terms=1, lift=0.0):
    """O and LSE in 64 bits but for the weights, which are 2^lift beside the row's largest score and rounded to
    `terms` terms of the type, and O.  bf16 with one term is divided by the rounded weights' sum."""
    B, Hq, Lq, D = q.shape
    o, lse = torch.zeros(q.shape, dtype=q.dtype), torch.zeros(B, Hq, Lq)
    for b, h, m, s, _, v in _heads(q, c, kv_lens, q_lens, causal, scale):
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - top) * 2.0 ** lift
        z = w.sum(1, keepdim=True)
        p = w.to(q.dtype).double()
        if terms == 2:
            p = p + (w - p).to(q.dtype).double()
        by = p.sum(1, keepdim=True) if terms == 1 and q.dtype == torch.bfloat16 else z
        o[b, h, :m] = ((p @ v) / by).to(q.dtype)
        lse[b, h, :m] = (top + torch.log(z) - lift * math.log(2))[:, 0]
    return o, lse


# ------------------------------------------------------------------- inputs that show it

def dominant(c, q, seed):
    """Keys and queries for scores of 0 at every sequence's first key and -20 to -28 at the others, in steps of
    an eighth, in units of scale = ln 2 (so weights of 2^-20 to 2^-28 of the largest), with large positive values
    beside the first key's: small weights carry most of O."""
    g = torch.Generator().manual_seed(seed)
    c.k.zero_()
    c.k[..., 0] = -(20 + torch.randint(0, 65, c.k.shape[:-1], generator=g) / 8).to(c.dtype)
    c.v.copy_(((0.5 + torch.rand(c.v.shape, generator=g) / 2) * 2.0 ** 15).to(c.dtype))
    for b in range(c.B):
        c.k[c.table[b, 0], :, 0, 0] = 0
        c.v[c.table[b, 0], :, 0] = 1
    q.zero_()
    q[..., 0] = 1
    return math.log(2)


def few_alike(c, q, seed):
    """Two or three keys of each sequence (the first ones, which every row sees) stand out with similar
    scores, all others far below; values of about 2: what a weight's rounding does to O is largest there."""
    g = torch.Generator().manual_seed(seed)
    c.k.zero_()
    c.k[..., 0] = -16
    for b in range(c.B):
        c.k[c.table[b, 0], :, :3, :2] = torch.randn(c.H, 3, 2, generator=g).to(c.dtype)
    c.v.copy_((torch.randn(c.v.shape, generator=g).sign() * (1.5 + torch.rand(c.v.shape, generator=g))).to(c.dtype))
    q.zero_()
    q[..., 0] = 1
    q[..., 1] = torch.randn(q.shape[:-1], generator=g).to(q.dtype)
    return 1.0
