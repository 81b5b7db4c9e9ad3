"""The 8-bit cache on the GPU against its definition in 64 bits (cache_reference): writing
and reading must give the very codes, scales and values; attention is held to the bounds
that cache_reference.attention derives."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FILL = -7.0   # what rows that a call must not write hold


def fa2():
    import io_aware_exact_fa2_gb300
    return io_aware_exact_fa2_gb300


class Cache:
    """A pool with random codes, scales of different strength and a page table over it, on both sides."""

    def __init__(self, B, H, D, page, lens, seed, spare=2, slot_major=False, nan_after=True):
        self.rng = np.random.default_rng(seed)
        self.B, self.H, self.D, self.page = B, H, D, page
        need = [-(-int(n) // page) for n in lens]
        self.M = max(1, max(need))
        N = sum(need) + spare
        self.N = N
        self.table = np.full((B, self.M), -1)
        order = self.rng.permutation(N)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.k, self.v = (ref.encode(self.rng.standard_normal((N, H, page, D)) * 90) for _ in range(2))
        if nan_after:   # what lies behind a sequence's end must not matter
            for b in range(B):
                n = int(lens[b])
                if n % page:
                    for c in (self.k, self.v):
                        c[self.table[b, n // page], :, n % page:] = 0x7f
        self.ks, self.vs = (self.rng.integers(118, 123, (N, H)).astype(np.uint8) for _ in range(2))
        self.slot_major = slot_major

    def device(self):
        out = []
        for c in (self.k, self.v):
            t = torch.from_numpy(c).to(DEV)
            if self.slot_major:
                t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            out.append(t.view(torch.float8_e4m3fn))
        out += [torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu) for s in (self.ks, self.vs)]
        return (*out, torch.from_numpy(self.table.astype(np.int32)).to(DEV))


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=DEV)


def same(got, want):
    np.testing.assert_array_equal(got.view(torch.uint8).cpu().numpy(), want)


# -------------------------------------------------------------- write and read

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("L", [1, 2, 7, 40, 300])
@pytest.mark.parametrize("slot_major", [False, True])
def test_write_then_read(D, page, L, slot_major):
    B, H = 3, 2
    starts = [0, page - 1, 2 * page + 5]
    counts = [L, max(0, L - 3), L]
    c = Cache(B, H, D, page, [s + n for s, n in zip(starts, counts)], seed=D + page + L, slot_major=slot_major,
              nan_after=False)
    strength = 2.0 ** c.rng.integers(-9, 9, (B, H, L, 1))
    x = [ref.bf16(c.rng.standard_normal((B, H, L, D)) * strength) for _ in range(2)]
    dev = c.device()
    # the rows as a projection leaves them: [B, L, H, D]
    kd, vd = (t.to(DEV).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in x)
    fa2().fa2_cache_write(kd, vd, *dev, i32(starts), i32(counts))
    for t, codes, scale in zip(x, (c.k, c.v), (c.ks, c.vs)):
        ref.write(t.double().numpy(), codes, scale, c.table, starts, counts)
    for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        same(got, want)
    # everything back, a position more than there is for the first
    n = max(s + m for s, m in zip(starts, counts))
    out = [torch.full((B, n, H, D), FILL, dtype=torch.bfloat16, device=DEV).permute(0, 2, 1, 3) for _ in range(2)]
    ends = [s + m for s, m in zip(starts, counts)]
    fa2().fa2_cache_read(*dev, *out, i32([0] * B), i32(ends))
    for got, codes, scale in zip(out, (c.k, c.v), (c.ks, c.vs)):
        for b in range(B):
            for h in range(H):
                want, _ = ref.gather(codes, scale, c.table[b], h, ends[b])
                np.testing.assert_array_equal(got[b, h, :ends[b]].double().cpu().numpy(), want)
                assert torch.all(got[b, h, ends[b]:] == FILL)


def test_write_of_special_values():
    """Zeros, infinities, NaN, the largest and smallest bf16; alone in a page and beside others."""
    rows = np.zeros((1, 1, 6, 64), np.float32)
    rows[0, 0, 1, 3] = np.inf
    rows[0, 0, 1, 4] = 2.5
    rows[0, 0, 2, 5] = np.nan
    rows[0, 0, 3, :8] = [3.3e38, -3.3e38, 1e-38, -1e-38, 1e-40, -0.0, 448, 449]
    rows[0, 0, 4, :3] = [1.0, -np.inf, 2.0 ** -133]
    rows[0, 0, 5, :4] = [3.3895e38, 2.0 ** -20, 7.0, -7.25]
    x = ref.bf16(rows)
    for first, last in [(0, 6), (0, 1), (1, 2), (2, 3), (3, 4), (4, 5), (5, 6)]:
        c = Cache(1, 1, 64, 16, [16], seed=1)
        part = x[:, :, first:last]
        dev = c.device()
        fa2().fa2_cache_write(part.to(DEV).contiguous(), part.to(DEV).contiguous(), *dev, i32([0]))
        for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
            ref.write(part.double().numpy(), codes, scale, c.table, [0], [last - first])
        for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
            same(got, want)


def test_growing_page_rescales_and_other_slots_stay():
    """Tokens one by one, each call stronger or weaker than the last: scales only grow within a page."""
    c = Cache(2, 3, 128, 16, [40, 40], seed=5, nan_after=False)
    dev = c.device()
    for i in range(37):
        x = ref.bf16(c.rng.standard_normal((2, 3, 1, 128)) * 2.0 ** c.rng.integers(-30, 30))
        fa2().fa2_cache_write(x.to(DEV), x.to(DEV), *dev, i32([i, 36 - i]))
        for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
            ref.write(x.double().numpy(), codes, scale, c.table, [i, 36 - i], [1, 1])
    for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        same(got, want)


def test_positions_without_a_page():
    """Entries outside the pool, positions past the table, negative starts, counts past L: dropped, read as zeros."""
    c = Cache(4, 2, 64, 16, [64] * 4, seed=6, nan_after=False)
    c.table[0, 1] = -1
    c.table[1, 2] = c.N
    c.table[1, 0] = 2 ** 31 - 1
    c.table[2, 3] = -2 ** 31
    starts, counts = [5, 0, 40, -6], [50, 64, 2 ** 31 - 1, 20]
    x = ref.bf16(c.rng.standard_normal((4, 2, 64, 64)))
    dev = c.device()
    fa2().fa2_cache_write(x.to(DEV), x.to(DEV), *dev, i32(starts), i32(counts))
    for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
        ref.write(x.double().numpy(), codes, scale, c.table, starts, counts)
    for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        same(got, want)
    out = [torch.full((4, 2, 70, 64), FILL, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa2().fa2_cache_read(*dev, *out, i32([0, 3, 2 ** 31 - 1, -6]), i32([70, 66, 4, -1]))
    got = out[0].double().cpu().numpy()
    for h in range(2):
        want, _ = ref.gather(c.k, c.ks, c.table[0], h, 70)
        np.testing.assert_array_equal(got[0, h], want)
        want, _ = ref.gather(c.k, c.ks, c.table[1], h, 69)
        np.testing.assert_array_equal(got[1, h, :66], want[3:])
    assert np.all(got[1, :, 66:] == FILL) and np.all(got[2, :, :4] == 0) and np.all(got[2, :, 4:] == FILL)
    assert np.all(got[3] == FILL)


def test_empty_calls():
    c = Cache(2, 1, 64, 16, [20, 20], seed=7)
    dev = c.device()
    x = torch.zeros(2, 1, 0, 64, dtype=torch.bfloat16, device=DEV)
    fa2().fa2_cache_write(x, x, *dev, i32([0, 0]))
    fa2().fa2_cache_read(*dev, x, x, i32([0, 0]))
    fa2().fa2_cache_attn(x, *dev, i32([20, 20]), x, torch.zeros(2, 1, 0, device=DEV))
    x = torch.ones(2, 1, 3, 64, dtype=torch.bfloat16, device=DEV)
    fa2().fa2_cache_write(x, x, *dev, i32([4, 19]), i32([0, -5]))
    for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        same(got, want)


# ------------------------------------------------------------------- attention

def attend(c, G, Lq, kv_lens, q_lens=None, causal=True, window=None, workspace=True, q=None, strided=False, dev=None,
           check=True, scale=None, repeat=1):
    B, H, D = c.B, c.H, c.D
    q = ref.bf16(c.rng.standard_normal((B, H * G, Lq, D)) * 0.7) if q is None else q
    dev = c.device() if dev is None else dev
    qd = q.to(DEV)
    if strided:   # [B, L, H, D] storage
        qd = qd.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        o = torch.full((B, Lq, H * G, D + 8), FILL, dtype=torch.bfloat16, device=DEV)[..., :D].permute(0, 2, 1, 3)
    else:
        o = torch.full((B, H * G, Lq, D), FILL, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H * G, Lq), FILL, device=DEV)
    ws = fa2().fa2_cache_attn_workspace(qd, dev[0]) if workspace else None
    scale = D ** -0.5 if scale is None else scale
    for _ in range(repeat):
        fa2().fa2_cache_attn(qd, *dev, i32(kv_lens), o, lse, causal=causal, q_lens=None if q_lens is None else i32(q_lens),
                             window=window, scale=scale, workspace=ws)
    status, code = fa2().fa2_cache_get_device_error()
    assert status == 0, f"device error {code:#x}"
    if ws is not None:   # left ready for the next call
        assert not ws[:1024].any()
    if check:
        want = ref.attention(q.double().numpy(), c.k, c.v, c.ks, c.vs, c.table, kv_lens, q_lens, causal, window, scale)
        ref.check_attention(o.cpu(), lse.cpu(), want, FILL)
    return o, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Lq", [(1, 1), (4, 1), (8, 1), (5, 3), (16, 1), (3, 6), (8, 4)])
@pytest.mark.parametrize("workspace", [False, True])
def test_attention(D, page, G, Lq, workspace):
    lens = [1, 700, 129, 64, 33]
    c = Cache(5, 2, D, page, lens, seed=D + page + G)
    attend(c, G, Lq, lens, workspace=workspace, strided=G == 5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq,G", [(9, 4), (40, 1), (33, 5), (130, 2), (64, 8)])
def test_attention_of_many_rows(D, Lq, G):
    lens = [300, 131, 64]
    c = Cache(3, 2, D, 32, lens, seed=D + Lq)
    attend(c, G, Lq, lens, [Lq, 1, min(Lq, 50)], strided=True)
    attend(c, G, Lq, lens, [min(Lq, 7), Lq, 0])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_from_nothing(D):
    """No keys, one key, fewer keys than queries (rows before the first key see nothing), no queries."""
    lens = [0, 1, 3, 16, 17, 50]
    c = Cache(6, 1, D, 16, lens, seed=D)
    attend(c, 2, 5, lens, [5, 5, 5, 0, 1, 4])
    attend(c, 2, 5, lens, [5, 5, 5, 0, 1, 4], causal=False)
    attend(c, 4, 1, lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 15, 16, 100, 5000])
def test_window(D, window):
    lens = [40, 333, 1, 160]
    c = Cache(4, 2, D, 16, lens, seed=D + window)
    attend(c, 4, 1, lens, window=window)
    attend(c, 3, 21, lens, [21, 13, 21, 2], window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 4, 70])
def test_all_keys_visible(D, Lq):
    lens = [90, 17, 200]
    c = Cache(3, 2, D, 64, lens, seed=D)
    attend(c, 2, Lq, lens, [Lq, min(Lq, 3), Lq], causal=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 5, 80])
def test_missing_pages_are_not_seen(D, Lq):
    lens = [200, 100, 48, 100]
    c = Cache(4, 2, D, 16, lens, seed=D + 1)
    c.table[0, 3:9] = -1
    c.table[1, 0] = c.N
    c.table[2, :] = -5
    c.table[3, 6] = 2 ** 31 - 1      # the newest tokens' own page
    attend(c, 4, Lq, lens)
    # lengths outside the table's reach are taken as the nearest inside
    c.k[(c.k & 0x7f) == 0x7f] = 0
    c.v[(c.v & 0x7f) == 0x7f] = 0
    attend(c, 4, Lq, [2 ** 31 - 1, -3, 48, 13 * 16 + 5])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 6, 90])
def test_nan_and_infinity_reach_only_rows_that_see_them(D, Lq):
    """NaN codes and NaN scales in keys and values; rows behind them are NaN, earlier ones untouched."""
    lens = [120, 120, 120, 120, 120]
    c = Cache(5, 1, D, 16, lens, seed=D + 2)
    pos = 117
    page, slot = c.table[:, pos // 16], pos % 16
    c.k[page[0], 0, slot, 5] = 0x7f
    c.v[page[1], 0, slot, 9] = 0xff
    c.v[page[1], 0, slot - 1, D - 1] = 0x7f
    c.ks[c.table[2, 7], 0] = 255
    c.vs[c.table[4, 7], 0] = 255
    q = ref.bf16(c.rng.standard_normal((5, 3, Lq, D)))
    q[3, 1, 0, 2] = float("inf")
    q[3, 2, Lq - 1, 0] = float("nan")
    attend(c, 3, Lq, lens, q=q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 64])
def test_pages_of_very_different_strength(D, Lq):
    """Value scales far apart, a dominating first key, queries of any magnitude, all-zero pages at the least scale."""
    lens = [1000, 900]
    c = Cache(2, 2, D, 16, lens, seed=D + 3)
    c.vs[:] = c.rng.integers(118 - 12, 118 + 6, c.vs.shape)
    zero = c.table[0, 20:30]
    c.v[zero] = 0
    c.vs[zero] = 127 - 96
    c.ks[:, 1] -= 3
    q = c.rng.standard_normal((2, 4, Lq, D)) * 2.0 ** c.rng.integers(-3, 1, (2, 4, Lq, 1))
    q[0, 3] = 0
    c.k[c.table[0, 0], :, 0] &= 0x7f
    q[0, 0] = np.abs(q[0, 0]) * 3        # a sink
    attend(c, 2, Lq, lens, q=ref.bf16(q))
    attend(c, 2, Lq, lens, q=ref.bf16(q * 2.0 ** -60), scale=1.0)
    attend(c, 2, Lq, lens, q=ref.bf16(q * 2.0 ** 60), scale=2.0 ** -62)


def test_long_context_is_shared_out_and_merged():
    """One sequence's keys over all SMs, again and again with one workspace: the same bits each time."""
    lens = [20011, 5]
    c = Cache(2, 1, 128, 64, lens, seed=9)
    q = ref.bf16(c.rng.standard_normal((2, 8, 1, 128)))
    o, lse = attend(c, 8, 1, lens, q=q)
    again = attend(c, 8, 1, lens, q=q, check=False, repeat=5)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    attend(c, 8, 1, lens, q=q, workspace=False)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_of_a_long_context(D):
    """Blocks of rows cut over many CTAs and merged; the same bits each time, and without a workspace."""
    lens = [2500, 700]
    c = Cache(2, 1, D, 32, lens, seed=D + 4)
    q = ref.bf16(c.rng.standard_normal((2, 2, 90, D)))
    o, lse = attend(c, 2, 90, lens, [90, 71], q=q)
    again = attend(c, 2, 90, lens, [90, 71], q=q, check=False, repeat=5)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    attend(c, 2, 90, lens, [90, 71], q=q, workspace=False)


def test_many_sequences():
    """More sequences than threads of a block, most of them short or empty."""
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 40, 700)
    c = Cache(700, 1, 64, 16, lens, seed=10)
    attend(c, 2, 2, lens, rng.integers(0, 3, 700))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, pages strided apart; positions in its last pages."""
    N, H, page, D = 40, 2, 64, 128
    stride = 128 << 20
    raw = torch.zeros(stride * (N - 1) + H * page * D, dtype=torch.uint8, device=DEV)
    kc = torch.as_strided(raw, (N, H, page, D), (stride, page * D, D, 1))
    c = Cache(1, H, D, page, [300], seed=11, spare=N - 5)
    assert c.N == N
    c.table[0, :5] = [39, 0, 38, 20, 37]
    c.k[(c.k & 0x7f) == 0x7f] = 0
    c.v[(c.v & 0x7f) == 0x7f] = 0
    kc.copy_(torch.from_numpy(c.k).to(DEV))
    dev = list(c.device())
    dev[0] = kc.view(torch.float8_e4m3fn)
    attend(c, 4, 2, [300], dev=tuple(dev))
    x = ref.bf16(c.rng.standard_normal((1, H, 300, D)))
    fa2().fa2_cache_write(x.to(DEV), x.to(DEV), *dev, i32([0]))
    for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
        ref.write(x.double().numpy(), codes, scale, c.table, [0], [300])
    attend(c, 4, 2, [300], dev=tuple(dev))
    out = [torch.zeros(1, H, 300, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa2().fa2_cache_read(*dev, *out, i32([0]))
    for h in range(H):
        np.testing.assert_array_equal(out[0][0, h].double().cpu().numpy(), ref.gather(c.k, c.ks, c.table[0], h, 300)[0])


def test_shared_prefix_pages():
    """Two sequences whose tables name the same first pages, and one page twice in one table."""
    lens = [100, 80, 60]
    c = Cache(3, 2, 128, 16, lens, seed=12, nan_after=False)
    c.table[1, :4] = c.table[0, :4]
    c.table[2, 1] = c.table[2, 0]
    attend(c, 4, 3, lens)


# ----------------------------------------------- as a server uses them together

@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (256, 1)])
def test_a_conversation(D, G):
    """A ragged batch of prompts is written and attended to (a chunk at a time), then tokens one by one,
    then drafted ones; everything against the reference after each step.  What is read back goes
    through the dense forward pass and gives the same attention."""
    B, H, page, Lmax = 3, 2, 16, 60
    final = [150, 90, 100]
    c = Cache(B, H, D, page, final, seed=13, nan_after=False)
    dev = c.device()
    held = np.zeros(B, int)

    def step(counts, L):
        nonlocal held
        x = [ref.bf16(c.rng.standard_normal((B, H, L, D)) * 2.0 ** c.rng.integers(-2, 2)) for _ in range(2)]
        fa2().fa2_cache_write(x[0].to(DEV), x[1].to(DEV), *dev, i32(held), i32(counts))
        for t, codes, scale in zip(x, (c.k, c.v), (c.ks, c.vs)):
            ref.write(t.double().numpy(), codes, scale, c.table, held, counts)
        held = held + np.array(counts)
        attend(c, G, L, held, counts, dev=dev)
        for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
            same(got, want)

    step([60, 33, 1], Lmax)
    step([60, 20, 57], Lmax)
    for _ in range(4):
        step([1, 1, 1], 1)
    step([5, 2, 4], 5)
    n = int(held[0])
    k, v = (torch.empty(1, H, n, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    row = dev[4][:1].contiguous()
    fa2().fa2_cache_read(*dev[:4], row, k, v, i32([0]))
    q = ref.bf16(c.rng.standard_normal((1, H, n, D))).to(DEV)
    o, lse = torch.empty_like(q), torch.empty(1, H, n, device=DEV)
    fa2().fa2_fwd(q, k, v, o, lse, causal=True)
    o2, lse2 = torch.empty_like(q), torch.empty(1, H, n, device=DEV)
    fa2().fa2_cache_attn(q, *dev[:4], row, i32([n]), o2, lse2)
    # two kernels' weights, rounded to bf16 and to fp16 (2^-8 and 2^-11 of sum w |v| <= max |v|), and two
    # roundings of O (2^-8 of it each)
    assert (lse - lse2).abs().max() <= 1e-3
    assert (o.float() - o2.float()).abs().max() <= (3 * 2.0 ** -8 + 2.0 ** -10) * float(v.float().abs().max())


def test_captured_and_replayed_with_other_lengths():
    """A step captured once: later replays see new lengths, tokens and pages in the same buffers."""
    B, H, D, page, G = 2, 2, 128, 16, 4
    c = Cache(B, H, D, page, [200, 200], seed=14, nan_after=False)
    dev = c.device()
    k, v = (torch.zeros(B, H, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros(B, H * G, 1, D, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(B, H * G, 1, device=DEV)
    starts, lens = i32([0, 0]), i32([1, 1])
    ws = fa2().fa2_cache_attn_workspace(q, dev[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa2().fa2_cache_write(k, v, *dev, starts)
        fa2().fa2_cache_attn(q, *dev, lens, o, lse, workspace=ws)
    for held in ([0, 150], [1, 151], [40, 7], [198, 0]):
        x = [ref.bf16(c.rng.standard_normal((B, H, 1, D))) for _ in range(2)]
        qn = ref.bf16(c.rng.standard_normal((B, H * G, 1, D)))
        k.copy_(x[0]), v.copy_(x[1]), q.copy_(qn)
        starts.copy_(i32(held)), lens.copy_(i32([h + 1 for h in held]))
        graph.replay()
        torch.cuda.synchronize()
        for t, codes, scale in zip(x, (c.k, c.v), (c.ks, c.vs)):
            ref.write(t.double().numpy(), codes, scale, c.table, held, [1, 1])
        want = ref.attention(qn.double().numpy(), c.k, c.v, c.ks, c.vs, c.table, [h + 1 for h in held], None, True, None,
                             D ** -0.5)
        ref.check_attention(o.cpu(), lse.cpu(), want)


def test_on_another_stream():
    """Work handed to a stream that is not the current one runs there, after what is queued on it."""
    c = Cache(2, 2, 64, 16, [80, 50], seed=15, nan_after=False)
    dev = c.device()
    x = ref.bf16(c.rng.standard_normal((2, 2, 30, 64)))
    q = ref.bf16(c.rng.standard_normal((2, 4, 1, 64)))
    xd, qd = torch.zeros_like(x, device=DEV), q.to(DEV)
    o, lse = torch.zeros_like(qd), torch.zeros(2, 4, 1, device=DEV)
    starts, lens = i32([50, 20]), i32([80, 50])
    side = torch.cuda.Stream(DEV)
    big = torch.zeros(64 << 20, device=DEV)
    later = x.to(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big.add_(1.0)
        xd.copy_(later)      # the rows are there only after the additions
    fa2().fa2_cache_write(xd, xd, *dev, starts, stream=side)
    fa2().fa2_cache_attn(qd, *dev, lens, o, lse, stream=side)
    side.synchronize()
    for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
        ref.write(x.double().numpy(), codes, scale, c.table, [50, 20], [30, 30])
    want = ref.attention(q.double().numpy(), c.k, c.v, c.ks, c.vs, c.table, [80, 50], None, True, None, 64 ** -0.5)
    ref.check_attention(o.cpu(), lse.cpu(), want)


def test_more_work_than_can_be_counted_is_refused():
    """A table for 2^30 positions and 2^15 query rows: 2^31 tiles and more."""
    c = Cache(1, 1, 64, 16, [40], seed=17)
    dev = list(c.device())
    dev[4] = torch.full((1, 1 << 26), -1, dtype=torch.int32, device=DEV)
    q = torch.zeros(1, 1, 1 << 15, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(1, 1, 1 << 15, device=DEV)
    with pytest.raises(RuntimeError, match="FA2_ERR_UNSUPPORTED"):
        fa2().fa2_cache_attn(q, *dev, i32([40]), o, lse)
    # the same table with a row: every page is missing
    q = q[:, :, :1].contiguous()
    fa2().fa2_cache_attn(q, *dev, i32([1 << 30]), o[:, :, :1].contiguous(), lse[:, :, :1].contiguous(),
                         workspace=fa2().fa2_cache_attn_workspace(q, dev[0]))
    assert fa2().fa2_cache_get_device_error() == (0, 0)


def test_a_small_workspace_is_refused():
    c = Cache(1, 1, 64, 16, [40], seed=16)
    dev = c.device()
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(1, 1, 1, device=DEV)
    ws = fa2().fa2_cache_attn_workspace(q, dev[0])
    with pytest.raises(RuntimeError, match="FA2_ERR_INVALID_ARG"):
        fa2().fa2_cache_attn(q, *dev, i32([40]), o, lse, workspace=ws[:-256])
    with pytest.raises(ValueError):
        fa2().fa2_cache_attn(q, *dev, i32([40]), o, lse, workspace=ws.cpu())
    with pytest.raises(ValueError):
        fa2().fa2_cache_attn(q, *dev, i32([40, 4]), o, lse)
    with pytest.raises(ValueError):
        fa2().fa2_cache_attn(q, *dev, torch.tensor([40]), o, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [None, 0, 37, 130])
def test_blocks_of_rows_over_pages_and_windows(D, page, window):
    """17 rows and more: row tiles that end, begin and miss a block; strided pools and rows."""
    lens = [290, 129, 77]
    c = Cache(3, 2, D, page, lens, seed=D + page, slot_major=page != 64)
    attend(c, 4, 66, lens, [66, 33, 5], window=window, strided=page == 16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(1, 16), (1, 17), (17, 1), (1, 127), (2, 64), (1, 129), (8, 32), (1, 257), (3, 129)])
def test_block_boundaries(D, G, Lq):
    """Rows at the sizes where blocks and their halves fill up, over one tile of keys and more."""
    lens = [Lq, Lq + 140]
    c = Cache(2, 1, D, 16, lens, seed=D + Lq)
    attend(c, G, Lq, lens)


def test_one_workspace_for_calls_of_every_kind():
    """Calls of different head dimensions and row counts take one workspace in turn: what one leaves in it
    must not look like another's state."""
    kinds = []
    for D, G, Lq, lens in [(64, 8, 1, [3000, 40]), (128, 4, 40, [1500, 300]), (64, 4, 90, [1200, 800]), (256, 1, 60, [900, 70]),
                           (128, 16, 1, [2500, 2500]), (256, 8, 1, [1800, 10]), (64, 16, 1, [2222, 1111])]:
        c = Cache(2, 1, D, 16, lens, seed=D + Lq)
        q = ref.bf16(c.rng.standard_normal((2, G, Lq, D)))
        dev, qd, kv = c.device(), q.to(DEV), i32(lens)
        o, lse = attend(c, G, Lq, lens, q=q, dev=dev)
        kinds.append((dev, qd, kv, o, lse, fa2().fa2_cache_attn_workspace(qd, dev[0]).numel()))
    ws = torch.zeros(max(k[-1] for k in kinds), dtype=torch.uint8, device=DEV)
    order = np.random.default_rng(18).permutation(np.repeat(np.arange(len(kinds)), 6))
    for i in order:
        dev, qd, kv, o, lse, _ = kinds[i]
        o2, lse2 = torch.full_like(o, FILL), torch.full_like(lse, FILL)
        fa2().fa2_cache_attn(qd, *dev, kv, o2, lse2, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa2().fa2_cache_get_device_error() == (0, 0)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace, give the bits that each gives alone."""
    calls = []
    for G, Lq, D in [(8, 1, 64), (4, 60, 128)]:
        lens = [2000, 900]
        c = Cache(2, 2, D, 32, lens, seed=G)
        q = ref.bf16(c.rng.standard_normal((2, 2 * G, Lq, D)))
        dev, qd = c.device(), q.to(DEV)
        o, lse = attend(c, G, Lq, lens, q=q, dev=dev)
        calls.append((dev, qd, i32(lens), o, lse, fa2().fa2_cache_attn_workspace(qd, dev[0]), torch.cuda.Stream(DEV)))
    outs = [[(torch.zeros_like(o), torch.zeros_like(lse)) for _ in range(8)] for _, _, _, o, lse, _, _ in calls]
    torch.cuda.synchronize()
    for i in range(8):
        for (dev, qd, kv, _, _, ws, stream), out in zip(calls, outs):
            fa2().fa2_cache_attn(qd, *dev, kv, *out[i], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for (_, _, _, o, lse, _, _), out in zip(calls, outs):
        assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in out)
    assert fa2().fa2_cache_get_device_error() == (0, 0)


def test_two_graphs_with_their_own_workspaces():
    """A step and a prompt chunk captured apart, replayed on two streams."""
    runs = []
    for G, Lq in [(4, 1), (4, 50)]:
        lens = [1300, 700]
        c = Cache(2, 1, 128, 16, lens, seed=G + Lq)
        q = ref.bf16(c.rng.standard_normal((2, G, Lq, 128)))
        dev, qd = c.device(), q.to(DEV)
        o, lse = attend(c, G, Lq, lens, q=q, dev=dev)
        o2, lse2, kv = torch.zeros_like(o), torch.zeros_like(lse), i32(lens)
        ws = fa2().fa2_cache_attn_workspace(qd, dev[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa2().fa2_cache_attn(qd, *dev, kv, o2, lse2, workspace=ws)
        runs.append((graph, torch.cuda.Stream(DEV), o, lse, o2, lse2, dev, qd, kv, ws))
    for _ in range(5):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, o, lse, o2, lse2, *_ in runs:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            o2.zero_(), lse2.zero_()
        torch.cuda.synchronize()
    assert fa2().fa2_cache_get_device_error() == (0, 0)


@pytest.mark.parametrize("Lq", [1, 30])
def test_a_padded_batch(Lq):
    """Sequences that only pad the batch: no length, no pages, no query rows (or rows that see nothing)."""
    lens = [200, 0, 90, 0, 0]
    c = Cache(5, 2, 128, 16, lens, seed=19 + Lq)
    attend(c, 4, Lq, lens, [Lq, 0, Lq, Lq, 0])
    c.table[1] = c.table[3] = 2 ** 31 - 1
    attend(c, 4, Lq, [200, 50, 90, 50, 0], [Lq, Lq, Lq, Lq, 0])


def test_sizes_past_an_int_are_not_cut_off():
    lens = [50, 20]
    c = Cache(2, 1, 64, 16, lens, seed=20)
    q = ref.bf16(c.rng.standard_normal((2, 4, 1, 64)))
    o, lse = attend(c, 4, 1, lens, q=q)
    o2, lse2 = attend(c, 4, 1, lens, q=q, window=2 ** 32 + 1, check=False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dev = c.device()
    for window in (-2, -2 ** 32):
        with pytest.raises(RuntimeError, match="FA2_ERR_INVALID_ARG"):
            fa2().fa2_cache_attn(q.to(DEV), *dev, i32(lens), o, lse, window=window)
    many = torch.zeros(64, dtype=torch.bfloat16, device=DEV).expand(2, 1, 2 ** 32 + 1, 64)
    with pytest.raises(ValueError):
        fa2().fa2_cache_write(many, many, *dev, i32([0, 0]))
    with pytest.raises(ValueError):
        fa2().fa2_cache_attn(many, *dev, i32(lens), many, lse)


def test_first_calls_of_a_process_may_be_captured():
    """Nothing that a first call sets up (kernel attributes, the error word) is missed or refused in a capture."""
    code = """
import torch, io_aware_exact_fa2_gb300 as f
dev = torch.device("cuda:0")
k = torch.ones(1, 1, 3, 64, dtype=torch.bfloat16, device=dev)
c = [torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
s = [torch.zeros(2, 1, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu) for _ in range(2)]
cache = (*c, *s, torch.tensor([[1, 0]], dtype=torch.int32, device=dev))
start, held = torch.zeros(1, dtype=torch.int32, device=dev), torch.full((1,), 3, dtype=torch.int32, device=dev)
back = [torch.zeros_like(k) for _ in range(2)]
outs = [(torch.zeros(1, n, 3, 64, dtype=torch.bfloat16, device=dev), torch.zeros(1, n, 3, device=dev)) for n in (2, 8)]
qs = [torch.ones_like(o) for o, _ in outs]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    f.fa2_cache_write(k, k, *cache, start)
    f.fa2_cache_read(*cache, *back, start)
    for q, (o, lse) in zip(qs, outs):
        f.fa2_cache_attn(q, *cache, held, o, lse)
graph.replay()
torch.cuda.synchronize()
assert all(bool((t == 1).all()) for t in (*back, *(o for o, _ in outs)))
print("done")
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0 and out.stdout.strip().endswith("done"), out.stderr[-2000:]
