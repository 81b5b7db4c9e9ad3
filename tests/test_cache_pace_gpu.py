"""Results of attention over the 8-bit cache must not depend on the pace of its warps: with the
library's test switch FA2_TEST_STALL=2 the second of the two warps that exchange a row's largest
|q| reads its partner's tens of microseconds late (in the last row tile of a block of many rows),
and the warp that loads the keys of few rows begins as late, while the others run ahead as far as
they may."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from test_cache_gpu import DEV, FILL, Cache, attend, fa2, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(17, 1), (2, 33), (1, 128), (4, 40), (1, 3), (16, 1)])
@pytest.mark.parametrize("workspace", [False, True])
def test_a_late_warp(monkeypatch, D, G, Lq, workspace):
    """Query rows whose halves (the two warps' shares) are of very different size, so that a number
    exchanged at the wrong time shows; units of one row tile twice, of two, and of one alone."""
    lens = [Lq, 700, Lq + 140]
    c = Cache(3, 2, D, 32, lens, seed=D + G + Lq)
    q = c.rng.standard_normal((3, 2 * G, Lq, D)) * 0.7
    q[..., :D // 2] *= 2.0 ** -6
    q = ref.bf16(q)
    o, lse = attend(c, G, Lq, lens, q=q, workspace=workspace)
    monkeypatch.setenv("FA2_TEST_STALL", "2")
    late, late_lse = attend(c, G, Lq, lens, q=q, workspace=workspace)
    assert torch.equal(o, late) and torch.equal(lse, late_lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(20, 1), (2, 70)])
@pytest.mark.parametrize("workspace", [False, True])
def test_from_unit_to_unit(D, G, Lq, workspace):
    """More blocks of rows than CTAs: every warp takes its next block's sequence, head and tiles from its
    first lane, for blocks of one tile and of several, of few rows and of many, in turn."""
    B, H = 50, 4
    rng = np.random.default_rng(D + Lq)
    lens = rng.integers(1, 400, B)
    c = Cache(B, H, D, 16, lens, seed=D + G)
    attend(c, G, Lq, lens, rng.integers(0, Lq + 1, B), workspace=workspace)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(8, 1), (16, 1), (20, 1), (3, 100)])
def test_every_counter_is_left_at_zero(D, G, Lq):
    """Two contexts over all CTAs, up to three an SM: the counters of all of them (8 bytes a CTA, room for
    four CTAs an SM, in 256-byte steps) are zero after each call, and each gives the same bits."""
    lens = [60011, 20007]
    c = Cache(2, 1, D, 128, lens, seed=D + G, nan_after=False)
    dev, q = c.device(), ref.bf16(c.rng.standard_normal((2, G, Lq, D))).to(DEV)
    kv = i32(lens)
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    region = (sms * 4 * 8 + 255) // 256 * 256
    ws = fa2().fa2_cache_attn_workspace(q, dev[0])
    assert ws.numel() > region
    outs = []
    for _ in range(3):
        o, lse = torch.zeros_like(q), torch.zeros(2, G, Lq, device=DEV)
        fa2().fa2_cache_attn(q, *dev, kv, o, lse, workspace=ws)
        assert not ws[:region].any()
        outs.append((o, lse))
    assert ws[region:].any()    # (parts were left there)
    assert all(torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1]) for o, lse in outs)
    assert torch.isfinite(outs[0][0]).all()
    assert fa2().fa2_cache_get_device_error() == (0, 0)


@pytest.mark.parametrize("Lq", [1, 64])
def test_empty_sequences_behind_the_last_cost_little(Lq):
    """A batch padded to 4096 sequences, eight of them live: the same bits as of the eight alone, and not
    many times their time (1.4 of it, where reading each empty sequence's length took 18)."""
    B, H, G, D, page, n = 8, 8, 4, 128, 64, 4000
    c = Cache(B, H, D, page, [n] * B, seed=Lq, nan_after=False)
    dev = c.device()
    times, outs = [], []
    q0 = torch.randn(B, H * G, Lq, D, device=DEV).to(torch.bfloat16)
    for batch in (B, 4096):
        table = torch.zeros(batch, c.M, dtype=torch.int32, device=DEV)
        table[:B] = dev[4]
        kv, ql = (torch.zeros(batch, dtype=torch.int32, device=DEV) for _ in range(2))
        kv[:B], ql[:B] = n, Lq
        q = torch.zeros(batch, H * G, Lq, D, dtype=torch.bfloat16, device=DEV)
        q[:B] = q0
        o, lse = torch.full_like(q, FILL), torch.full((batch, H * G, Lq), FILL, device=DEV)
        ws = fa2().fa2_cache_attn_workspace(q, dev[0])
        best = float("inf")
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):   # (more device time than host time)
                fa2().fa2_cache_attn(q, *dev[:4], table, kv, o, lse, q_lens=ql, workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        outs.append((o[:B], lse[:B]))
        assert torch.all(o[B:] == FILL) and torch.all(lse[B:] == FILL)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert times[1] <= 5 * times[0], times
