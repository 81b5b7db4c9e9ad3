"""The 8-bit cache's bounded waits: one that runs out is reported by fa2_cache_get_device_error, the
kernel winds down, writes nothing but its rows, and the next call on the context is right.

The time-outs are made on purpose: FA2_TEST_STALL=2 makes some warps tens of microseconds late, and with
FA2_TEST_WAIT_LIMIT_NS=1 the issuing warp does not wait so long; then the waits of the softmax, loading
and converting warps on it run out in turn.  Nothing faults: a role that has given up waiting runs on to
its end, with addresses that do not depend on what it waited for, and the copies and products in
flight are waited for (with the full bound of a second) before a CTA goes.
"""
import pytest
import torch

import cache_reference as ref
from test_cache_gpu import DEV, FILL, Cache, attend, fa2, i32

pytestmark = pytest.mark.gpu

FA2_ERR_TIMEOUT = 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(1, 1), (16, 1), (20, 1), (4, 60)])
@pytest.mark.parametrize("workspace", [False, True])
def test_a_time_out_is_reported_and_the_next_call_is_right(monkeypatch, D, G, Lq, workspace):
    lens, q_lens = [3000, 700], [Lq, max(1, Lq - 7)]
    c = Cache(2, 1, D, 16, lens, seed=D + G + Lq)
    q = ref.bf16(c.rng.standard_normal((2, G, Lq, D)))
    dev, qd = c.device(), q.to(DEV)
    assert fa2().fa2_cache_get_device_error() == (0, 0)
    # rows of o lie apart, and behind the last sequence's there are others
    wide = torch.full((2, G, Lq, D + 8), FILL, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, G, Lq), FILL, device=DEV)
    ws = fa2().fa2_cache_attn_workspace(qd, dev[0]) if workspace else None
    monkeypatch.setenv("FA2_TEST_STALL", "2")
    monkeypatch.setenv("FA2_TEST_WAIT_LIMIT_NS", "1")
    for _ in range(3):
        if workspace:
            ws.zero_()
        fa2().fa2_cache_attn(qd, *dev, i32(lens), wide[..., :D], lse, q_lens=i32(q_lens), workspace=ws)
        st, code = fa2().fa2_cache_get_device_error()
        assert st == FA2_ERR_TIMEOUT, (st, hex(code))
        # softmax, loading, issuing (and converting) warps; never a CTA's wait for its own work
        assert code >> 8 in ((12, 13, 14) if G * Lq <= 16 else (8, 9, 10, 11)), hex(code)
        assert fa2().fa2_cache_get_device_error() == (0, 0)   # read and cleared
    assert torch.all(wide[..., D:] == FILL)
    for b in range(2):
        assert torch.all(wide[b, :, q_lens[b]:] == FILL) and torch.all(lse[b, :, q_lens[b]:] == FILL)
    monkeypatch.delenv("FA2_TEST_STALL")
    monkeypatch.delenv("FA2_TEST_WAIT_LIMIT_NS")
    attend(c, G, Lq, lens, q_lens, q=q, dev=dev, workspace=workspace)
