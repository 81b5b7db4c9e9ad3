"""Attention over the 16-bit cache to the bounds that include/fa2_paged.h promises for each form
(paged_bounds): how many terms a weight has, small fp16 weights, finite bf16 values of any size; and the
dense passes' workloads through the cache, every element, to the dense passes' own bar."""
import pytest
import torch

import oracle
import paged_bounds as bounds
import paged_reference as ref
from io_aware_exact_fa2_gb300.workloads import WORKLOADS, workload_inputs
from paged_reference import Cache
from parity import compare

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, FP16 = torch.bfloat16, torch.float16
MOST = float(torch.finfo(BF16).max)


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=DEV)


def run(q, dev, kv_lens, q_lens, causal, scale, workspace):
    import io_aware_exact_fa2_gb300 as fa2
    qd = q.to(DEV)
    o, lse = torch.zeros_like(qd), torch.zeros(q.shape[:3], device=DEV)
    ws = fa2.fa2_paged_attn_workspace(qd, dev[0]) if workspace else None
    fa2.fa2_paged_attn(qd, *dev, i32(kv_lens), o, lse, causal=causal, q_lens=None if q_lens is None else i32(q_lens),
                       scale=scale, workspace=ws)
    status, code = fa2.fa2_paged_get_device_error()
    assert status == 0, f"device error {code:#x}"
    return o.cpu(), lse.cpu()


def check(c, q, kv_lens, q_lens=None, causal=True, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    want, dev = bounds.attention(q, c, kv_lens, q_lens, causal, scale), c.device()
    for workspace in (True, False):
        ref.check_attention(*run(q, dev, kv_lens, q_lens, causal, scale, workspace), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("G,Lq", [(17, 1), (3, 6), (1, 23), (8, 4)])
def test_17_to_32_rows_have_two_terms(D, dtype, G, Lq):
    lens = [700, 129, 40]
    c = Cache(3, 2, D, 16, lens, seed=D + G, dtype=dtype, odd_after=False)
    q = c.randn(3, 2 * G, Lq, D).to(dtype)
    check(c, q, lens)
    check(c, q, lens, causal=False, scale=bounds.few_alike(c, q, G))


@pytest.mark.parametrize("Lq", [1, 20, 33, 140])
def test_wide_bf16_heads_have_two_terms(Lq):
    """D = 256: as the dense pass has them, for any number of rows."""
    lens = [700, 257, 140]
    c = Cache(3, 1, 256, 32, lens, seed=Lq, dtype=BF16, odd_after=False)
    q = c.randn(3, 2, Lq, 256).to(BF16)
    check(c, q, lens)
    check(c, q, lens, causal=False, scale=bounds.few_alike(c, q, Lq))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("Lq", [1, 5, 40, 300])
def test_small_weights_of_large_values(D, dtype, Lq):
    """One key far above all others, whose values are so large that they carry most of O."""
    lens = [2000, 500]
    c = Cache(2, 1, D, 64, lens, seed=D + Lq, dtype=dtype, odd_after=False)
    q = torch.zeros(2, 4, Lq, D, dtype=dtype)
    check(c, q, lens, [Lq, min(Lq, 100)], scale=bounds.dominant(c, q, D))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(4, 1), (8, 3), (4, 10), (4, 50)])
@pytest.mark.parametrize("size", [2.0 ** 122, MOST])
def test_largest_finite_values(D, G, Lq, size):
    """One to three keys with values of the largest size, in a sequence's only tile; then keys that stand out
    by less than what makes a row's reference rise, behind 200 others, with values of the largest size."""
    lens = [1, 2, 3]
    c = Cache(3, 1, D, 16, lens, seed=D + Lq, odd_after=False)
    c.v.copy_((c.v.sign() * size).to(BF16))
    q = (c.randn(3, G, Lq, D) * 0.1).to(BF16)
    check(c, q, lens, [1, min(Lq, 2), min(Lq, 3)])
    lens = [210, 300]
    c = Cache(2, 1, D, 16, lens, seed=D + Lq, odd_after=False)
    q = torch.zeros(2, G, Lq, D, dtype=BF16)
    q[..., 0] = 1
    c.k.zero_()
    for b in range(2):
        for p in (203, 204, 205):                  # 2^7.5 of the others' weights
            c.k[c.table[b, p // 16], :, p % 16, 0] = 7.5
            c.v[c.table[b, p // 16], :, p % 16] = (c.v[c.table[b, p // 16], :, p % 16].sign() * size).to(BF16)
    check(c, q, lens, [min(Lq, 5), Lq], causal=False, scale=0.6931471805599453)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Lq", [1, 6, 70, 200])
@pytest.mark.parametrize("power", [117, -110, -125])
def test_values_of_any_size_in_parts(D, Lq, power):
    """Values that are all very large or very small, keys shared out among CTAs."""
    lens = [3000, 900]
    c = Cache(2, 1, D, 32, lens, seed=D + Lq, odd_after=False)
    c.v.copy_((c.v.float().clamp(-4, 4) * 2.0 ** power).to(BF16))
    q = c.randn(2, 2, Lq, D).to(BF16)
    check(c, q, lens, [Lq, min(Lq, 60)])


@pytest.mark.parametrize("name,mode", [("c2", "noncausal"), ("c3", "causal"), ("c5", "noncausal")])
def test_dense_workloads_through_the_cache(name, mode):
    """Appended to a cache and attended to by all their queries at once, to the dense forward's bar: 1e-2, and
    half a step of O's where |O| >= 4.  (c5: D = 256, every 64th key eight times as large.)"""
    import io_aware_exact_fa2_gb300 as fa2
    w = WORKLOADS[name]
    q, k, v = workload_inputs(w)
    page = 64
    M = -(-w.Lk // page)
    g = torch.Generator().manual_seed(1)
    table = torch.randperm(w.B * M, generator=g).reshape(w.B, M).to(torch.int32).to(DEV)
    cache = [torch.zeros(w.B * M, w.H, page, w.D, dtype=BF16, device=DEV) for _ in range(2)]
    fa2.fa2_paged_append(k.to(DEV), v.to(DEV), *cache, table, i32([0] * w.B))
    want = oracle.attention(q, k, v, mode == "causal", w.scale)
    for workspace in (True, False):
        got = run(q, (*cache, table), [w.Lk] * w.B, None, mode == "causal", w.scale, workspace)
        print(name, mode, workspace, compare(*got, *want))
