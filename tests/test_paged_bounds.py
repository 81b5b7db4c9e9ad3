"""What paged_bounds lets through, on the CPU: weights rounded as the 16-bit cache's attention rounds them are
within its bounds, and a lost second term or a lift that is not there is not."""
import pytest
import torch

import paged_bounds as bounds
import paged_reference as ref
from paged_reference import Cache

BF16, FP16 = torch.bfloat16, torch.float16


def passes(c, q, kv_lens, scale, causal=False, terms=1, lift=0.0):
    want = bounds.attention(q, c, kv_lens, causal=causal, scale=scale)
    try:
        ref.check_attention(*bounds.rounded(q, c, kv_lens, causal=causal, scale=scale, terms=terms, lift=lift), want)
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D,rows", [(64, 17), (128, 32), (64, 8), (256, 16)])
def test_a_lost_second_term_shows(D, rows, dtype):
    """Rows that are promised two terms, 17 to 32 of D = 64 and 128 among them."""
    c = Cache(1, 1, D, 16, [48], seed=D + rows, dtype=dtype, odd_after=False)
    q = c.randn(1, rows, 1, D).to(dtype)
    scale = bounds.few_alike(c, q, rows)
    lift = 6.0 if dtype == FP16 else -12.0
    assert passes(c, q, [48], scale, terms=2, lift=lift)
    assert not passes(c, q, [48], scale, terms=1, lift=lift)


def test_wide_bf16_heads_have_two_terms_for_any_rows():
    c = Cache(1, 1, 256, 16, [48], seed=1, dtype=BF16, odd_after=False)
    q = c.randn(1, 1, 40, 256).to(BF16)
    scale = bounds.few_alike(c, q, 1)
    assert passes(c, q, [48], scale, terms=2, lift=-12.0)
    assert not passes(c, q, [48], scale, terms=1, lift=-12.0)


@pytest.mark.parametrize("rows,terms", [(40, 1), (8, 2)])
def test_small_fp16_weights_need_the_lift(rows, terms):
    c = Cache(1, 1, 64, 16, [700], seed=rows, dtype=FP16, odd_after=False)
    q = torch.zeros(1, rows, 1, 64, dtype=FP16)
    scale = bounds.dominant(c, q, rows)
    assert passes(c, q, [700], scale, terms=terms, lift=6.0)
    assert not passes(c, q, [700], scale, terms=terms, lift=0.0)


def test_bf16_weights_need_no_lift():
    c = Cache(1, 1, 64, 16, [700], seed=3, dtype=BF16, odd_after=False)
    q = torch.zeros(1, 40, 1, 64, dtype=BF16)
    scale = bounds.dominant(c, q, 3)
    assert passes(c, q, [700], scale, terms=1, lift=-12.0)
