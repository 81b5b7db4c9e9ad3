"""Limits of the 8-bit cache's calls that the host can see, without a GPU: the largest that is taken
(which then finds no device) and the smallest that is refused."""
import pytest
import torch

from test_cache_abi import CUDA_ERR, INVALID, UNSUPPORTED, P, attn, cache, lib, ll3, write   # noqa: F401 (lib: a fixture)


# pages that L rows can touch, or pieces of 8192 / D rows; keys and values; B H heads: 2^31 - 1 at most
@pytest.mark.parametrize("f,D,page,L,heads_in,heads_over", [
    ("fa2_cache_write", 64, 16, 1 << 30, 15, 16),              # 2^26 + 1 pages
    ("fa2_cache_write", 128, 128, 1 << 30, 127, 128),          # 2^23 + 1
    ("fa2_cache_write", 256, 16, 1, (1 << 30) - 1, 1 << 30),   # one
    ("fa2_cache_read", 64, 16, 1 << 30, 127, 128),             # 2^23 pieces of 128 rows
    ("fa2_cache_read", 256, 64, 1 << 30, 31, 32),              # 2^25 of 32
    ("fa2_cache_read", 128, 16, 65, (1 << 29) - 1, 1 << 29),   # two of 64
])
def test_more_blocks_than_a_launch_counts_are_refused(lib, f, D, page, L, heads_in, heads_over):   # noqa: F811
    rows = ll3(1 << 38, 1 << 38, D)
    strides = dict(k_page=D * page, k_head=D * page, k_slot=D, v_page=D * page, v_head=D * page, v_slot=D)
    assert write(lib, cache(lib, B=heads_over, H=1, D=D, page_size=page, **strides), ks=rows, vs=rows, L=L, f=f) == UNSUPPORTED
    if not torch.cuda.is_available():   # (the pointers are not real)
        assert write(lib, cache(lib, B=heads_in, H=1, D=D, page_size=page, **strides), ks=rows, vs=rows, L=L, f=f) == CUDA_ERR


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38])
def test_a_scale_that_log2_e_takes_past_fp32_is_refused(lib, scale):   # noqa: F811
    assert attn(lib, cache(lib), scale=scale) == INVALID
    if not torch.cuda.is_available():
        assert attn(lib, cache(lib), scale=2.35e38) == CUDA_ERR
