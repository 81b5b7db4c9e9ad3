"""Attention over a cache with NaN values: the numbers beside them.  A key that not every row sees has
its NaN codes taken out of the product and put back into the rows and columns they reach; the other
columns, and the rows before the key, must be what they are without it."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from test_cache_gpu import Cache, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Lq", [(1, 1), (3, 5), (3, 30), (4, 70)])
@pytest.mark.parametrize("window", [None, 20])
@pytest.mark.parametrize("workspace", [False, True])
def test_columns_beside_nan_values(D, G, Lq, window, workspace):
    """NaN codes in the newest tokens' values (seen by some rows), in old ones (by all, or by none behind
    a window), beside a missing page, and a page whose value scale is NaN."""
    lens = [400, 290, 131]
    c = Cache(3, 2, D, 16, lens, seed=D + G + Lq)
    for b, h, pos, d in [(0, 0, 399, 3), (0, 0, 398, D - 1), (0, 1, 380, 17), (0, 1, 20, 40), (0, 0, 140, 0),
                         (1, 0, 289, 33), (1, 0, 270, 34), (1, 1, 5, 2), (1, 1, 288, 2), (2, 0, 130, 63)]:
        c.v[c.table[b, pos // 16], h, pos % 16, d] = 0x7f | (pos % 2) << 7
    c.vs[c.table[2, 7], 1] = 255
    c.table[1, 16] = -1
    q = ref.bf16(c.rng.standard_normal((3, 2 * G, Lq, D)))
    o, lse = attend(c, G, Lq, lens, q=q, window=window, workspace=workspace, check=False)
    ref.check_beside_nan(o.cpu(), lse.cpu(), q.double().numpy(), c.k, c.v, c.ks, c.vs, c.table, lens, None, True, window,
                         D ** -0.5)
