"""The check of attention beside NaN values (cache_reference.check_beside_nan), on the CPU."""
import numpy as np
import pytest
import torch

import cache_reference as ref


def test_a_wrong_number_beside_a_nan_is_found():
    rng = np.random.default_rng(0)
    n, D = 128, 64
    k, v = (ref.encode(rng.standard_normal((8, 1, 16, D)) * 90) for _ in range(2))
    v[3, 0, 2, 5] = 0x7f
    one = np.full((8, 1), 120, np.uint8)
    q = ref.bf16(rng.standard_normal((1, 1, 2, D))).double().numpy()
    args = (q, k, v, one, one, np.arange(8)[None], [n], None, True, None, D ** -0.5)
    o, lse, _, _ = ref.attention(*args)
    assert np.isnan(o[..., 5]).all() and np.isnan(o).sum() == 2
    o, lse = torch.from_numpy(o), torch.from_numpy(lse)
    ref.check_beside_nan(o, lse, *args)
    for at, wrong in (((0, 0, 1, 6), 123.0), ((0, 0, 0, 5), 1.0), ((0, 0, 0, 9), float("nan")),
                      ((0, 0, 0, 0), float(o[0, 0, 0, 0]) + 0.05)):
        planted = o.clone()
        planted[at] = wrong
        with pytest.raises(AssertionError):
            ref.check_beside_nan(planted, lse, *args)
    with pytest.raises(AssertionError):
        ref.check_beside_nan(o, lse + 1e-2, *args)
