"""The 64-bit format in torch operations against the numpy oracle (no GPU)."""

import numpy as np
import pytest
import torch

import q8_torch64 as q64
from oracle import q8


@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 128), (50, 300), (130, 517)])
def test_the_two_forms_of_the_format_agree(rows, cols):
    rng = np.random.default_rng(rows)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-140, 100, (rows, 1))) * np.exp2(rng.integers(-14, 1, (1, cols)))
    x[0, 0], x[-1, -1] = 0.0, 448.0
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    codes, scales = q8.encode(x)
    got = q64.encode(torch.from_numpy(x))
    assert np.array_equal(got[0].numpy(), codes) and np.array_equal(got[1].numpy(), scales)
    assert np.array_equal(q64.decode(*got).numpy(), q8.decode(codes, scales))
