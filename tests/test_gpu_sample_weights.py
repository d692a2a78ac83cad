"""The integer weights of a draw, to 2^-36 of their size: a min_p that far below or above a
token's weight keeps it or not."""
import math

import numpy as np
import pytest
import torch

import cross_entropy_rl_gb300 as ll

pytestmark = pytest.mark.gpu


# The header gives weights to 2^-37 of their size, in units of 2^-46 of the largest (rounded: half a
# unit is 2^-37 of a weight of 2^-10, the least one here), and min_p is a number of such units,
# rounded up: 2^-36 of such a weight.
@pytest.mark.parametrize("side", [-1, 1])
@pytest.mark.parametrize("T", [1.0, 0.61, 1.7])
@pytest.mark.parametrize("offset", [0.0, 1000.0])
def test_to_2_to_the_minus_36(offset, T, side):
    rng = np.random.default_rng(17)
    u = torch.tensor([1 - 2.0 ** -24], device="cuda")  # the last token left
    wrong = []
    for _ in range(150):
        a = rng.uniform(-math.log(2) * 10, -0.01)
        top = np.float32(rng.uniform(1, 4) + offset)
        x = np.float32(float(top) + a * T)
        exact = math.exp((float(x) - float(top)) / T)
        row = torch.full((1, 40), float(top) - 200 * T, device="cuda")
        row[0, 3], row[0, 20] = float(top), float(x)
        min_p = exact * (1 + side * (2.0 ** -37 + (2.0 ** -46 + 2.0 ** -47) / exact))
        token = int(ll.sample(row, u, temperature=T, min_p=min_p)[0])
        if token != (3 if side > 0 else 20):
            wrong.append((top, x, exact, token))
    assert not wrong
