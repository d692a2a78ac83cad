"""The floor under the tokens that a min_p may leave: below its border, also where the border
comes out next to 0 as the difference of two numbers that are not."""
import math

import numpy as np
import pytest
import torch

from test_gpu_sample import check, uniforms

pytestmark = pytest.mark.gpu


# 1e-9 from the border (of a weight): more than the weights' 2^-37, less than an FP32 rounding
@pytest.mark.parametrize("near", [-1e-9, 1e-9])
@pytest.mark.parametrize("T", [1.0, 0.37, 5.0])
@pytest.mark.parametrize("at", [0.0, 2.0 ** -23, -3e-7])
def test_a_border_next_to_0(T, at, near):
    at = float(np.float32(at))
    for i in range(24):
        top = float(np.float32((0.0625 + 0.19 * i) * T))
        x = torch.full((8, 400), -9.0 * T, device="cuda")
        x[:, 7] = top
        x[:, 50:90] = at  # left for near < 0, else not
        check(x, uniforms(8, i), min_p=math.exp((at - top) / T) * (1 + near), temperature=T)
