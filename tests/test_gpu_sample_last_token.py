"""A random number of 1 or more takes the last token left, however little it weighs."""
import pytest
import torch

import cross_entropy_rl_gb300 as ll
from test_gpu_sample import TORCH, check, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=950), dict(top_k=40), dict(min_p=1e-25), dict(min_p=0.5),
                                dict(top_p=0.8), dict(top_k=990, min_p=1e-22), dict(temperature=0.0),
                                dict(temperature=0.3), dict(temperature=float(2 ** 20))], ids=str)
def test_last_tokens_of_no_weight(dtype, kw):
    # the last 100 of 1000 tokens weigh e^-40 to e^-60: less than 2^-46 of the largest
    x = rows(6, 1000, dtype, 71)
    x[:, 900:] = torch.linspace(-40, -60, 100, device="cuda").to(TORCH[dtype])
    x[1, 950:] = float("-inf")
    x[2, 940:] = x[2, 939]  # equal ones, of which top_k leaves the first
    x[3, 990:] = float("nan")
    u = torch.tensor([1.0, 1.5, 1.0, float("inf"), 1.0, 1 - 2.0 ** -24], device="cuda")
    check(x, u, **kw)
    x[:, 17] = x[0, 12] = float("inf")  # only these are drawn
    assert ll.sample(x, u.clamp(min=1.0), **kw)[0].tolist() == [12 if kw.get("temperature") == 0.0 else 17] + [17] * 5


def test_of_a_large_vocabulary():
    x = rows(3, 300001, "f32", 72)
    x[:, 250000:] = -70.0
    u = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    for kw in (dict(), dict(top_k=260000), dict(min_p=1e-40)):
        check(x, u, **kw)
