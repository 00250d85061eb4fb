"""Norm rows of the largest finite values: the sum of their squares is beyond fp32 even for rows of
thousands of values, and the scale is right all the same (tolerance of check_norm: the sum's additions,
halved by the square root, and six roundings)."""

import numpy as np
import pytest
import torch

from speculative_decoding_04_b200 import dspark as D
from tests.test_gpu_head_q8 import DT, check_norm, f32, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 31, 256, 4095, 4096, 5120, 8200, 16383, 16384, 40000])
def test_norm_of_the_largest_values(dtype, d):
    rng = np.random.default_rng(d)
    top = float(torch.finfo(DT[dtype]).max)
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    x = np.stack([top * sign, 2.0 ** 127 * sign, top * sign * rng.random(d), 1e30 * rng.normal(size=d),
                  2.0 ** 64 * sign, np.where(np.arange(d) == d // 2, top, 0.0), 2.0 ** 58 * sign])
    for ld, off in ((d, 0), (d + 8, 8), (d + 1, 1), (d + 3, 3)):
        t = strided(x, dtype, ld, off)
        for gain in (1.0, 2.0 ** -100, 2.0 ** -20):
            g = torch.full((d,), gain, dtype=DT[dtype], device="cuda")
            q, s, _ = D.rmsnorm_q8(t, g, 1e-6)
            assert torch.all(s > 0)
            check_norm(f32(t), f32(g), 1e-6, q, s)
