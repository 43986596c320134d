"""Every product and sum of kvq_append's rotation is rounded by itself: enough rows that a contracted product would show in the
rotated queries and in the codes (a fused one moves a bf16 result about once in 2^15 elements)."""
import pytest
import torch

import append_model as M
from test_append_gpu import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp8_e4m3_unscaled", "fp8_e4m3_page"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_no_product_is_contracted(kind, d, pairs):
    c = Cache(kind, 2, d, batch=2, room=30, seed=d)
    q, k, v = c.rows(600, 16)
    c.append([400, 200], q, k, v, angles=M.angles_of(400, d), pairs=pairs)


@pytest.mark.parametrize("pairs", [False, True])
def test_no_product_is_contracted_in_wide_rows(pairs):
    c = Cache("fp8_e4m3", 1, 576, batch=1, room=20, mla=True, dv=512, seed=3)
    q, k, _ = c.rows(300, 32)
    c.append([300], q, k, None, angles=M.angles_of(300, 64), first=512, pairs=pairs)


def test_zeros_and_huge_values_turn_as_they_should():
    """Products that are zero keep their signs, and no result is NaN that the definition's is not."""
    c = Cache("fp8_e5m2_unscaled", 1, 64, batch=1, room=4, seed=4)
    q, k, v = c.rows(50, 4)
    for x in (q, k, v):
        x[::3] = 0.0
        x[1::3, :, ::2] = -0.0
        x[2::7] *= 2.0 ** 100
    angles = M.angles_of(64, 64)
    angles[5:9, :32], angles[5:9, 32:] = 0.0, -1.0
    c.append([50], q, k, v, angles=angles)
