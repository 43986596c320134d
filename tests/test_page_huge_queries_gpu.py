"""Queries near the ends of bf16's range over fp8_e4m3_page, with the softmax scale to match: both kernels of kvq_extend (a wide
table makes a call count as large) and the decode.  Tolerances as tests/test_page_attention_gpu.py derives them; queries
near 2^-118 lose up to 2^-19 of their row's largest element, which moves a score (sum |k_i| sm_scale |q| below 64 there) by at most
64 * 4 * 2^-19 = 2^-11, inside what that derivation leaves."""
import pytest
import torch

from test_page_attention_gpu import check, decode, extend, pool, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [0, 4200])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [-118, -100, 99, 102, 110, 124])
def test_sizes(room, d, power):
    lens, start = [200, 61], [0, 70, 110]
    scale = d ** -0.5 * 2.0 ** -power
    p = pool(lens, 8, 2, d, seed=2, room=room)
    q = (queries(110, 8, d, p[4]).float() * 2.0 ** power).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    check(extend(q, p, lens, start, scale), q, p, lens, start, scale)
    q = q[:2].contiguous()
    check(decode(q, p, lens, scale), q, p, lens, None, scale)
