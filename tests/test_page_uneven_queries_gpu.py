"""Query rows with one element far larger than the rest, in a dimension where the keys are zero, so that the small ones
decide: both kernels of kvq_extend (a wide table makes a call count as large) and the decode.

Elements of 2^-13 of the row's largest and more enter exactly, so tolerances are those of
tests/test_page_attention_gpu.py; smaller ones may be off by 2^-21 of the largest in the kernel for many rows, which moves a score by
at most x = sm_scale * 2^-21 * largest * max sum |k_i| and the output by (e^(2 x) - 1) of sum p |v|."""
import math

import pytest
import torch

import append_model as M
from test_page_attention_gpu import check, decode, extend, pool, queries

pytestmark = pytest.mark.gpu


def uneven(hq, d, room, largest):
    """Elements from 0.5 to 2 beside one of `largest`, in another dimension from row to row among four."""
    lens, start = [300, 61], [0, 70, 110]
    p = pool(lens, hq, 2, d, seed=6, room=room)
    dims = [0, 31, d // 2 + 1, d - 1]
    p[1][..., dims] = torch.where((p[1][..., dims] & 0x7F) == 0x7F, p[1][..., dims], torch.stack(
        [torch.zeros_like(p[1][:, 0][..., dims]), p[1][:, 1][..., dims]], 1))
    q = (torch.rand(110, hq, d, generator=p[4], device="cuda") * 1.5 + 0.5)
    q = torch.where(torch.rand(q.shape, generator=p[4], device="cuda") < 0.5, -q, q).to(torch.bfloat16)
    q[:, :, dims] = 0
    for i, x in enumerate(dims):
        q[i::4, :, x] = largest
    return lens, start, p, q


@pytest.mark.parametrize("room", [0, 4200])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [6, 8, 10, 12])
def test_exact_down_to_a_part_in_8192(room, d, power):
    lens, start, p, q = uneven(8, d, room, 2.0 ** power)
    check(extend(q, p, lens, start, d ** -0.5), q, p, lens, start, d ** -0.5)
    q = q[:2].contiguous()
    check(decode(q, p, lens, d ** -0.5), q, p, lens, None, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [14, 16])
def test_smaller_elements(d, power):
    lens, start, p, q = uneven(8, d, 4200, 1.75 * 2.0 ** power)
    layout, codes, scales, table, g = p
    out = extend(q, p, lens, start, d ** -0.5).double()
    clean = torch.where((codes & 0x7F) == 0x7F, 0, codes)
    used = table[table >= 0].long()
    keys = M.page_values(clean[used], scales[used])[:, 0].abs().sum(-1).max().item()
    x = d ** -0.5 * 2.0 ** -21 * 1.75 * 2.0 ** power * keys
    ref, mag = M.attend64(q, clean, torch.nan_to_num(scales), table, lens, start, d ** -0.5, torch.zeros_like(out))
    assert ((out - ref).abs() <= (2.5e-3 + math.expm1(2 * x)) * mag + 1e-9).all()
