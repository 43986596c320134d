"""Pages whose values are far apart in size over fp8_e4m3_page, the large ones in a dimension of their own: the others must not
lose what the large page does not touch.  Both kernels of kvq_extend (a wide table makes a call count as large) and the decode.

P, the f16 that meets a token's codes, is off by at most 2^-11 of itself, or where it is below f16's normal range by 2^-25 of the
row's reference, which is 2^-7 of the row's largest p times scale or less.  Codes take up to 2^-14 of a page's scale where that is
more than 2^4 below a page's before it, so what P carries of the scales is within 2^4 while these are within 2^18: p is off by
at most 2^-11 of itself or 2^-28 of the row's largest p, and by as much more as a scale is further below.  What
tests/test_page_attention_gpu.py derives besides (2.5e-3 of sum p |v|) is for the scores and the first of the two."""
import pytest
import torch

import append_model as M
from test_page_attention_gpu import decode, extend, pool, queries

pytestmark = pytest.mark.gpu


def bound(q, p, lens, start, scale):
    """The definition's output and how far off it may be."""
    layout, codes, scales, table, g = p
    codes = torch.where((codes & 0x7F) == 0x7F, 0, codes)
    scales = torch.nan_to_num(scales)
    ref, mag = M.attend64(q, codes, scales, table, lens, start, scale, torch.zeros(q.shape, dtype=torch.float64, device="cuda"))
    low = torch.zeros_like(ref)
    hq, G = q.shape[1], q.shape[1] // layout.num_kv_heads
    for b, n in enumerate(lens):
        page = table[b, :-(-n // 16)].long()
        k = M.page_values(codes, scales)[page][:, 0].transpose(1, 2).flatten(0, 1)[:n].repeat_interleave(G, 1)  # [n, Hq, D]
        s = scales[page, 1].double()
        v = M.page_values(codes, scales)[page][:, 1].abs() * (s.amax(0) / s * 2.0 ** -18).clamp(min=1.0)[..., None, None]
        v = v.transpose(1, 2).flatten(0, 1)[:n].repeat_interleave(G, 1)
        rows = [b] if start is None else range(start[b], start[b + 1])
        for r in rows:
            see = n if start is None else n - (start[b + 1] - 1 - r)
            w = torch.softmax(torch.einsum("thd,hd->th", k[:see], q[r].double()) * scale, 0)
            low[r] = w.amax(0)[:, None] * v[:see].sum(0)
    return ref, 2.5e-3 * mag + 2.0 ** -28 * low + 1e-30


def values(lens, hq, hkv, d, room, far):
    """The pages' values around 1; the second page of every sequence has one element 2^far times as large, and zeros beside it."""
    p = pool(lens, hq, hkv, d, seed=8, spread=0.0, room=room)
    layout, codes, scales, table, g = p
    used = table[table >= 0].long()
    scales[used, 1] = 2.0 ** (-8 - far / 2)
    big = table[:, 1].long()
    codes[big, 1] = 0
    codes[big, 1, :, 5, 3] = 0x7E  # 448
    scales[big, 1] = 2.0 ** (far / 2)
    return p


@pytest.mark.parametrize("room", [0, 4200])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("far", [12, 20, 22, 24, 28, 32, 40])
def test_extend(room, d, far):
    lens, start = [200, 61], [0, 70, 110]
    p = values(lens, 8, 2, d, room, far)
    q = queries(110, 8, d, p[4])
    ref, off = bound(q, p, lens, start, d ** -0.5)
    assert ((extend(q, p, lens, start, d ** -0.5).double() - ref).abs() <= off).all()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 1, 128), (40, 2, 128), (16, 2, 256)])
@pytest.mark.parametrize("far", [12, 20, 22, 24, 28, 32, 40])
def test_decode(hq, hkv, d, far):
    lens = [200, 3000, 48]
    p = values(lens, hq, hkv, d, 0, far)
    q = queries(3, hq, d, p[4])
    ref, off = bound(q, p, lens, None, d ** -0.5)
    assert ((decode(q, p, lens, d ** -0.5).double() - ref).abs() <= off).all()
