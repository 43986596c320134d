"""kvq_extend over fp8_e4m3_page through tables far wider than the sequences: the call counts as large, which small ones need
to reach the kernel for many rows.  Tolerances as tests/test_page_attention_gpu.py derives them."""
import pytest
import torch

from test_page_attention_gpu import HEADS, check, extend, pool, queries

pytestmark = pytest.mark.gpu
WIDE = 4200


def starts(new):
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return start


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("old,new", [([0], [30]), ([5, 100, 0, 0, 16], [3, 1, 0, 40, 60]), ([33] * 9, [20] * 9), ([0, 0], [300, 127])])
def test_extend(old, new, hq, hkv, d):
    lens = [a + b for a, b in zip(old, new)]
    p = pool(lens, hq, hkv, d, seed=len(lens), room=WIDE)
    q = queries(sum(new) + 3, hq, d, p[4])
    for dtype in (torch.float32, torch.bfloat16):
        check(extend(q, p, lens, starts(new), d ** -0.5, dtype), q, p, lens, starts(new), d ** -0.5)


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_pages_and_late_maxima(d, room):
    lens = [400, 48, 100, 33]
    p = pool(lens, 8, 2, d, seed=3, room=room, spread=0.0)
    table, scales = p[3], p[2]
    for i, page in enumerate(table[0, :25].tolist()):
        scales[page, 0] *= 2.0 ** (i // 4 - 3)
    table[0, ::3] = -1
    table[1] = -1
    table[2, :5] = -1
    table[3, 2] = -1
    start = [0, 150, 190, 250, 270]
    q = queries(270, 8, d, p[4])
    out = extend(q, p, lens, start, d ** -0.5)
    check(out, q, p, lens, start, d ** -0.5)
    assert (out[150:190] == 0).all()


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_far_apart_in_size(d, room):
    lens = [500, 64]
    p = pool(lens, 8, 2, d, seed=4, room=room)
    layout, codes, scales, table, g = p
    used = torch.unique(table[table >= 0]).long()
    e = torch.randint(-32, 33, (used.numel(), layout.num_kv_heads), generator=g, device="cuda").double()
    scales[used, 1] = torch.pow(2.0, e).float()
    scales[used, 0] = torch.pow(2.0, (e % 5) - 12).float()
    q = queries(264, 8, d, g)
    check(extend(q, p, lens, [0, 200, 264], d ** -0.5), q, p, lens, [0, 200, 264], d ** -0.5)


@pytest.mark.parametrize("room", [0, WIDE])
def test_bad_pages_and_bad_sequences(room):
    d, lens = 128, [100, 60, 80]
    p = pool(lens, 8, 2, d, seed=9, room=room)
    q = queries(150, 8, d, p[4])
    start = [0, 40, 101, 131]  # sequence 1: more new tokens than stored ones
    check(extend(q, p, lens, start, d ** -0.5, status=-1), q, p, lens, start, d ** -0.5)
    start = [0, 60, 90, 130]
    p[3][1, 1] = p[0].num_pages
    check(extend(q, p, lens, start, d ** -0.5, status=-1), q, p, lens, start, d ** -0.5)
