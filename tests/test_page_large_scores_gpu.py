"""Scores far from zero over fp8_e4m3_page: the softmax does not know where zero is, and scores further apart than exponentials
reach leave the largest alone.  One token's key is twice or half as large as all others', so their scores are far apart: it has all
the weight, and the output is its value but for the rounding of its P to fp16, 2^-11.  kvq_extend's kernel for many rows (a
wide table makes a call count as large) gives rows up whose scores, times log2(e), pass 2^22: NaN and a report."""
import math

import pytest
import torch

from test_page_attention_gpu import check, decode, extend, pool, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room,power", [(0, -14), (0, -4), (0, 10), (0, 60), (0, 75), (0, 90), (4200, -14), (4200, -20)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_has_all_the_weight(room, d, power, sign):
    """Keys of 1.125 * 2^32 in dimension 1; queries of 2^power, or -2^power, and a bit there (products and scores have many
    bits, whose rounding is large beside what an exponential takes)."""
    lens, start = [200, 40], [0, 40, 80]
    p = pool(lens, 4, 2, d, seed=7, room=room)
    layout, codes, scales, table, g = p
    used = table[table >= 0].long()
    scales[used, 0] = 2.0 ** 32
    codes[used, 0] = 0
    codes[used, 0, :, :, 1] = 0x39
    best = [37, 0]
    for b, t in enumerate(best):
        codes[table[b, t // 16].long(), 0, :, t % 16, 1] = 0x41 if sign > 0 else 0x31
    q = torch.zeros(80, 4, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 1] = sign * 2.0 ** power * (1.0 + torch.arange(80, device="cuda")[:, None] / 128)

    def value(b, t):
        page = table[b, t // 16].long()
        return (codes[page, 1, :, t % 16].view(torch.float8_e4m3fn).float() * scales[page, 1][:, None]).repeat_interleave(2, 0)

    def near(out, v):
        return bool(((out - v).abs() <= 2.0 ** -10 * v.abs()).all())

    out = extend(q, p, lens, start, 1.0)
    assert near(out[:40], value(0, best[0])) and near(out[40:], value(1, best[1]))
    two = q[:2].contiguous()
    out = decode(two, p, lens, 1.0)
    assert near(out[0], value(0, best[0])) and near(out[1], value(1, best[1]))
    assert torch.equal(decode(two, p, [1, 1], 1.0), torch.stack([value(0, 0), value(1, 0)])), "one token alone"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [-9, -4, 10, 60, 90])
@pytest.mark.parametrize("sign", [1, -1])
def test_many_rows_are_given_up_one_by_one(d, power, sign):
    lens, start = [3000, 61], [0, 70, 110]
    p = pool(lens, 8, 2, d, seed=9, room=4200)
    layout, codes, scales, table, g = p
    used = table[table >= 0].long()
    codes[used, 0, :, :, 1] = torch.where((codes[used, 0, :, :, 1] & 0x7F) == 0x7F, codes[used, 0, :, :, 1], 0x38)
    scales[used, 0] = 2.0 ** -5  # every key has 2^-5 in dimension 1, so scores from 2^(power + 32) on are all of one sign
    q = queries(110, 8, d, g)
    q[:, :, 1] = 0
    clean, far = q.clone(), torch.zeros(110, 8, dtype=torch.bool, device="cuda")
    far[3::9, 2] = far[5::17, 7] = True
    q[:, :, 1] = torch.where(far, sign * 2.0 ** (power + 37), 0.0)
    # (power -9 stays below the border at head_dim 256: 2^23 * 4 / 16 * log2(e) = 3.0e6)
    past = 2.0 ** (power + 32) * d ** -0.5 * 4 * math.log2(math.e) > 2.0 ** 22
    assert past or (power, d) == (-9, 256)
    out = extend(q, p, lens, start, d ** -0.5 * 4, status=-1 if past else 0)
    assert torch.isnan(out[far]).all() if past else torch.isfinite(out).all()
    out[far] = extend(clean, p, lens, start, d ** -0.5 * 4)[far]
    check(out, clean, p, lens, start, d ** -0.5 * 4)
