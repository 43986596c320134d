"""Query rows and keys of zeros over fp8_e4m3_page under softmax scales of any size: scores are 0, whatever a factor between codes
and scores under- or overflows to.  Both kernels of kvq_extend (a wide table makes a call count as large) and the decode;
tolerances as tests/test_page_attention_gpu.py derives them."""
import pytest
import torch

from test_page_attention_gpu import check, decode, extend, pool, queries

pytestmark = pytest.mark.gpu
WIDE = 4200


def smallest_keys(p):
    """Pages of zero keys with the least scale, as an append of zeros leaves them, beside the others."""
    layout, codes, scales, table, g = p
    some = table[:, 1::3]
    some = some[some >= 0].long()
    codes[some, 0] = 0
    scales[some, 0] = 2.0 ** -32


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -12, 2.0 ** -36, 2.0 ** -60, 2.0 ** -120, 1e-44])
def test_rows_of_zeros(room, d, scale):
    lens, start = [200, 61], [0, 70, 110]
    p = pool(lens, 8, 2, d, seed=1, room=room)
    smallest_keys(p)
    q = queries(110, 8, d, p[4])
    q[::3] = 0
    q[1, 2] = 0
    out = extend(q, p, lens, start, scale)
    check(out[::3], *subset(q, p, lens, start, scale, slice(None, None, 3)))
    if scale < 1e-3:  # (scores of the others stay small)
        check(out, q, p, lens, start, scale)


def subset(q, p, lens, start, scale, rows):
    """What `check` needs to look at some rows alone: each as a sequence's last one."""
    pages, at, n = [], [], []
    for b in range(len(lens)):
        for r in range(start[b], start[b + 1]):
            pages.append(b)
            n.append(lens[b] - (start[b + 1] - 1 - r))
    keep = list(range(start[-1]))[rows]
    table = p[3][[pages[r] for r in keep]]
    return q[rows], (p[0], p[1], p[2], table, p[4]), [n[r] for r in keep], None, scale


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("f", [2.0 ** -60, 2.0 ** 60])
def test_queries_of_every_size_with_the_scale_to_match(room, d, f):
    lens, start = [200, 61], [0, 70, 110]
    p = pool(lens, 8, 2, d, seed=2, room=room)
    q = queries(110, 8, d, p[4])
    q[::7, 3] = 0
    big = (q.float() * f).to(torch.bfloat16)
    check(extend(big, p, lens, start, d ** -0.5 / f), big, p, lens, start, d ** -0.5 / f)


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_of_zeros_under_a_factor_past_the_largest_float(room, d):
    lens, start, scale = [200, 61], [0, 70, 110], 2.0 ** 100
    p = pool(lens, 8, 2, d, seed=3, room=room)
    p[1][:, 0] = torch.where((p[1][:, 0] & 0x7F) == 0x7F, p[1][:, 0], 0)
    used = p[3][p[3] >= 0].long()
    p[2][used, 0] = 2.0 ** 32
    q = (queries(110, 8, d, p[4]).float() * 2.0 ** 60).to(torch.bfloat16)
    check(extend(q, p, lens, start, scale), q, p, lens, start, scale)
    q = q[:2].contiguous()
    check(decode(q, p, lens, scale), q, p, lens, None, scale)
    check(decode(q, p, lens, -scale), q, p, lens, None, -scale)
