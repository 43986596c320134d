"""A query row that holds an infinity or a NaN gives NaN over fp8_e4m3_page, in both kernels of kvq_extend (a wide table makes a
call count as large) and the decode, and leaves the other rows alone.  Tolerances of these as
tests/test_page_attention_gpu.py derives them."""
import pytest
import torch

from test_page_attention_gpu import check, decode, extend, pool, queries

pytestmark = pytest.mark.gpu
BAD = [float("inf"), float("-inf"), float("nan")]


def spoil(q):
    """q with a bad element in some heads' rows, zeros there in its twin, and which rows these are."""
    clean, bad = q.clone(), torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for i, x in enumerate(BAD * 2):
        row, head = (11 * i + 3) % q.shape[0], (3 * i + 1) % q.shape[1]
        q[row, head, (29 * i) % q.shape[2]] = x
        clean[row, head] = 0
        bad[row, head] = True
    return clean, bad


@pytest.mark.parametrize("room", [0, 4200])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_extend(room, d):
    lens, start = [200, 61, 40], [0, 70, 110, 120]
    p = pool(lens, 8, 2, d, seed=4, room=room)
    p[1][:, 0] |= torch.where((p[1][:, 0] & 0x7F) == 0x7F, 0, 0x80).to(torch.uint8)  # keys below zero: no score is +inf
    p[3][2] = -1
    q = queries(120, 8, d, p[4])
    clean, bad = spoil(q)
    q[115, 2, 5] = float("inf")  # (a row that sees nothing)
    out, ref = extend(q, p, lens, start, d ** -0.5), extend(clean, p, lens, start, d ** -0.5)
    assert torch.isnan(out[bad]).all() and (out[110:120] == 0).all()
    out[bad] = ref[bad]
    check(out, clean, p, lens, start, d ** -0.5)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 1, 64), (40, 2, 256)])
def test_decode(hq, hkv, d):
    lens = [33, 5000, 1, 700, 16, 90, 250]
    p = pool(lens, hq, hkv, d, seed=5)
    p[1][:, 0] |= torch.where((p[1][:, 0] & 0x7F) == 0x7F, 0, 0x80).to(torch.uint8)
    q = queries(len(lens), hq, d, p[4])
    clean, bad = spoil(q)
    out, ref = decode(q, p, lens, d ** -0.5), decode(clean, p, lens, d ** -0.5)
    assert torch.isnan(out[bad]).all()
    out[bad] = ref[bad]
    check(out, clean, p, lens, None, d ** -0.5)
