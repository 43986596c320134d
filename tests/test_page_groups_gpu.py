"""Groups of many query heads to a key head over fp8_e4m3_page: more than half a tile's 128 rows to a token, and more than a tile,
cut into parts of which the last may be smaller.  Both kernels of kvq_extend (a wide table makes a call count as large) and the
decode; tolerances as tests/test_page_attention_gpu.py derives them."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from test_page_attention_gpu import KIND, check, decode, extend, ints, pool, queries

pytestmark = pytest.mark.gpu
WIDE = 9000
GROUPS = [(65, 1), (72, 1), (128, 1), (129, 1), (130, 1), (258, 2), (300, 1)]


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("hq,hkv", GROUPS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_extend(room, hq, hkv, d):
    lens, start = [90, 17, 200], [0, 5, 6, 13]
    p = pool(lens, hq, hkv, d, seed=hq, room=room)
    q = queries(15, hq, d, p[4])
    for dtype in (torch.float32, torch.bfloat16):
        check(extend(q, p, lens, start, d ** -0.5, dtype), q, p, lens, start, d ** -0.5)


@pytest.mark.parametrize("hq,hkv", GROUPS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode(hq, hkv, d):
    lens = [90, 1, 700]
    p = pool(lens, hq, hkv, d, seed=hq)
    q = queries(3, hq, d, p[4])
    check(decode(q, p, lens, d ** -0.5), q, p, lens, None, d ** -0.5)


@pytest.mark.parametrize("hq,hkv,d", [(130, 1, 64), (16, 8, 128), (16, 2, 256)])
def test_same_results_each_time_and_on_two_streams_at_once(hq, hkv, d):
    lens, start = [3000, 300, 77], [0, 200, 250, 327]
    p = pool(lens, hq, hkv, d, seed=3, room=WIDE)
    layout, codes, scales, table, g = p
    q = queries(327, hq, d, g)
    want = extend(q, p, lens, start, d ** -0.5)
    assert torch.equal(extend(q, p, lens, start, d ** -0.5), want)
    sl, st = ints(lens), ints(start)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [(torch.full_like(want, float("nan")), kvq.alloc_extend_workspace("cuda", layout, 327, hq, table.shape[1], kind=KIND,
                                                                            batch=3)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (out, ws) in zip(streams, work):
            with torch.cuda.stream(s):
                kvq.kvq_extend(q, codes, scales, table, sl, st, out, ws, layout, KIND, d ** -0.5)
    torch.cuda.synchronize()
    for out, ws in work:
        assert kvq.kvq_workspace_status(ws) == 0 and torch.equal(out, want)
