"""What kvq_append and the calls over fp8_e4m3_page report: wherever the wrong number lies, each call its own report and nothing
of the call before."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

import append_model as M
from test_append_gpu import KINDS, Cache
from test_page_attention_gpu import check, decode, extend, ints, pool, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("at", [0, 31, 32, 33, 95, 299])
def test_a_position_outside_anywhere_in_a_long_sequence(kind, at):
    """Sequences of up to 32 new tokens are looked through by one thread, longer ones by 32."""
    c = Cache(kind, 2, 64, batch=3, room=20, seed=at)
    new = [1, 300, 2]
    q, k, v = c.rows(303, 2)
    positions = torch.arange(303).clamp(max=60).tolist()
    c.append(new, q, k, v, angles=M.angles_of(61, 64), positions=positions)
    q, k, v = c.rows(3, 2)
    c.append([1, 1, 1], q, k, v, angles=M.angles_of(400, 64))
    c = Cache(kind, 2, 64, batch=3, room=20, seed=at)
    q, k, v = c.rows(303, 2)
    positions[1 + at] = 61 if at % 2 else -5
    c.append(new, q, k, v, angles=M.angles_of(61, 64), positions=positions, status=-1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [0, 2, 17])
def test_a_page_outside_the_pool_anywhere_in_a_long_sequence(kind, page):
    c = Cache(kind, 2, 64, batch=2, room=20, seed=page)
    keep = int(c.table[1, page])
    c.table[1, page] = c.layout.num_pages + page
    c.dtable.copy_(c.table)
    q, k, v = c.rows(290, 2)
    c.append([2, 288], q, k, v, angles=M.angles_of(512, 64), status=-1)
    c.table[1, page] = keep
    c.dtable.copy_(c.table)
    q, k, v = c.rows(2, 2)
    c.append([1, 1], q, k, v, angles=M.angles_of(512, 64))


@pytest.mark.parametrize("kind", KINDS)
def test_places_past_the_table_of_angles(kind):
    c = Cache(kind, 2, 64, batch=40, room=4, seed=1)
    q, k, v = c.rows(40 + 50, 2)
    new = [1] * 39 + [51]
    c.append(new, q, k, v, angles=M.angles_of(51, 64))
    q, k, v = c.rows(40, 2)
    c.append([1] * 40, q, k, v, angles=M.angles_of(51, 64), status=-1)


@pytest.mark.parametrize("lens,hq,hkv", [([20], 2, 1), ([300, 40, 5000], 8, 2)])
@pytest.mark.parametrize("new", [1, 16])
def test_reports_of_small_and_large_attention_calls(lens, hq, hkv, new):
    """One CTA, which has the status word, and many, whose reports are collected; a report does not outlive its call."""
    d = 128
    p = pool(lens, hq, hkv, d, seed=2)
    layout, codes, scales, table, g = p
    start = [new * i for i in range(len(lens) + 1)]
    q, qn = queries(len(lens), hq, d, g), queries(start[-1], hq, d, g)
    ws = kvq.alloc_workspace(layout, len(lens), hq, table.shape[1], kind="fp8_e4m3_page")
    wx = kvq.alloc_extend_workspace("cuda", layout, start[-1], hq, table.shape[1], kind="fp8_e4m3_page", batch=len(lens))
    out, outn = torch.empty_like(q), torch.empty_like(qn)
    good = table.clone()
    for wrong in (True, False, True, False):
        table.copy_(good)
        if wrong:
            table[-1, (lens[-1] - 1) // 16] = layout.num_pages
        kvq.kvq_decode(q, codes, scales, table, ints(lens), out, ws, layout, "fp8_e4m3_page", 0.1)
        assert kvq.kvq_workspace_status(ws) == (-1 if wrong else 0)
        kvq.kvq_extend(qn, codes, scales, table, ints(lens), ints(start), outn, wx, layout, "fp8_e4m3_page", 0.1)
        assert kvq.kvq_workspace_status(wx) == (-1 if wrong else 0)
    check(decode(q, p, lens, 0.1), q, p, lens, None, 0.1)
    check(extend(qn, p, lens, start, 0.1), qn, p, lens, start, 0.1)
