"""kvq_append where byte offsets pass 32 bits, and two appends at once.  The arithmetic does not depend on where a page lies or on
what else runs, so results are compared bit by bit with those of tests/append_model.py on the CPU or of a small pool."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

import append_model as M
from test_append_gpu import KINDS, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
def test_pages_past_32_bits(kind):
    """The same steps into a small pool and into the last pages of one of more than 2^32 codes."""
    d, hkv = 128, 2
    c = Cache(kind, hkv, d, batch=2, room=3, seed=1)
    n = (1 << 32) // (2 * hkv * 16 * d) + 2000
    first = n - c.layout.num_pages
    L = kvq.Layout(n, 16, hkv, d, d)
    codes, scales = kvq.alloc_pool(L, kind=kind)
    codes[first:], scales[first:] = c.dcodes, c.dscales
    before = codes[:first].view(torch.int64).sum()
    table = c.dtable + first
    angles = M.angles_of(48, d)
    for new in ([20, 3], [1, 1], [0, 17]):
        q, k, v = c.rows(sum(new), 4)
        c.append(new, q, k, v, angles=angles)
        lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
        start = torch.tensor([0, new[0], sum(new)], dtype=torch.int32).cuda()
        kvq.kvq_append(codes, None if "unscaled" in kind else scales, k.cuda(), v.cuda(), table, lens, start, c.ws, L, kind,
                       q=q.cuda(), q_out=torch.empty_like(q, device="cuda"), cos_sin=angles.cuda())
        assert kvq.kvq_workspace_status(c.ws) == 0
        assert torch.equal(codes[first:], c.dcodes)
        if "unscaled" not in kind:
            bits = torch.int32 if kind == "fp8_e4m3_page" else torch.int16
            assert torch.equal(scales[first:].view(bits), c.dscales.view(bits))
    assert codes[:first].view(torch.int64).sum() == before, "a page elsewhere was written"


@pytest.mark.parametrize("kind", KINDS)
def test_two_appends_at_once(kind):
    """Two sequences' prompts into one pool, each on a stream and with a workspace of its own."""
    d = 128
    c = Cache(kind, 2, d, batch=2, room=40, seed=2)
    lens, n = [600, 531], 1131
    q, k, v = c.rows(n, 8)
    angles = M.angles_of(640, d)
    dq, dk, dv, cs = q.cuda(), k.cuda(), v.cuda(), angles.cuda()
    out = torch.empty_like(dq)
    streams = [torch.cuda.Stream() for _ in range(2)]
    parts = [(0, 600), (600, 1131)]
    args = [(c.dtable[b:b + 1], torch.tensor([lens[b]], dtype=torch.int32).cuda(),
             torch.tensor([0, hi - lo], dtype=torch.int32).cuda(), kvq.alloc_append_workspace()) for b, (lo, hi) in enumerate(parts)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (lo, hi), (table, sl, st, ws) in zip(streams, parts, args):
            with torch.cuda.stream(s):
                kvq.kvq_append(c.dcodes, None if "unscaled" in kind else c.dscales, dk[lo:hi], dv[lo:hi], table, sl, st, ws,
                               c.layout, kind, q=dq[lo:hi], q_out=out[lo:hi], cos_sin=cs)
    torch.cuda.synchronize()
    want = torch.empty_like(q)
    M.append(c.codes, c.scales, q, k, v, c.table, lens, [0, 600, 1131], c.layout, kind, angles, q_out=want)
    for a in args:
        assert kvq.kvq_workspace_status(a[3]) == 0
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16)) and torch.equal(c.dcodes.cpu(), c.codes)
    if "unscaled" not in kind:
        bits = torch.int32 if kind == "fp8_e4m3_page" else torch.int16
        assert torch.equal(c.dscales.cpu().view(bits), c.scales.view(bits))
