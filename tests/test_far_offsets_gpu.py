"""Prompts, drafted tokens and pages where byte and element offsets pass 32 bits, and calls that run at the same time.
The arithmetic does not depend on where a page or a row lies or on what else runs, so results are compared bit by bit
with the same call on a small pool or on its own."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from plain64 import prompt64
from test_tree_gpu import RAGGED, Case

pytestmark = pytest.mark.gpu


def far_pool(c):
    """The pages of case c as the last ones of a pool of more than 2^32 bytes, and its table there."""
    per_page = c.codes[0].numel()
    pages = (1 << 32) // per_page + 1000 + c.L.num_pages
    L = kvq.Layout(pages, c.L.page_size, c.L.num_kv_heads, c.L.head_dim, c.L.v_dim, c.L.mla)
    codes = torch.empty(L.codes_shape(), dtype=torch.uint8, device="cuda")
    first = pages - c.L.num_pages
    codes[first:] = c.codes
    scales = None
    if c.scales is not None:
        scales = torch.empty(L.scales_shape(), dtype=c.scales.dtype, device="cuda")
        scales[first:] = c.scales
    near = (c.table >= 0) & (c.table < c.L.num_pages)
    return L, codes, scales, torch.where(near, c.table + first, c.table), first


@pytest.mark.parametrize("hq,hkv,d,mla,kind,path", [(16, 2, 256, False, "fp8_e4m3", 0), (32, 8, 128, False, "q8_0", 0),
                                                    (8, 2, 128, False, "fp8_e4m3_unscaled", 1),
                                                    (128, 1, 576, True, "fp8_e4m3", 0)])
def test_a_pool_past_32_bits(hq, hkv, d, mla, kind, path):
    c = Case(hq, hkv, d, kind, mla=mla, seed=5, **RAGGED)
    near, _ = c.run(path)
    c.check(near, tensor=path != 1)
    small = (c.codes, c.scales, c.table, c.L)
    L, codes, scales, table, first = far_pool(c)
    c.codes, c.scales, c.table, c.L = codes, scales, table, L
    far, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    assert torch.equal(far.view(torch.int32), near.view(torch.int32))

    # compaction there and in the small pool
    B = len(c.lens)
    keep = torch.tensor([[0x5A5A5A5A5A5A5A5 ^ (b * 77)] for b in range(B)], dtype=torch.int64).cuda()
    pws = kvq.alloc_pages_workspace(L, B, table.shape[1])
    lens = [torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2)]
    kvq.kvq_pages_compact(small[0], small[1], small[2], c.dl, c.ds, keep, lens[0], pws, small[3], kind)
    kvq.kvq_pages_compact(codes, scales, table, c.dl, c.ds, keep, lens[1], pws, L, kind)
    assert torch.equal(lens[0], lens[1]) and kvq.kvq_workspace_status(pws) == 0
    assert torch.equal(codes[first:], small[0])
    assert scales is None or torch.equal(scales[first:].view(torch.int16), small[1].view(torch.int16))

    # copies from the far end to the near one and back
    n = small[3].num_pages
    lo, hi = (torch.arange(a, a + n, dtype=torch.int32, device="cuda") for a in (0, first))
    kvq.kvq_pages_copy(codes, scales, hi, lo, L, kind)
    assert torch.equal(codes[:n], small[0])
    codes[first:].zero_()
    kvq.kvq_pages_copy(codes, scales, lo, hi, L, kind)
    assert torch.equal(codes[first:], small[0])
    assert scales is None or torch.equal(scales[:n].view(torch.int16), small[1].view(torch.int16))


def test_prompts_past_32_bits():
    """64 heads of 128 over one kv head, 600 prompts of 512 tokens: 2.5e9 elements of q, and of out."""
    hq, d, n, count = 64, 128, 512, 600
    total = n * count
    assert total * hq * d > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k = torch.empty(total, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty(total, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.empty_like(q)
    start = torch.arange(0, total + 1, n, dtype=torch.int32).cuda()
    ws = kvq.alloc_prompt_workspace()
    kvq.kvq_prompt(q, k, v, start, out, ws, sm_scale=d ** -0.5)
    assert kvq.kvq_workspace_status(ws) == 0
    for b in (0, 1, 255, 256, 511, 512, 513, count - 1):       # (element 2^31 lies in prompt 512)
        r = slice(b * n, (b + 1) * n)
        ref = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
        ref, mag = prompt64(q[r], k[r], v[r], [0, n], d ** -0.5, ref)
        # P in bf16 and the rest as in the tests of kvq_prompt, and the output's own rounding
        bound = 2.0 ** -7 * 0.8 * mag + 1e-6
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        assert ((out[r].double() - ref).abs() <= bound).all(), b
        one = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_prompt(q[r], k[r], v[r], start[:2].contiguous(), one, ws, sm_scale=d ** -0.5)
        assert torch.equal(out[r].view(torch.int16), one.view(torch.int16)), b


def test_calls_at_the_same_time():
    """Three streams: a prompt, drafted tokens over a cache, drafted tokens over the latent row, each with its own
    workspace, started together again and again."""
    a = Case(32, 8, 128, "q8_0", seed=1, **RAGGED)
    m = Case(64, 1, 576, "fp8_e4m3", mla=True, seed=2, **RAGGED)
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [700, 31, 1500, 1, 260]
    total = sum(lens)
    q = torch.empty(total, 16, 256, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k = torch.empty(total, 2, 256, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty(total, 2, 256, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    start = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    pws = kvq.alloc_prompt_workspace()

    def prompt():
        out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        kvq.kvq_prompt(q, k, v, start, out, pws, sm_scale=1 / 16)
        return out

    (ra, wa), (rm, wm), rp = a.run(), m.run(), prompt()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = []
        for s, f in zip(streams, (lambda: a.run(ws=wa)[0], lambda: m.run(ws=wm)[0], prompt)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for x, ref in zip(got, (ra, rm, rp)):
            assert torch.equal(x.view(torch.int32), ref.view(torch.int32))
        for w in (wa, wm, pws):
            assert kvq.kvq_workspace_status(w) == 0
