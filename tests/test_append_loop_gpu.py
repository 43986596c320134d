"""A serving loop as the calls are meant to be used together: pages are given, prompts appended and attended to, sequences
forked, tokens appended and decoded one at a time, chains of drafts appended, attended to and cut back."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

import append_model as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 3, 64), (4, 1, 256)])
def test_prompts_forks_tokens_and_drafts(hq, hkv, d):
    kind, B, room = "fp8_e4m3_page", 4, 12
    g = torch.Generator(device="cuda").manual_seed(d)
    L = kvq.Layout(B * room + 3, 16, hkv, d, d)
    codes, scales = kvq.alloc_pool(L, kind=kind)
    codes.fill_(0xFF)
    scales.fill_(float("nan"))
    table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(L.num_pages, dtype=torch.int32, device="cuda")
    pws = kvq.alloc_pages_workspace(L, B, room)
    aws = kvq.alloc_append_workspace()
    angles = M.angles_of(room * 16, d).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(new):
        """Appends new[b] tokens to every sequence and attends with them; both against the definition."""
        want = (lens + i32(new)).tolist()
        kvq.kvq_pages_resize(table, lens, refs, i32(range(B)), i32(want), pws, L)
        assert kvq.kvq_workspace_status(pws) == 0 and lens.tolist() == want
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        rows = torch.randn(start[-1], hq + 2 * hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        mine, own = codes.cpu(), scales.cpu()
        out_q = torch.empty(q.shape, dtype=torch.bfloat16)
        M.append(mine, own, q.cpu(), k.cpu(), v.cpu(), table.cpu(), want, start, L, kind, angles.cpu(), q_out=out_q)
        turned = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_append(codes, scales, k, v, table, lens, i32(start), aws, L, kind, q=q, q_out=turned, cos_sin=angles)
        assert kvq.kvq_workspace_status(aws) == 0
        assert torch.equal(codes.cpu(), mine) and torch.equal(turned.cpu().view(torch.int16), out_q.view(torch.int16))
        out = torch.empty(turned.shape, dtype=torch.float32, device="cuda")
        single = all(n == 1 for n in new)
        if single:
            ws = kvq.alloc_workspace(L, B, hq, room, kind=kind)
            kvq.kvq_decode(turned, codes, scales, table, lens, out, ws, L, kind, d ** -0.5)
        else:
            ws = kvq.alloc_extend_workspace("cuda", L, start[-1], hq, room, kind=kind, batch=B)
            kvq.kvq_extend(turned, codes, scales, table, lens, i32(start), out, ws, L, kind, d ** -0.5)
        assert kvq.kvq_workspace_status(ws) == 0
        clean = torch.where((codes & 0x7F) == 0x7F, 0, codes)
        ref, mag = M.attend64(turned, clean, torch.nan_to_num(scales), table, want, None if single else start, d ** -0.5,
                              torch.zeros(turned.shape, dtype=torch.float64, device="cuda"))
        err = (out.double() - ref).abs()
        assert (err <= 2.5e-3 * mag + 1e-9).all(), float((err / mag).max())  # as in test_page_attention_gpu.py

    step([37, 5, 90, 1])
    step([1, 1, 1, 1])
    src, dst = i32([0, 2]), i32([1, 3])  # sequences 1 and 3 go on from 0 and 2
    cs, cd = torch.empty_like(src), torch.empty_like(src)
    kvq.kvq_pages_fork(table, lens, refs, src, dst, cs, cd, pws, L)
    assert kvq.kvq_workspace_status(pws) == 0
    kvq.kvq_pages_copy(codes, scales, cs, cd, L, kind)
    for _ in range(3):
        step([1, 1, 1, 1])
    before = lens.clone()
    step([6, 4, 2, 5])          # drafts, of which some are accepted
    kept = before + i32([2, 4, 0, 1])
    kvq.kvq_pages_resize(table, lens, refs, i32(range(B)), kept, pws, L)
    step([1, 1, 1, 1])
    step([0, 30, 0, 3])


@pytest.mark.parametrize("hkv", [1, 2, 3])
def test_page_copies_take_the_scales_along(hkv):
    L = kvq.Layout(40, 16, hkv, 64, 64)
    g = torch.Generator(device="cuda").manual_seed(hkv)
    codes = torch.randint(0, 256, L.codes_shape(), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    scales = torch.randn(L.page_scales_shape(), generator=g, device="cuda")
    src = torch.tensor([3, 7, -1, 7, 40, 1], dtype=torch.int32, device="cuda")
    dst = torch.tensor([30, 31, 32, 33, 34, -1], dtype=torch.int32, device="cuda")
    want = codes.clone(), scales.clone()
    for x in want:
        x[30], x[31], x[33] = x[3].clone(), x[7].clone(), x[7].clone()
    kvq.kvq_pages_copy(codes, scales, src, dst, L, "fp8_e4m3_page")
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
