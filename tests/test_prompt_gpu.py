"""kvq_prompt on the GPU against the definition in 64 bits.

Tolerance, relative to sum_t p_t |v_t| of the row: P is rounded to bf16, at most 2^-8 of each p; q.k in fp32 (256
products at most, sum |q_i k_i| * sm_scale below 64 here) is off by less than 64 * 256 * 2^-24 = 1e-3 in the worst order,
which changes p and the normaliser by as much each: 2^-8 + 2e-3 < 2^-7 * 0.8.  That is far above what occurs, so
the mean over all outputs is held to a quarter of 2^-8.  A bf16 output adds its own rounding, 2^-8 of the value."""
import random

import numpy as np
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from plain64 import attend, prompt64

pytestmark = pytest.mark.gpu


def inputs(lens, hq, hkv, d, seed=0, behind=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = sum(lens) + behind
    q = (torch.randn(t, hq, d, generator=g, device="cuda") * scale).to(torch.bfloat16)
    k = (torch.randn(t, hkv, d, generator=g, device="cuda")
         * torch.exp(0.5 * torch.randn(hkv, d, generator=g, device="cuda"))).to(torch.bfloat16)
    v = torch.randn(t, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    start = [0] + [int(x) for x in np.cumsum(lens)]
    return q, k, v, start


def run(q, k, v, start, dtype=torch.float32, out=None, scale=None):
    if out is None:
        out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ws = kvq.alloc_prompt_workspace()
    ws.fill_(0x5A)
    kvq.kvq_prompt(q, k, v, torch.tensor(start, dtype=torch.int32).cuda(), out, ws,
                   sm_scale=q.shape[2] ** -0.5 if scale is None else scale)
    return out, ws


def check(out, q, k, v, start, dtype=torch.float32, skipped=(), extra=1.0):
    ref = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    covered = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    mag = torch.zeros_like(ref)
    for b, (r0, r1) in enumerate(zip(start[:-1], start[1:])):
        if b in skipped or r1 <= r0:
            continue
        covered[r0:r1] = True
        step = max(1, (1 << 27) // ((r1 - r0) * q.shape[1]))
        if r1 - r0 <= 2500:
            ref[r0:r1], mag[r0:r1] = prompt64(q[r0:r1], k[r0:r1], v[r0:r1], [0, r1 - r0], q.shape[2] ** -0.5,
                                              ref[r0:r1].clone())
        else:
            for a in range(r0, r1, step):
                z = min(r1, a + step)
                seen = torch.arange(r0, z, device="cuda")[None] <= torch.arange(a, z, device="cuda")[:, None]
                ref[a:z], mag[a:z] = attend(q[a:z], k[r0:z].double(), v[r0:z].double(), seen, q.shape[2] ** -0.5)
    assert torch.isnan(out[~covered]).all(), "rows that no sequence covers were written"
    got, ref, mag = out[covered].double(), ref[covered], mag[covered]
    assert torch.isfinite(got).all()
    bound, mean = 2.0 ** -7 * 0.8 * extra * mag + 1e-6, 2.0 ** -10 * extra * mag.mean() + 1e-6
    if dtype == torch.bfloat16:
        bound, mean = bound + 2.0 ** -8 * (ref.abs() + bound), mean + 2.0 ** -8 * ref.abs().mean()
    err = (got - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())
    assert err.numel() == 0 or err.mean() <= mean, (float(err.mean()), float(mean))


HEADS = [(8, 2, 128), (16, 8, 128), (5, 5, 128), (3, 1, 128), (12, 2, 64), (7, 7, 64), (9, 3, 64), (16, 2, 256),
         (3, 3, 256)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [127, 128, 129], [0, 5, 0, 300, 64, 1, 513, 0], [256], [700, 31, 700]])
def test_packed_prompts(lens, hq, hkv, d):
    q, k, v, start = inputs(lens, hq, hkv, d, seed=len(lens), behind=3)
    out, ws = run(q, k, v, start)
    assert kvq.kvq_workspace_status(ws) == 0
    check(out, q, k, v, start)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (16, 2, 256)])
@pytest.mark.parametrize("lens", [[5000], [2048, 1500, 3000, 17], [40] * 300])
def test_more_items_than_multiprocessors(lens, hq, hkv, d):
    q, k, v, start = inputs(lens, hq, hkv, d, seed=7)
    for dtype in (torch.float32, torch.bfloat16):
        out, ws = run(q, k, v, start, dtype)
        assert kvq.kvq_workspace_status(ws) == 0
        check(out, q, k, v, start, dtype)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 64), (4, 1, 256)])
def test_what_lies_outside_a_sequence_does_not_matter(hq, hkv, d):
    """NaN and infinities in rows behind the last sequence, between sequences and in other sequences."""
    lens = [100, 77, 300, 30]
    q, k, v, start = inputs(lens, hq, hkv, d, seed=2, behind=50)
    alone = []
    for r0, r1 in zip(start[:-1], start[1:]):
        o, _ = run(q[r0:r1].clone(), k[r0:r1].clone(), v[r0:r1].clone(), [0, r1 - r0])
        alone.append(o)
    for poison in (float("nan"), float("inf"), -float("inf")):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for x in (q2, k2, v2):
            x[start[1]:start[2]] = poison     # sequence 1
            x[start[4]:] = poison             # behind the last one
        out, ws = run(q2, k2, v2, start)
        assert kvq.kvq_workspace_status(ws) == 0
        for b in (0, 2, 3):
            assert torch.equal(out[start[b]:start[b + 1]], alone[b])
        assert torch.isnan(out[start[4]:]).all()


def test_strides_of_one_projection():
    """q, k, v as slices of one [T, (Hq + 2 Hkv) D] projection, heads first, and a strided output."""
    lens, hq, hkv, d = [200, 333], 8, 2, 128
    q, k, v, start = inputs(lens, hq, hkv, d, seed=3)
    want, _ = run(q, k, v, start)
    t = q.shape[0]
    packed = torch.cat([q, k, v], 1).contiguous()
    got, ws = run(packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:], start)
    assert kvq.kvq_workspace_status(ws) == 0 and torch.equal(got, want)
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    buf = torch.full((hq, t + 5, d + 8), float("nan"), device="cuda")
    got, _ = run(*heads_first, start, out=buf[:, :t, :d].transpose(0, 1))
    assert torch.equal(got, want) and torch.isnan(buf[:, t:]).all() and torch.isnan(buf[:, :, d:]).all()
    one = torch.cat([k[:, :1], v[:, :1]], 1).contiguous()      # one kv head: its stride says nothing
    want, _ = run(q, k[:, :1].contiguous(), v[:, :1].contiguous(), start)
    got, _ = run(q, one[:, :1], one[:, 1:], start)
    assert torch.equal(got, want)


@pytest.mark.parametrize("d", [128, 256])
def test_large_scores_and_a_late_maximum(d):
    q, k, v, start = inputs([900, 260], 8, 2, d, seed=5, scale=8.0)
    k[850] *= 4.0
    out, ws = run(q, k, v, start)
    assert kvq.kvq_workspace_status(ws) == 0
    # sum |q_i k_i| * sm_scale reaches 64 * 8 * 4 here: the score's part of the tolerance grows by 32
    check(out, q, k, v, start, extra=(2.0 ** -8 + 2 * 32e-3) / (2.0 ** -7 * 0.8))


def test_bad_sequences_are_skipped_and_reported():
    q, k, v, start = inputs([50, 60, 70], 8, 2, 128, seed=1)
    for bad, skipped in (([0, 50, 40, 180], (1,)), ([0, 50, 110, 181], (2,)), ([-1, 50, 110, 180], (0,))):
        out, ws = run(q, k, v, bad)
        assert kvq.kvq_workspace_status(ws) == -1
        if bad[2] == 40:   # the last sequence then starts inside the first: rows 40 .. 179 are its own
            assert torch.isfinite(out).all()
        else:
            check(out, q, k, v, start, skipped=skipped)
    out, ws = run(q, k, v, [0, 0, 0, 0])
    assert kvq.kvq_workspace_status(ws) == 0 and torch.isnan(out).all()


def test_a_captured_call_replays_with_new_contents():
    q, k, v, start = inputs([300, 40, 900], 16, 8, 128, seed=8)
    ds = torch.tensor(start, dtype=torch.int32).cuda()
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    ws = kvq.alloc_prompt_workspace()
    kvq.kvq_prompt(q, k, v, ds, out, ws, sm_scale=128 ** -0.5)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kvq.kvq_prompt(q, k, v, ds, out, ws, sm_scale=128 ** -0.5)
    for lens in ([300, 40, 900], [1000, 0, 240], [1, 1238, 1]):
        q2, k2, v2, start = inputs(lens, 16, 8, 128, seed=lens[0])
        for x, y in ((q, q2), (k, k2), (v, v2)):
            x.copy_(y)
        ds.copy_(torch.tensor(start, dtype=torch.int32))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        check(out, q, k, v, start)


def test_a_prompt_then_a_decode_over_its_stored_rows():
    """Prompt attention, the store of the same rows, and the next token's decode: the decode of the prompt's last query
    over the stored cache is the prompt attention's last row up to the cache's 8 bits."""
    lens, hq, hkv, d = [100, 33], 8, 2, 128
    q, k, v, start = inputs(lens, hq, hkv, d, seed=11)
    out, _ = run(q, k, v, start)
    L = kvq.Layout(16, 16, hkv, d, d)
    codes, scales = kvq.alloc_pool(L)
    table = torch.full((2, 8), -1, dtype=torch.int32)
    table[0, :7], table[1, :3] = torch.arange(7, dtype=torch.int32), torch.arange(7, 10, dtype=torch.int32)
    slots = torch.cat([torch.arange(100), 7 * 16 + torch.arange(33)]).cuda()
    kvq.kvq_store(codes, scales, k, v, slots, L, "q8_0")
    last = torch.tensor([99, 132]).cuda()
    od = torch.empty(2, hq, d, dtype=torch.float32, device="cuda")
    kvq.kvq_decode(q[last].contiguous(), codes, scales, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), od,
                   kvq.alloc_workspace(L, 2, hq, 8), L, "q8_0", d ** -0.5)
    # q8_0 keeps an element to 1 / 254 of its block's largest (about 4 in v): 0.016, and scores to about 0.03
    assert (od - out[last]).abs().max() < 0.016 + 2 * 0.03 * 1.0 + 2.0 ** -7 * 6
