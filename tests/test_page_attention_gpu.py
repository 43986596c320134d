"""kvq_decode and kvq_extend over a cache with a scale per page (fp8_e4m3_page) against the definition in 64 bits.

Tolerance, relative to sum_t p_t |v_t| of the row: K, V and q enter exactly; P is rounded to fp16, at most 2^-11 of each p;
q.k in fp32 sums (256 products at most, sum |q_i k_i| * sm_scale below 64 here) is off by less than 64 * 256 * 2^-24 =
1e-3 in the worst order, which changes p and the normaliser by as much each: 2^-11 + 2e-3 < 2.5e-3.  That is far above what
occurs, so the mean over all outputs is held to 2^-11.  A bf16 output adds its own rounding, 2^-8 of the value."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

import append_model as M

pytestmark = pytest.mark.gpu
KIND = "fp8_e4m3_page"
HEADS = [(8, 2, 128), (16, 8, 128), (5, 5, 128), (10, 2, 128), (32, 8, 64), (7, 7, 64), (16, 2, 256), (3, 1, 256),
         (40, 2, 128), (17, 1, 64)]


def pool(lens, hq, hkv, d, seed=0, spread=0.5, room=0):
    """Codes and scales as an append leaves them, pages apart by powers of two; rows behind a sequence's end and pages of no
    sequence hold NaN codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // 16) for x in lens]
    n = sum(need) + 5
    x = torch.randn(n, 2, hkv, 16, d, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(n, 2, hkv, 1, 1, generator=g, device="cuda"))
    m, e = torch.frexp(x.abs().amax((-1, -2)))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    scales = torch.pow(2.0, e.double()).float()
    codes = (x / scales[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need) + room)), -1, dtype=torch.int32, device="cuda")
    at = 0
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    for b, p in enumerate(need):
        table[b, :p] = order[at:at + p]
        used[order[at:at + p].long()] = True
        if lens[b] % 16:
            codes[int(order[at + p - 1]), :, :, lens[b] % 16:] = 0x7F
        at += p
    codes[~used] = 0xFF
    scales[~used] = float("nan")
    return kvq.Layout(n, 16, hkv, d, d), codes, scales, table, g


def queries(rows, hq, d, g, scale=1.0):
    return (torch.randn(rows, hq, d, generator=g, device="cuda") * scale).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def decode(q, p, lens, scale, dtype=torch.float32, status=0):
    layout, codes, scales, table, g = p
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ws = kvq.alloc_workspace(layout, len(lens), q.shape[1], table.shape[1], kind=KIND)
    ws.fill_(0x5A)
    kvq.kvq_decode(q, codes, scales, table, ints(lens), out, ws, layout, KIND, scale)
    assert kvq.kvq_workspace_status(ws) == status
    return out


def extend(q, p, lens, start, scale, dtype=torch.float32, status=0):
    layout, codes, scales, table, g = p
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ws = kvq.alloc_extend_workspace("cuda", layout, q.shape[0], q.shape[1], table.shape[1], kind=KIND, batch=len(lens))
    ws.fill_(0x5A)
    kvq.kvq_extend(q, codes, scales, table, ints(lens), ints(start), out, ws, layout, KIND, scale)
    assert kvq.kvq_workspace_status(ws) == status
    return out


def check(out, q, p, lens, start, scale):
    layout, codes, scales, table, g = p
    codes = torch.where((codes & 0x7F) == 0x7F, 0, codes)  # (no code that counts is NaN)
    ref, mag = M.attend64(q, codes, torch.nan_to_num(scales), table, lens, start, scale,
                          torch.full(q.shape, float("nan"), dtype=torch.float64, device="cuda"))
    covered = ~torch.isnan(ref).flatten(1).any(1)
    if start is None:  # sequences without tokens give zeros
        empty = torch.tensor([x <= 0 for x in lens], device="cuda")
        ref[empty] = 0
        covered |= empty
    assert torch.isnan(out[~covered]).all(), "rows that no sequence covers were written"
    got, ref, mag = out[covered].double(), ref[covered], mag[covered]
    assert torch.isfinite(got).all()
    bound, mean = 2.5e-3 * mag + 1e-9, 2.0 ** -11 * mag.mean() + 1e-9
    if out.dtype == torch.bfloat16:
        bound, mean = bound + 2.0 ** -8 * (ref.abs() + bound), mean + 2.0 ** -8 * ref.abs().mean()
    err = (got - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())
    assert err.numel() == 0 or err.mean() <= mean, (float(err.mean()), float(mean))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [16], [17, 0, 300, 31, 1, 128, 129], [2000, 5], [4097]])
def test_decode(lens, hq, hkv, d):
    p = pool(lens, hq, hkv, d, seed=len(lens), room=2)
    q = queries(len(lens), hq, d, p[4])
    for dtype in (torch.float32, torch.bfloat16):
        check(decode(q, p, lens, d ** -0.5, dtype), q, p, lens, None, d ** -0.5)


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("old,new", [([0], [1]), ([5, 100, 0, 0, 16], [3, 1, 0, 40, 16]), ([700, 15], [200, 129]),
                                     ([33] * 9, [7] * 9), ([0, 0], [300, 127])])
def test_extend(old, new, hq, hkv, d):
    lens = [a + b for a, b in zip(old, new)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    p = pool(lens, hq, hkv, d, seed=len(lens), room=1)
    q = queries(start[-1] + 3, hq, d, p[4])
    for dtype in (torch.float32, torch.bfloat16):
        check(extend(q, p, lens, start, d ** -0.5, dtype), q, p, lens, start, d ** -0.5)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 256), (32, 8, 64), (40, 2, 128)])
def test_many_sequences_and_long_ones(hq, hkv, d):
    """Runs that begin and end inside sequences, many short tiles in one CTA, and tiles over many CTAs."""
    for lens in ([20000], [30] * 300, [9000, 1, 1, 5000, 16, 40, 7000, 333]):
        p = pool(lens, hq, hkv, d, seed=7)
        q = queries(len(lens), hq, d, p[4])
        check(decode(q, p, lens, d ** -0.5), q, p, lens, None, d ** -0.5)
        new = [min(x, 1 + 13 * i % 50) for i, x in enumerate(lens)]
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        q = queries(start[-1], hq, d, p[4])
        check(extend(q, p, lens, start, d ** -0.5), q, p, lens, start, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_pages(d):
    lens = [400, 48, 100, 33]
    p = pool(lens, 8, 2, d, seed=3)
    table = p[3]
    table[0, ::3] = -1
    table[1] = -1
    table[2, :-1] = -1
    table[3, 2] = -1
    q = queries(4, 8, d, p[4])
    out = decode(q, p, lens, d ** -0.5)
    check(out, q, p, lens, None, d ** -0.5)
    assert (out[1] == 0).all()
    start = [0, 50, 60, 100, 120]
    q = queries(120, 8, d, p[4])
    out = extend(q, p, lens, start, d ** -0.5)
    check(out, q, p, lens, start, d ** -0.5)
    assert (out[50:60] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_far_apart_in_size(d):
    """Scales from 2^-32 to 2^32 beside one another: a page of huge V with hardly any weight, pages of tiny V with most."""
    lens = [500, 64]
    p = pool(lens, 8, 2, d, seed=4)
    layout, codes, scales, table, g = p
    used = torch.unique(table[table >= 0]).long()
    e = torch.randint(-32, 33, (used.numel(), layout.num_kv_heads), generator=g, device="cuda").double()
    scales[used, 1] = torch.pow(2.0, e).float()
    scales[used, 0] = torch.pow(2.0, (e % 5) - 12).float()
    q = queries(2, 8, d, g)
    check(decode(q, p, lens, d ** -0.5), q, p, lens, None, d ** -0.5)
    start = [0, 200, 232]
    q = queries(232, 8, d, g)
    check(extend(q, p, lens, start, d ** -0.5), q, p, lens, start, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_maxima_that_come_late_and_queries_of_every_size(d):
    """Scores that rise along the sequence (the reference moves again and again), q rows of zeros, of one huge element, and
    of sizes from 2^-60 to 2^60 with the scale to match."""
    lens = [900]
    p = pool(lens, 8, 2, d, seed=5, spread=0.0)
    layout, codes, scales, table, g = p
    for i, page in enumerate(table[0, :57].tolist()):
        scales[page, 0] *= 2.0 ** (i // 8 - 5)
    q = queries(1, 8, d, g)
    q[0, 1] = 0
    q[0, 2] = 0
    q[0, 2, 5] = 2.0
    check(decode(q, p, lens, d ** -0.5), q, p, lens, None, d ** -0.5)
    for f in (2.0 ** -60, 2.0 ** 60):
        big = (q.float() * f).to(torch.bfloat16)
        check(decode(big, p, lens, d ** -0.5 / f), big, p, lens, None, d ** -0.5 / f)
    check(decode(q, p, lens, -d ** -0.5), q, p, lens, None, -d ** -0.5)  # (the decode takes any finite scale)
    start = [0, 300]
    q = queries(300, 8, d, g)
    check(extend(q, p, lens, start, d ** -0.5), q, p, lens, start, d ** -0.5)


def test_a_long_even_context_loses_nothing():
    """One token far above 40000 equal ones that outweigh it together: probabilities of 2^-17 of the largest."""
    d, lens = 128, [40000]
    p = pool(lens, 4, 1, d, seed=6)
    layout, codes, scales, table, g = p
    codes[:, 0] = 0
    first = int(table[0, 0])
    codes[first, 0, 0, 0, 0] = 0x38  # 1.0
    scales[:, 0] = 1.0
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16, device="cuda")
    q[0, :, 0] = torch.tensor([8.0, 10.0, 11.0, 12.0])
    check(decode(q, p, lens, 1.0), q, p, lens, None, 1.0)
    check(extend(q, p, lens, [0, 1], 1.0), q, p, lens, [0, 1], 1.0)


def test_bad_pages_and_bad_sequences():
    d = 128
    lens = [100, 60, 80]
    p = pool(lens, 8, 2, d, seed=8)
    p[3][1, 1] = p[0].num_pages
    q = queries(3, 8, d, p[4])
    check(decode(q, p, lens, d ** -0.5, status=-1), q, p, lens, None, d ** -0.5)
    p = pool(lens, 8, 2, d, seed=9)
    q = queries(150, 8, d, p[4])
    start = [0, 20, 90, 110]  # sequence 1: more new tokens than stored ones
    check(extend(q, p, lens, start, d ** -0.5, status=-1), q, p, lens, start, d ** -0.5)
    start = [0, 20, 30, 151]  # sequence 2: past the rows
    out = extend(q, p, lens, start, d ** -0.5, status=-1)
    check(out, q, p, lens[:2], start[:3], d ** -0.5)


def test_same_results_each_time_and_on_any_stream():
    lens, d = [5000, 300, 77], 128
    p = pool(lens, 16, 8, d, seed=10)
    q = queries(3, 16, d, p[4])
    want = decode(q, p, lens, d ** -0.5)
    for _ in range(3):
        assert torch.equal(decode(q, p, lens, d ** -0.5), want)
    layout, codes, scales, table, g = p
    ws = kvq.alloc_workspace(layout, 3, 16, table.shape[1], kind=KIND)
    out, sl = torch.empty_like(want), ints(lens)
    call = lambda: kvq.kvq_decode(q, codes, scales, table, sl, out, ws, layout, KIND, d ** -0.5)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_without_a_workspace():
    lens, d = [3000, 1, 200], 256
    p = pool(lens, 16, 2, d, seed=11)
    layout, codes, scales, table, g = p
    q = queries(3, 16, d, g)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    kvq.kvq_decode_noalloc(q, codes, scales, table, ints(lens), out, layout, KIND, d ** -0.5)
    assert kvq.kvq_noalloc_status() == 0
    check(out, q, p, lens, None, d ** -0.5)


def test_offsets_past_32_bits():
    """Pages near the end of a pool of more than 2^32 codes."""
    d, hkv, lens = 256, 2, [1000, 40]
    per_page = 2 * hkv * 16 * d
    n = (1 << 32) // per_page + 4096
    small = pool(lens, 8, hkv, d, seed=12)
    layout = kvq.Layout(n, 16, hkv, d, d)
    codes, scales = kvq.alloc_pool(layout, kind=KIND)
    k = small[1].shape[0]
    codes[n - k:] = small[1]
    scales[n - k:] = small[2]
    table = torch.where(small[3] >= 0, small[3] + (n - k), -1)
    big = (layout, codes, scales, table, small[4])
    q = queries(2, 8, d, small[4])
    assert torch.equal(decode(q, big, lens, d ** -0.5), decode(q, small, lens, d ** -0.5))
    start = [0, 600, 620]
    q = queries(620, 8, d, small[4])
    assert torch.equal(extend(q, big, lens, start, d ** -0.5), extend(q, small, lens, start, d ** -0.5))
