"""kvq_tree on the GPU against the definition in 64 bits.

Tolerances, relative to sum_t p_t |V_t| of the row (the reference gives it).  On the tensor cores P is rounded to bf16,
at most 2^-8 of each p; a share of the exponentials comes from a cubic with 1.5e-4; q.K in fp32 (at most 256 products,
sum |q_i k_i| below 64 here) is off by less than 64 * 256 * 2^-24 = 1e-3 in the worst order, and a rounding of the
score by e changes p by e.  Numerator and normaliser both carry the last two: 2^-8 + 2 * (1.5e-4 + 1e-3) < 2^-7 * 0.8.
On the CUDA cores P stays fp32: 2 * 1e-3 (MLA: 576 products, 2.2e-3 each) < 2^-7.8.  The bounds of the worst order
are far above what occurs, so the mean over all outputs is held to a quarter of 2^-8.  A bf16 output adds its own rounding, 2^-8 of
the value."""
import random

import numpy as np
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from plain64 import tree64

pytestmark = pytest.mark.gpu
PAGE = 16


def masks(r, n, words, kind="tree"):
    rows = []
    for i in range(n):
        if kind == "chain":
            m = (1 << (i + 1)) - 1
        elif kind == "any":
            m = r.getrandbits(64 * words)
        else:
            p = r.randint(-1, i - 1)
            m = (rows[p] if p >= 0 else 0) | 1 << i
        rows.append(m)
    return rows


def as_words(rows, words):
    x = np.array([[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for m in rows], np.uint64).reshape(-1, words)
    return torch.from_numpy(x.view(np.int64)).cuda()


class Case:
    def __init__(self, hq, hkv, d, kind, ctx, drafted, words=1, mla=False, masked=0.0, mask="tree", seed=0, behind=3,
                 spare=4):
        r = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.words, self.mla = kind, words, mla
        self.hq, self.v_dim = hq, 512 if mla else d
        self.lens = [c + n for c, n in zip(ctx, drafted)]
        self.start = [0] + list(np.cumsum(drafted))
        self.total = self.start[-1] + behind                    # rows behind the last sequence
        need = sum(-(-x // PAGE) for x in self.lens)
        self.L = kvq.Layout(need + spare, PAGE, hkv, d, self.v_dim, mla)
        room = max(1, max(-(-x // PAGE) for x in self.lens)) + 2
        order = list(range(need + spare))
        r.shuffle(order)
        t = np.full((len(ctx), room), -1, np.int32)
        for b, x in enumerate(self.lens):
            for c in range(-(-x // PAGE)):
                p = order.pop()
                t[b, c] = p if r.random() >= masked else -1
            for c in range(-(-x // PAGE), room):                # entries behind the sequence are never read
                t[b, c] = 1 << 30
        self.table = torch.from_numpy(t).cuda()
        self.codes, self.scales = kvq.alloc_pool(self.L)
        self.codes.fill_(0x7F)                                  # NaN codes wherever nothing is stored
        self.scales.fill_(0x7C00)                               # infinite scales
        slots, rows = [], sum(self.lens)
        for b, x in enumerate(self.lens):
            slots += [int(t[b, i // PAGE]) * PAGE + i % PAGE if t[b, i // PAGE] >= 0 else -1 for i in range(x)]
        k = torch.randn(rows, hkv, d, generator=g, device="cuda") * torch.exp(
            0.5 * torch.randn(hkv, d, generator=g, device="cuda"))
        v = torch.randn(rows, hkv, d, generator=g, device="cuda")
        slots = torch.tensor(slots, dtype=torch.int64).cuda()
        k, v = k.to(torch.bfloat16), None if mla else v.to(torch.bfloat16)
        if "unscaled" in kind:
            kvq.kvq_store_unscaled(self.codes, k, v, slots, self.L, kind)
            self.scales = None
        else:
            kvq.kvq_store(self.codes, self.scales, k, v, slots, self.L, kind)
        self.q = (torch.randn(self.total, hq, d, generator=g, device="cuda") / d ** 0.5).to(torch.bfloat16)
        self.mask = as_words([m for n in drafted for m in masks(r, n, words, mask)] + [0] * behind, words)
        self.dl = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.ds = torch.tensor(self.start, dtype=torch.int32).cuda()

    def run(self, path=0, dtype=torch.float32, ws=None):
        out = torch.full((self.total, self.hq, self.v_dim), float("nan"), dtype=dtype, device="cuda")
        if ws is None:
            ws = kvq.alloc_tree_workspace(self.L, len(self.lens), self.total, self.hq, self.table.shape[1], path)
            ws.fill_(0x5A)
        kvq.kvq_tree(self.q, self.codes, self.scales, self.table, self.dl, self.ds, self.mask, out, ws, self.L, self.kind,
                     1.0, path)
        return out, ws

    def check(self, out, dtype=torch.float32, tensor=True, skipped=()):
        ref = torch.zeros(self.total, self.hq, self.v_dim, dtype=torch.float64, device="cuda")
        ref, mag = tree64(self.q, self.codes, self.scales, self.kind, self.table, self.lens, self.start, self.mask,
                          self.v_dim, self.mla, 1.0, ref, skipped)
        covered = torch.zeros(self.total, dtype=torch.bool, device="cuda")
        for b in range(len(self.lens)):
            if b not in skipped:
                covered[self.start[b]:self.start[b + 1]] = True
        assert torch.isnan(out[~covered]).all(), "rows that no sequence covers were written"
        got, ref, mag = out[covered].double(), ref[covered], mag[covered]
        assert torch.isfinite(got).all()
        rel = 2.0 ** -7 * 0.8 if tensor else 2.0 ** -7.8
        bound = rel * mag + 1e-6
        mean = 2.0 ** -10 * mag.mean() + 1e-6
        if dtype == torch.bfloat16:
            bound, mean = bound + 2.0 ** -8 * (ref.abs() + bound), mean + 2.0 ** -8 * ref.abs().mean()
        err = (got - ref).abs()
        assert (err <= bound).all(), float((err / bound).max())
        assert err.numel() == 0 or err.mean() <= mean, (float(err.mean()), float(mean))


RAGGED = dict(ctx=[0, 5, 200, 33, 1000, 127, 1, 640], drafted=[1, 16, 0, 64, 7, 2, 33, 13])


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 8, 128), (16, 2, 256), (6, 2, 128), (12, 1, 256), (5, 5, 128),
                                      (40, 1, 128)])
def test_ragged_trees_on_the_flash_kernel(hq, hkv, d, kind):
    c = Case(hq, hkv, d, kind, seed=hq + d, **RAGGED)
    out, ws = c.run()
    assert kvq.kvq_workspace_status(ws) == 0
    c.check(out)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e5m2_unscaled"])
@pytest.mark.parametrize("hq,hkv,d,path", [(6, 2, 64, 0), (8, 8, 64, 0), (8, 2, 128, 1), (12, 4, 256, 1)])
def test_ragged_trees_on_the_cuda_cores(hq, hkv, d, path, kind):
    c = Case(hq, hkv, d, kind, seed=hq + d, **RAGGED)
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    c.check(out, tensor=False)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e4m3_unscaled"])
@pytest.mark.parametrize("hq,path", [(128, 0), (128, 1), (16, 2), (64, 2)])
def test_trees_over_latent_rows(hq, path, kind):
    c = Case(hq, 1, 576, kind, [0, 200, 33, 700], [5, 16, 0, 9], mla=True, masked=0.1, seed=hq)
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    c.check(out, tensor=path != 1)


@pytest.mark.parametrize("words", [1, 2, 3, 4])
@pytest.mark.parametrize("hq,hkv,d,path", [(8, 2, 128, 0), (16, 2, 256, 0), (4, 2, 64, 0), (8, 2, 128, 1)])
def test_any_mask_of_several_words(hq, hkv, d, path, words):
    """Masks that are no trees, up to 256 drafted tokens, masked pages, and rows whose mask leaves nothing."""
    n = 64 * words
    c = Case(hq, hkv, d, "fp8_e4m3", [0, 300, 15, 0], [n, n - 1, 17, 40], words=words, masked=0.15, mask="any", seed=words)
    c.mask[c.start[3]:c.start[3] + 20] = 0           # nothing before them either: zeros
    c.mask[c.start[0] + 3] = 0
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    assert (out[c.start[3]:c.start[3] + 20] == 0).all() and (out[c.start[0] + 3] == 0).all()
    c.check(out, tensor=path == 0 and d != 64)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 256)])
@pytest.mark.parametrize("batch,ctx,n", [(1, 20000, 8), (3, 9000, 64), (70, 600, 5), (200, 17, 3), (1, 1, 1)])
def test_splits_over_few_and_many_sequences(batch, ctx, n, hq, hkv, d):
    r = random.Random(batch)
    c = Case(hq, hkv, d, "fp8_e4m3", [r.randint(max(0, ctx // 2), ctx) for _ in range(batch)],
             [r.randint(1, n) for _ in range(batch)], seed=batch, behind=1)
    for dtype in (torch.float32, torch.bfloat16):
        out, ws = c.run(dtype=dtype)
        assert kvq.kvq_workspace_status(ws) == 0
        c.check(out, dtype)


def test_large_scores_and_a_late_maximum():
    """The running maximum moves late and far: a context of small scores, then one key that dominates."""
    c = Case(8, 2, 128, "fp8_e4m3", [3000, 700], [6, 40], seed=5)
    c.q.mul_(8.0)
    out, ws = c.run()
    assert kvq.kvq_workspace_status(ws) == 0
    ref = torch.zeros(c.total, 8, 128, dtype=torch.float64, device="cuda")
    ref, mag = tree64(c.q, c.codes, c.scales, c.kind, c.table, c.lens, c.start, c.mask, 128, False, 1.0, ref)
    n = c.start[-1]
    # scores are 8 times larger, and with them the fp32 error of q.K in the tolerance above: 2^-8 + 2 * (1.5e-4 + 8e-3)
    assert ((out[:n].double() - ref[:n]).abs() <= 0.0205 * mag[:n] + 1e-6).all()


def test_a_chain_is_what_extend_computes():
    c = Case(16, 8, 128, "q8_0", [100, 700, 0], [30, 64, 5], mask="chain", behind=0)
    out, ws = c.run()
    ref = torch.empty_like(out)
    kvq.kvq_extend(c.q, c.codes, c.scales, c.table, c.dl, c.ds, ref, kvq.alloc_extend_workspace(), c.L, c.kind)
    c.check(out)
    c.check(ref)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 2, 64)])
def test_bad_sequences_and_pages_are_skipped_and_reported(hq, hkv, d):
    for what in ("long", "words", "page", "table"):
        c = Case(hq, hkv, d, "fp8_e4m3", [50, 60, 70], [9, 20, 4], seed=3)
        skipped = ()
        if what == "long":
            c.dl[1] = 19                       # fewer tokens than drafted ones
            skipped = (1,)
        elif what == "words":                  # 65 drafted tokens in one word
            c = Case(hq, hkv, d, "fp8_e4m3", [50, 60, 70], [9, 65, 4], words=2, seed=3)
            c.mask, c.words = c.mask[:, :1].contiguous(), 1
            skipped = (1,)
        elif what == "page":
            c.table[2, 1] = c.L.num_pages
        else:
            c.dl[0] = c.table.shape[1] * PAGE + 1
            skipped = (0,)
        out, ws = c.run()
        assert kvq.kvq_workspace_status(ws) == -1, what
        c.check(out, tensor=d != 64, skipped=skipped)


def test_nothing_to_do():
    c = Case(8, 2, 128, "fp8_e4m3", [40, 20], [0, 0], behind=2)
    out, ws = c.run()
    assert kvq.kvq_workspace_status(ws) == 0 and torch.isnan(out).all()


def test_a_captured_call_replays_with_new_contents():
    c = Case(16, 2, 256, "fp8_e4m3", [400, 90, 3000], [12, 64, 3], seed=8)
    out, ws = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, _ = c.run(ws=ws)
    for k in range(3):
        c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator(device="cuda").manual_seed(k), device="cuda") / 16)
        c.mask.copy_(as_words([m for n in (12, 64, 3) for m in masks(random.Random(k), n, 1)] + [0] * 3, 1))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        c.check(out)


def test_a_speculative_step_end_to_end():
    """Grow, store the drafts, attend, compact the accepted path, release, and decode the next token: the decode
    sees exactly the accepted tokens."""
    r = random.Random(1)
    hq, hkv, d, ctx, n = 8, 2, 128, [37, 100, 16], [9, 16, 5]
    L = kvq.Layout(40, PAGE, hkv, d, d)
    codes, scales = kvq.alloc_pool(L)
    table = torch.full((3, 9), -1, dtype=torch.int32).cuda()
    lens, refs = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(40, dtype=torch.int32).cuda()
    seqs = torch.arange(3, dtype=torch.int32).cuda()
    ws = kvq.alloc_pages_workspace(L, 3, 9)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731

    def slots(lo, hi):
        return torch.cat([table[b, torch.arange(a, z).cuda() // PAGE].long() * PAGE + torch.arange(a, z).cuda() % PAGE
                          for b, (a, z) in enumerate(zip(lo, hi))])

    def rows(count):
        return [torch.randn(count, hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2)]

    torch.manual_seed(4)
    kvq.kvq_pages_resize(table, lens, refs, seqs, i32(ctx), ws, L)
    k0, v0 = rows(sum(ctx))
    kvq.kvq_store(codes, scales, k0, v0, slots([0] * 3, ctx), L, "q8_0")
    total = [a + b for a, b in zip(ctx, n)]
    kvq.kvq_pages_resize(table, lens, refs, seqs, i32(total), ws, L)
    k1, v1 = rows(sum(n))
    kvq.kvq_store(codes, scales, k1, v1, slots(ctx, total), L, "q8_0")
    tree = [masks(r, x, 1) for x in n]
    mask = as_words([m for t in tree for m in t], 1)
    start = i32([0] + list(np.cumsum(n)))
    q = (torch.randn(sum(n), hq, d, device="cuda") / d ** 0.5).to(torch.bfloat16)
    out = torch.empty(sum(n), hq, d, dtype=torch.float32, device="cuda")
    tw = kvq.alloc_tree_workspace(L, 3, sum(n), hq, 9)
    kvq.kvq_tree(q, codes, scales, table, lens, start, mask, out, tw, L, "q8_0")
    assert kvq.kvq_workspace_status(tw) == 0
    leaf = [r.randrange(x) for x in n]
    keep = torch.stack([mask[int(start[b]) + leaf[b]] for b in range(3)])
    new = torch.zeros(3, dtype=torch.int32).cuda()
    kvq.kvq_pages_compact(codes, scales, table, lens, start, keep, new, ws, L, "q8_0", page_refs=refs)
    assert kvq.kvq_workspace_status(ws) == 0
    kvq.kvq_pages_resize(table, lens, refs, seqs, new, ws, L)
    paths = [[j for j in range(n[b]) if tree[b][leaf[b]] >> j & 1] for b in range(3)]
    assert new.tolist() == [c + len(p) for c, p in zip(ctx, paths)] == lens.tolist()
    assert refs.sum().item() == sum(-(-x // PAGE) for x in lens.tolist())
    # the leaf's row of the tree attention is the decode of its query over the compacted cache
    qd = torch.stack([q[int(start[b]) + leaf[b]] for b in range(3)])
    od = torch.empty(3, hq, d, dtype=torch.float32, device="cuda")
    kvq.kvq_decode(qd, codes, scales, table, lens, od, kvq.alloc_workspace(L, 3, hq, 9), L, "q8_0")
    ot = torch.stack([out[int(start[b]) + leaf[b]] for b in range(3)])
    # both are within 2^-7 * 0.8 of sum p |V| <= max |V| < 6 of the exact value
    assert (od - ot).abs().max() <= 2 * 2.0 ** -7 * 0.8 * 6
    # and the cache is byte for byte what storing the accepted rows alone gives
    c2, s2 = kvq.alloc_pool(L)
    c2.copy_(codes)
    s2.copy_(scales)
    first = np.concatenate([[0], np.cumsum(n)])
    pick = torch.tensor([int(first[b]) + j for b in range(3) for j in paths[b]]).cuda()
    kvq.kvq_store(c2, s2, k1[pick].contiguous(), v1[pick].contiguous(), slots(ctx, new.tolist()), L, "q8_0")
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
