"""Page operations of the cache on the GPU against a plain host model: every table entry, length, count, copy
list and pool byte equal.  Covers lists in any order, parents replaced by their children, lengths of 0, whole
and partly filled last pages, masked pages, pools of several 8192-page chunks, too few free pages, bad lists,
every pool kind, odd layouts, two streams and a captured graph."""
import random

import numpy as np
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from pages_model import PAGE, Model, pages

pytestmark = pytest.mark.gpu

LAYOUTS = {"gqa128": (8, 128, 128, False), "gqa256": (2, 256, 256, False), "d64": (3, 64, 64, False),
           "d32": (1, 32, 32, False), "mla": (1, 576, 512, True)}


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def layout(key, num_pages):
    h, d, dv, mla = LAYOUTS[key]
    return kvq.Layout(num_pages, PAGE, h, d, dv, mla)


def pool(L, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, L.codes_shape(), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(-32768, 32768, L.scales_shape(), generator=g, dtype=torch.int16, device="cuda")
    return codes, (None if "unscaled" in kind else scales)


def tables(r, num_pages, lens, room, masked=0.0):
    order = list(range(num_pages))
    r.shuffle(order)
    t, refs = np.full((len(lens), room), -1, np.int32), np.zeros(num_pages, np.int32)
    for b, x in enumerate(lens):
        for c in range(pages(x)):
            p = order.pop()
            if r.random() >= masked:
                t[b, c] = p
                refs[p] += 1
    return t, refs


def same(model, table, lens, refs):
    assert np.array_equal(table.cpu().numpy(), model.table)
    assert np.array_equal(lens.cpu().numpy(), model.lens)
    assert np.array_equal(refs.cpu().numpy(), model.refs)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled"])
@pytest.mark.parametrize("key", list(LAYOUTS))
def test_copies_of_pages(key, kind):
    r = random.Random(key + kind)
    L = layout(key, 97)
    codes, scales = pool(L, kind, 1)
    m = Model([], [], [], [codes.cpu().numpy()] + ([] if scales is None else [scales.cpu().numpy()]))
    order = list(range(97))
    r.shuffle(order)
    for n in (1, 3, 40):
        dst, src = order[:n], [r.choice(order[n:]) for _ in range(n)]     # one page may feed many
        src[0], dst[n // 2] = (-1, dst[n // 2]) if n > 1 else (src[0], dst[0])
        kvq.kvq_pages_copy(codes, scales, dev(src), dev(dst), L, kind)
        m.copy(src, dst)
        # pairs outside the pool are skipped
        kvq.kvq_pages_copy(codes, scales, dev([97, 0, -5]), dev([0, 97, 1]), L, kind)
        assert np.array_equal(codes.cpu().numpy(), m.pools[0])
        assert scales is None or np.array_equal(scales.cpu().numpy(), m.pools[1])
    kvq.kvq_pages_copy(codes, scales, dev([]), dev([]), L, kind)
    assert np.array_equal(codes.cpu().numpy(), m.pools[0])


def _fork(model, L, src, dst, table, lens, refs, ws):
    cs, cd = torch.full((len(src),), 77, dtype=torch.int32).cuda(), torch.full((len(src),), 77, dtype=torch.int32).cuda()
    kvq.kvq_pages_fork(table, lens, refs, dev(src), dev(dst), cs, cd, ws, L)
    return cs, cd


@pytest.mark.parametrize("num_pages", [300, 8192, 20011])
@pytest.mark.parametrize("masked", [0.0, 0.2])
@pytest.mark.parametrize("seed", range(4))
def test_forks_follow_the_model(seed, masked, num_pages):
    r = random.Random(seed * 7 + num_pages)
    B = 12
    lens = [r.choice([0, 1, 15, 16, 17, 32, 100, r.randrange(160)]) for _ in range(B)]
    if num_pages > 300:
        lens[3] = 2500 * PAGE + r.choice([0, 5])
    room = max(pages(x) for x in lens) + 3
    t, refs = tables(r, num_pages, lens, room, masked)
    L = layout("d32", num_pages)
    m = Model(t, lens, refs)
    table, dl, dr = dev(t), dev(lens), dev(refs)
    ws = kvq.alloc_pages_workspace(L, B, room)
    for step in range(6):
        n = [B, 1, 5, B, 7, 3][step]
        dst = r.sample(range(B), n)
        if step == 3:
            dst = list(range(B))
        # keep the one long row from being multiplied past the pool
        src = [r.choice([x for x in range(B) if m.lens[x] < 1000] or [0]) for _ in range(n)]
        ws.fill_(0x5A)
        cs, cd = _fork(m, L, src, dst, table, dl, dr, ws)
        want = m.fork(src, dst)
        assert want is not None
        assert kvq.kvq_workspace_status(ws) == 0
        assert (cs.cpu().tolist(), cd.cpu().tolist()) == want
        same(m, table, dl, dr)


def test_a_long_row_is_shared_and_released():
    num_pages, room = 20000, 6000
    lens = [5000 * PAGE + 3, 40, 0, 17]
    r = random.Random(5)
    t, refs = tables(r, num_pages, lens, room)
    L = layout("d32", num_pages)
    m = Model(t, lens, refs)
    table, dl, dr = dev(t), dev(lens), dev(refs)
    ws = kvq.alloc_pages_workspace(L, 4, room)
    for src, dst in (([0, 0, 0], [1, 2, 3]), ([1, 1, 3, 0], [0, 1, 2, 3]), ([2], [0])):
        cs, cd = _fork(m, L, src, dst, table, dl, dr, ws)
        assert (cs.cpu().tolist(), cd.cpu().tolist()) == m.fork(src, dst)
        same(m, table, dl, dr)
    for new in ([0, 5, 90000, 17], [4096 * PAGE, 0, 0, 0], [0, 0, 0, 0]):
        kvq.kvq_pages_resize(table, dl, dr, dev([2, 0, 3, 1]), dev(new), ws, L)
        assert m.resize([2, 0, 3, 1], new)
        same(m, table, dl, dr)
    assert int(dr.sum()) == 0


@pytest.mark.parametrize("num_pages", [257, 8193, 16384])
@pytest.mark.parametrize("seed", range(4))
def test_resizes_follow_the_model(seed, num_pages):
    r = random.Random(seed + num_pages)
    B, top = 9, num_pages * PAGE // 9
    lens = [r.choice([0, 1, 16, r.randrange(top // 2)]) for _ in range(B)]
    room = pages(top) + 1
    t, refs = tables(r, num_pages, lens, room, 0.1)
    L = layout("d32", num_pages)
    m = Model(t, lens, refs)
    table, dl, dr = dev(t), dev(lens), dev(refs)
    ws = kvq.alloc_pages_workspace(L, B, room)
    for _ in range(6):
        seqs = r.sample(range(B), r.randrange(1, B + 1))
        new = [r.choice([0, 1, 16, 17, int(m.lens[s]), r.randrange(top)]) for s in seqs]
        kvq.kvq_pages_resize(table, dl, dr, dev(seqs), dev(new), ws, L)
        assert kvq.kvq_workspace_status(ws) == 0
        assert m.resize(seqs, new)
        same(m, table, dl, dr)


def test_too_few_free_pages_and_bad_lists_change_nothing():
    L = layout("d32", 10)
    lens = [40, 50, 0]  # 3 + 4 pages
    t, refs = tables(random.Random(1), 10, lens, 8)
    m = Model(t, lens, refs)
    table, dl, dr = dev(t), dev(lens), dev(refs)
    ws = kvq.alloc_pages_workspace(L, 4, 8)
    kvq.kvq_pages_resize(table, dl, dr, dev([2, 0]), dev([49, 16]), ws, L)   # 4 of 3 free; row 0's come later
    assert kvq.kvq_workspace_status(ws) == -10
    same(m, table, dl, dr)
    kvq.kvq_pages_resize(table, dl, dr, dev([2]), dev([48]), ws, L)
    assert kvq.kvq_workspace_status(ws) == 0 and m.resize([2], [48])
    same(m, table, dl, dr)
    cs, cd = _fork(m, L, [0, 1], [1, 2], table, dl, dr, ws)                  # one copy, no page left
    assert kvq.kvq_workspace_status(ws) == -10
    assert cs.cpu().tolist() == cd.cpu().tolist() == [-1, -1]
    same(m, table, dl, dr)
    for seqs, new in (([0, 0], [1, 1]), ([3], [1]), ([-1], [1]), ([0], [-1]), ([0], [8 * PAGE + 1])):
        kvq.kvq_pages_resize(table, dl, dr, dev(seqs), dev(new), ws, L)
        assert kvq.kvq_workspace_status(ws) == -1
        same(m, table, dl, dr)
    for src, dst in (([0, 1], [2, 2]), ([3], [0]), ([0], [3]), ([0], [-1])):
        cs, cd = _fork(m, L, src, dst, table, dl, dr, ws)
        assert kvq.kvq_workspace_status(ws) == -1
        assert set(cs.cpu().tolist() + cd.cpu().tolist()) == {-1}
        same(m, table, dl, dr)
    kvq.kvq_pages_resize(table, dl, dr, dev([]), dev([]), ws, L)
    assert kvq.kvq_workspace_status(ws) == 0
    # a page that nobody counted is reported and its count stays 0
    dr.zero_()
    kvq.kvq_pages_resize(table, dl, dr, dev([0]), dev([0]), ws, L)
    assert kvq.kvq_workspace_status(ws) == -1 and int(dr.abs().sum()) == 0


def test_a_row_cut_back_into_a_shared_page_gets_its_own_before_it_grows():
    """Two full pages shared by a fork, one row cut back to 20 tokens: growing it would write into the other row's
    page and is refused; a fork onto itself copies that page, and then it grows."""
    L = layout("d32", 12)
    t, refs = tables(random.Random(1), 12, [32, 0], 8)
    codes, scales = pool(L, "q8_0", 5)
    m = Model(t, [32, 0], refs, [codes.cpu().numpy(), scales.cpu().numpy()])
    table, dl, dr = dev(t), dev([32, 0]), dev(refs)
    ws = kvq.alloc_pages_workspace(L, 2, 8)
    cs, cd = _fork(m, L, [0], [1], table, dl, dr, ws)
    assert (cs.cpu().tolist(), cd.cpu().tolist()) == m.fork([0], [1]) == ([-1], [-1])
    kvq.kvq_pages_resize(table, dl, dr, dev([0]), dev([20]), ws, L)
    assert kvq.kvq_workspace_status(ws) == 0 and m.resize([0], [20])
    same(m, table, dl, dr)
    for grown in (21, 40):
        kvq.kvq_pages_resize(table, dl, dr, dev([0]), dev([grown]), ws, L)
        assert kvq.kvq_workspace_status(ws) == -1
        same(m, table, dl, dr)
    cs, cd = _fork(m, L, [0], [0], table, dl, dr, ws)
    want = m.fork([0], [0])
    assert (cs.cpu().tolist(), cd.cpu().tolist()) == want and want[0][0] >= 0
    kvq.kvq_pages_copy(codes, scales, cs, cd, L, "q8_0")
    m.copy(*want)
    same(m, table, dl, dr)
    assert np.array_equal(codes.cpu().numpy(), m.pools[0]) and np.array_equal(scales.cpu().numpy(), m.pools[1])
    kvq.kvq_pages_resize(table, dl, dr, dev([0]), dev([40]), ws, L)
    assert kvq.kvq_workspace_status(ws) == 0 and m.resize([0], [40])
    same(m, table, dl, dr)


def test_new_lengths_may_be_the_lengths_themselves():
    L = layout("d32", 10)
    t, refs = tables(random.Random(1), 10, [40, 50], 8)
    m = Model(t, [40, 50], refs)
    table, dl, dr = dev(t), dev([40, 50]), dev(refs)
    ws = kvq.alloc_pages_workspace(L, 2, 8)
    kvq.kvq_pages_resize(table, dl, dr, dev([0, 1]), dl, ws, L)
    assert kvq.kvq_workspace_status(ws) == 0
    same(m, table, dl, dr)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e5m2_unscaled"])
@pytest.mark.parametrize("key", list(LAYOUTS))
@pytest.mark.parametrize("words", [1, 2, 4])
def test_compaction_follows_the_model(words, key, kind):
    r = random.Random(key + kind + str(words))
    drafted = [0, 1, 2, 17, 63, 64, 64 * words, 33]
    drafted = [min(n, 64 * words) for n in drafted]
    ctx = [5, 0, 31, 16, 100, 7, 40, 15]
    lens = [c + n for c, n in zip(ctx, drafted)]
    num_pages, room = sum(pages(x) for x in lens) + 5, max(pages(x) for x in lens)
    t, refs = tables(r, num_pages, lens, room)
    L = layout(key, num_pages)
    codes, scales = pool(L, kind, 3)
    m = Model(t, lens, refs, [codes.cpu().numpy()] + ([] if scales is None else [scales.cpu().numpy()]))
    kept = [[j for j in range(n) if r.random() < p] for n, p in zip(drafted, [.5, 1, .5, .3, .9, .1, .5, 0])]
    kept[2] = [1] if drafted[2] > 1 else kept[2]
    keep = np.zeros((8, words), np.uint64)
    for b, k in enumerate(kept):
        for j in k:
            keep[b, j // 64] |= np.uint64(1 << (j % 64))
        for j in range(drafted[b], 64 * words):      # bits behind the drafted tokens say nothing
            keep[b, j // 64] |= np.uint64(1 << (j % 64))
    new = torch.full((8,), -7, dtype=torch.int32).cuda()
    ws = torch.full((256,), 0x5A, dtype=torch.uint8).cuda()
    start = np.concatenate([[0], np.cumsum(drafted)])
    kvq.kvq_pages_compact(codes, scales, dev(t), dev(lens), dev(start), torch.from_numpy(keep.view(np.int64)).cuda(), new,
                          ws, L, kind, page_refs=dev(refs))
    want = [m.compact(b, drafted[b], kept[b]) for b in range(8)]
    assert kvq.kvq_workspace_status(ws) == 0
    assert new.cpu().tolist() == want
    assert np.array_equal(codes.cpu().numpy(), m.pools[0])
    assert scales is None or np.array_equal(scales.cpu().numpy(), m.pools[1])


def test_compaction_leaves_what_it_cannot_move():
    """Shared, masked and foreign pages and inconsistent numbers: those sequences stay, the others are compacted."""
    L = layout("gqa128", 40)
    lens, drafted = [40, 40, 40, 40, 40], [10, 10, 10, 10, 41]
    t, refs = tables(random.Random(2), 40, lens, 3)
    refs[t[0, 1]] += 1            # tokens 30, 31 of row 0 lie in a page that another row holds
    t[1, 2] = -1
    t[2, 2] = 40
    codes, scales = pool(L, "fp8_e4m3", 3)
    m = Model(t, lens, refs, [codes.cpu().numpy(), scales.cpu().numpy()])
    keep = torch.full((5, 1), 0b1010000010, dtype=torch.int64).cuda()
    new = torch.zeros(5, dtype=torch.int32).cuda()
    ws = torch.empty(256, dtype=torch.uint8).cuda()
    start = np.concatenate([[0], np.cumsum(drafted)])
    args = (codes, scales, dev(t), dev(lens), dev(start), keep, new, ws, L, "fp8_e4m3")
    kvq.kvq_pages_compact(*args, page_refs=dev(refs))
    assert kvq.kvq_workspace_status(ws) == -1
    m.compact(3, 10, [1, 7, 9])
    assert new.cpu().tolist() == [40, 40, 40, 33, 40]
    assert np.array_equal(codes.cpu().numpy(), m.pools[0]) and np.array_equal(scales.cpu().numpy(), m.pools[1])


def test_a_captured_speculative_step_replays_on_another_stream():
    """grow, compact, shrink captured once and replayed: every replay gives what the model gives."""
    L = layout("gqa128", 64)
    ctx, n = [37, 100, 16], [9, 4, 30]
    t, refs = tables(random.Random(4), 64, ctx, 12)
    codes, scales = pool(L, "q8_0", 9)
    m = Model(t, ctx, refs, [codes.cpu().numpy(), scales.cpu().numpy()])
    table, dl, dr = dev(t), dev(ctx), dev(refs)
    kept = [[0, 3, 8], [1], list(range(5, 30, 3))]
    keep = torch.tensor([[sum(1 << j for j in k)] for k in kept], dtype=torch.int64).cuda()
    new = torch.zeros(3, dtype=torch.int32).cuda()
    seqs, grown = dev([0, 1, 2]), dev([a + b for a, b in zip(ctx, n)])
    start = dev(np.concatenate([[0], np.cumsum(n)]))
    ws = kvq.alloc_pages_workspace(L, 3, 12)
    torch.cuda.synchronize()

    def step():
        kvq.kvq_pages_resize(table, dl, dr, seqs, grown, ws, L)
        kvq.kvq_pages_compact(codes, scales, table, dl, start, keep, new, ws, L, "q8_0", page_refs=dr)
        kvq.kvq_pages_resize(table, dl, dr, seqs, new, ws, L)

    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        assert m.resize([0, 1, 2], [a + b for a, b in zip(ctx, n)])
        left = [m.compact(b, n[b], kept[b]) for b in range(3)]
        assert m.resize([0, 1, 2], left)
        s.synchronize()
        assert kvq.kvq_workspace_status(ws) == 0
        assert new.cpu().tolist() == left
        same(m, table, dl, dr)
        assert np.array_equal(codes.cpu().numpy(), m.pools[0]) and np.array_equal(scales.cpu().numpy(), m.pools[1])
