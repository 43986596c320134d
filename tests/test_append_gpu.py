"""kvq_append on the GPU against its definition, bit for bit: pool, scales and rotated queries (tests/append_model.py
rounds every product, sum and quotient as the definition says, so nothing may differ)."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

import append_model as M

pytestmark = pytest.mark.gpu

KINDS = ("fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled", "fp8_e4m3_page")
GQA = [(8, 2, 128), (4, 4, 64), (6, 1, 256)]


def pages(n, size=16):
    return -(-n // size)


class Cache:
    """A pool, its tables over shuffled pages, and their twins on the CPU."""

    def __init__(self, kind, hkv, d, batch, room, mla=False, size=16, seed=0, dv=None):
        self.g = torch.Generator().manual_seed(seed)
        self.kind, self.size = kind, size
        n = batch * room + 3
        self.layout = kvq.Layout(n, size, hkv, d, d if dv is None else dv, mla)
        self.codes = torch.randint(0, 256, self.layout.codes_shape(), generator=self.g, dtype=torch.int32).to(torch.uint8)
        if kind == "fp8_e4m3_page":  # (a fresh page's scale does not matter)
            self.scales = torch.full(self.layout.page_scales_shape(), float("nan"))
        else:
            self.scales = torch.randint(0, 1 << 14, self.layout.scales_shape(), generator=self.g, dtype=torch.int32).to(torch.int16)
        self.table = torch.randperm(n, generator=self.g)[:batch * room].view(batch, room).to(torch.int32)
        self.lens = [0] * batch
        self.dcodes, self.dscales, self.dtable = self.codes.cuda(), self.scales.cuda(), self.table.cuda()
        self.ws = kvq.alloc_append_workspace()

    def rows(self, t, hq, spread=1.0):
        lay = self.layout
        make = lambda h: (torch.randn(t, h, lay.head_dim, generator=self.g) * spread).to(torch.bfloat16)  # noqa: E731
        return make(hq) if hq else None, make(lay.num_kv_heads), None if lay.mla else make(lay.num_kv_heads)

    def append(self, new, q, k, v, status=0, skipped=(), place=None, start=None, lens=None, **opt):
        """new: tokens per sequence.  Both sides, compared."""
        self.lens = [x + n for x, n in zip(self.lens, new)] if lens is None else lens
        if start is None:
            start = [0]
            for n in new:
                start.append(start[-1] + n)
        angles, positions = opt.get("angles"), opt.get("positions")
        first, pairs = opt.get("first", 0), opt.get("pairs", False)
        dq = dk = dv = dout = None
        put = place or (lambda x: x)
        dk, dv = put(k.cuda()), None if v is None else put(v.cuda())
        out = None
        if q is not None:
            dq = put(q.cuda())
            out = torch.full_like(q, float("nan"))
            dout = dq if opt.get("inplace") else put(out.cuda())
            if opt.get("inplace"):
                out = q.clone()
        self.ws.fill_(0x5A)
        kvq.kvq_append(self.dcodes, None if "unscaled" in self.kind else self.dscales, dk, dv, self.dtable,
                       torch.tensor(self.lens, dtype=torch.int32).cuda(), torch.tensor(start, dtype=torch.int32).cuda(),
                       self.ws, self.layout, self.kind, q=dq, q_out=dout, cos_sin=None if angles is None else angles.cuda(),
                       rot_offset=first, interleaved=pairs,
                       positions=None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda())
        assert kvq.kvq_workspace_status(self.ws) == status
        M.append(self.codes, self.scales, q, k, v, self.table, self.lens, start, self.layout, self.kind, angles, first, pairs,
                 positions, out, skipped)
        if q is not None:
            assert torch.equal(dout.cpu().view(torch.int16), out.view(torch.int16)), "rotated queries"
        assert torch.equal(self.dcodes.cpu(), self.codes), "codes"
        if "unscaled" not in self.kind:
            bits = torch.int32 if self.kind == "fp8_e4m3_page" else torch.int16
            assert torch.equal(self.dscales.cpu().view(bits), self.scales.view(bits)), "scales"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d", GQA)
@pytest.mark.parametrize("pairs", [False, True])
def test_steps_of_a_batch(kind, hq, hkv, d, pairs):
    """Prompts, further turns and single tokens of four sequences, one of them idle at times."""
    c = Cache(kind, hkv, d, batch=4, room=6, seed=d + hq)
    angles = M.angles_of(96, d if pairs else d // 2)
    for i, new in enumerate([[37, 1, 0, 16], [1, 1, 1, 1], [5, 0, 20, 33], [1, 1, 1, 1], [0, 15, 0, 2]]):
        q, k, v = c.rows(sum(new), hq, spread=1.5 ** i)
        c.append(new, q, k, v, angles=angles, pairs=pairs, first=0 if pairs else d // 4)


@pytest.mark.parametrize("kind", [k for k in KINDS if k != "fp8_e4m3_page"])
def test_latent_rows_turn_their_tail_alone(kind):
    c = Cache(kind, 1, 576, batch=2, room=4, mla=True, dv=512, seed=3)
    for new in ([30, 7], [1, 1]):
        q, k, v = c.rows(sum(new), 16)
        c.append(new, q, k, v, angles=M.angles_of(64, 64), first=512, pairs=True)


@pytest.mark.parametrize("kind,size,d", [("fp8_e4m3", 5, 96), ("q8_0", 32, 32), ("fp8_e5m2_unscaled", 1, 160)])
def test_other_page_sizes_and_widths(kind, size, d):
    c = Cache(kind, 3, d, batch=2, room=20, size=size, seed=1)
    for new in ([11, 3], [1, 9]):
        q, k, v = c.rows(sum(new), 5)
        c.append(new, q, k, v, angles=M.angles_of(30, 16), first=8)


@pytest.mark.parametrize("kind", KINDS)
def test_slices_of_one_projection_and_queries_in_place(kind):
    hq, hkv, d = 8, 2, 128
    c = Cache(kind, hkv, d, batch=2, room=4, seed=4)

    def slices(x):  # the rows of x inside wider ones
        wide = torch.zeros(x.shape[0], x.shape[1] + 5, d, dtype=x.dtype, device="cuda")
        wide[:, 2:2 + x.shape[1]] = x
        return wide[:, 2:2 + x.shape[1]]

    for inplace in (False, True):
        for new in ([20, 1], [1, 1]):
            q, k, v = c.rows(sum(new), hq)
            c.append(new, q, k, v, place=slices, inplace=inplace, angles=M.angles_of(64, d))


@pytest.mark.parametrize("kind", KINDS)
def test_keys_alone_and_no_rotation(kind):
    c = Cache(kind, 2, 64, batch=3, room=3, seed=5)
    for new in ([17, 0, 3], [1, 1, 1]):
        _, k, v = c.rows(sum(new), 0)
        c.append(new, None, k, v, angles=M.angles_of(48, 64))
        q, k, v = c.rows(sum(new), 4)
        c.append(new, q, k, v)


@pytest.mark.parametrize("kind", KINDS)
def test_given_positions_and_those_outside_the_table(kind):
    c = Cache(kind, 2, 128, batch=2, room=3, seed=6)
    q, k, v = c.rows(9, 4)
    c.append([5, 4], q, k, v, angles=M.angles_of(50, 128), positions=[9, 0, 49, 3, 3, 7, 8, 8, 9])
    q, k, v = c.rows(2, 4)
    c.append([1, 1], q, k, v, angles=M.angles_of(50, 128), positions=[50, 2], status=-1)
    q, k, v = c.rows(2, 4)
    c.append([1, 1], q, k, v, angles=M.angles_of(50, 128), positions=[1, -1], status=-1)


@pytest.mark.parametrize("kind", KINDS)
def test_masked_and_bad_pages_take_nothing(kind):
    c = Cache(kind, 2, 128, batch=3, room=3, seed=7)
    c.table[0, 1] = -1
    c.dtable.copy_(c.table)
    q, k, v = c.rows(40 + 20 + 1, 4)
    c.append([40, 20, 1], q, k, v, angles=M.angles_of(64, 128))
    c.table[1, 2] = c.layout.num_pages
    c.dtable.copy_(c.table)
    q, k, v = c.rows(1 + 25 + 1, 4)
    c.append([1, 25, 1], q, k, v, angles=M.angles_of(64, 128), status=-1)


@pytest.mark.parametrize("kind", KINDS)
def test_inconsistent_sequences_are_skipped_and_reported(kind):
    """More new tokens than stored ones; more stored than the table holds; rows behind the last sequence stay."""
    c = Cache(kind, 2, 128, batch=4, room=2, seed=8)
    q, k, v = c.rows(30, 4)
    c.append([4, 6, 5, 3], q, k, v, status=-1, skipped=(1, 2), lens=[4, 5, 33, 3], start=[0, 4, 10, 15, 18])
    c = Cache(kind, 2, 128, batch=3, room=2, seed=9)
    q, k, v = c.rows(12, 4)
    c.append([4, 0, 0], q, k, v, status=-1, skipped=(1, 2), lens=[4, 5, 9], start=[0, 4, 13, 9])


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled"])
@pytest.mark.parametrize("hkv,d,mla", [(2, 128, False), (1, 576, True)])
def test_without_a_rotation_it_stores_what_the_stores_store(kind, hkv, d, mla):
    c = Cache(kind, hkv, d, batch=3, room=5, mla=mla, dv=512 if mla else d, seed=10)
    new = [70, 1, 33]
    _, k, v = c.rows(sum(new), 0, spread=30.0)
    k[3, 0, :32] = 0
    codes, scales = c.codes.cuda(), c.scales.cuda()
    slots = [int(c.table[b, i // 16]) * 16 + i % 16 for b, n in enumerate(new) for i in range(n)]
    slots = torch.tensor(slots, dtype=torch.int64).cuda()
    if "unscaled" in kind:
        kvq.kvq_store_unscaled(codes, k.cuda(), None if mla else v.cuda(), slots, c.layout, kind)
    else:
        kvq.kvq_store(codes, scales, k.cuda(), None if mla else v.cuda(), slots, c.layout, kind)
    c.append(new, None, k, v)
    assert torch.equal(c.dcodes, codes) and torch.equal(c.dscales, scales)


def test_a_page_grows_its_scale_and_keeps_it():
    """Values around the borders of a scale (448 * 2^e and just above), zeros, values past the largest scale, values that
    fall out of the codes' range when the scale grows, and rows given up and written again."""
    c = Cache("fp8_e4m3_page", 2, 64, batch=1, room=2, seed=11)
    for x in (0.0, 2.0 ** -45, 2.0 ** -33, 1.0, 1.75, 1.7578125, 448.0, 450.0, 3.0, 2.0 ** 40, 3e38):
        _, k, v = c.rows(1, 0)
        k = (k.float().sign() * x).to(torch.bfloat16)
        v[:, 1] = 0
        c.append([1], None, k, v)
    assert float(c.scales[int(c.table[0, 0]), 0].max()) == 2.0 ** 32
    c.lens = [5]  # six rows given up: the scale stays
    _, k, v = c.rows(2, 0)
    c.append([2], None, k, v)
    assert float(c.scales[int(c.table[0, 0]), 0].max()) == 2.0 ** 32
    c.lens = [0]  # all of them: the page starts afresh
    _, k, v = c.rows(20, 0)
    c.append([20], None, k, v)
    assert float(c.scales[int(c.table[0, 0]), 0].max()) < 1.0


@pytest.mark.parametrize("kind", ["q8_0", "fp8_e4m3_page"])
def test_large_batches_and_long_rows(kind):
    """More sequences than a CTA has threads, most of them idle; and more heads than one CTA's rows."""
    c = Cache(kind, 2, 64, batch=700, room=2, seed=12)
    new = [(b % 7 == 3) * (1 + b % 19) for b in range(700)]
    q, k, v = c.rows(sum(new), 3)
    c.append(new, q, k, v, angles=M.angles_of(32, 64))
    c = Cache(kind, 40, 128, batch=2, room=2, seed=13)
    q, k, v = c.rows(3, 80)
    c.append([1, 2], q, k, v, angles=M.angles_of(32, 128), pairs=True)


def test_captured_and_replayed_on_a_stream_of_its_own():
    c = Cache("fp8_e4m3_page", 2, 128, batch=2, room=2, seed=14)
    q, k, v = c.rows(4, 4)
    angles = M.angles_of(32, 128).cuda()
    lens, start = torch.tensor([3, 1], dtype=torch.int32).cuda(), torch.tensor([0, 3, 4], dtype=torch.int32).cuda()
    dq, dk, dv, out = q.cuda(), k.cuda(), v.cuda(), torch.empty_like(q, device="cuda")
    call = lambda: kvq.kvq_append(c.dcodes, c.dscales, dk, dv, c.dtable, lens, start, c.ws, c.layout, c.kind, q=dq,  # noqa: E731
                                  q_out=out, cos_sin=angles)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        call()
    want = torch.empty_like(q)
    for k2 in (k, (k.float() * 3).to(torch.bfloat16)):
        dk.copy_(k2)
        graph.replay()
        assert kvq.kvq_workspace_status(c.ws) == 0
        M.append(c.codes, c.scales, q, k2, v, c.table, [3, 1], [0, 3, 4], c.layout, c.kind, angles.cpu(), q_out=want)
        assert torch.equal(c.dcodes.cpu(), c.codes) and torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))
