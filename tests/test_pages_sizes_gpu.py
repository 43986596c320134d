"""kvq_pages_* with pages of other sizes than 16 tokens, against the host model."""
import random

import numpy as np
import pytest
import torch

import pages_model
from block_quantized_bit_gb300 import kvq
from pages_model import Model, pages
from test_pages_gpu import LAYOUTS, dev, pool, same, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page_size", [1, 5, 32, 100])
@pytest.mark.parametrize("key", ["gqa128", "d32", "mla"])
def test_page_sizes(page_size, key, monkeypatch):
    monkeypatch.setattr(pages_model, "PAGE", page_size)
    r = random.Random(page_size)
    B, num_pages = 8, 6000 // page_size + 60
    lens = [0, 1, page_size, 3 * page_size + 1, 200, 333, 64, 2 * page_size]
    room = pages(600) + 2
    t, refs = tables(r, num_pages, lens, room)
    h, d, dv, mla = LAYOUTS[key]
    L = kvq.Layout(num_pages, page_size, h, d, dv, mla)
    for kind in ("q8_0", "fp8_e4m3_unscaled"):
        codes, scales = pool(L, kind, 3)
        m = Model(t, lens, refs, [codes.cpu().numpy()] + ([] if scales is None else [scales.cpu().numpy()]))
        table, dl, dr = dev(t), dev(lens), dev(refs)
        ws = kvq.alloc_pages_workspace(L, B, room)
        whole = kind != "q8_0" or page_size * h * d * (1 if mla else 2) // 16 % 16 == 0  # (else copies are refused)

        def equal():
            same(m, table, dl, dr)
            assert np.array_equal(codes.cpu().numpy(), m.pools[0])
            assert scales is None or np.array_equal(scales.cpu().numpy(), m.pools[1])

        for step in range(3):
            src, dst = [r.randrange(B) for _ in range(B)], r.sample(range(B), B)
            cs, cd = dev([77] * B), dev([77] * B)
            kvq.kvq_pages_fork(table, dl, dr, dev(src), dev(dst), cs, cd, ws, L)
            assert kvq.kvq_workspace_status(ws) == 0
            want = m.fork(src, dst)
            assert (cs.cpu().tolist(), cd.cpu().tolist()) == want
            if whole:
                kvq.kvq_pages_copy(codes, scales, cs, cd, L, kind)
                m.copy(*want)
            else:
                with pytest.raises(kvq.KvqError):
                    kvq.kvq_pages_copy(codes, scales, cs, cd, L, kind)
            equal()
            drafted = [r.randrange(65) for _ in range(B)]
            grown = [int(x) + n for x, n in zip(m.lens, drafted)]
            kvq.kvq_pages_resize(table, dl, dr, dev(range(B)), dev(grown), ws, L)
            assert kvq.kvq_workspace_status(ws) == 0 and m.resize(list(range(B)), grown)
            equal()
            kept = [[j for j in range(n) if r.random() < 0.4] for n in drafted]
            keep = np.array([[sum(1 << j for j in k)] for k in kept], np.uint64)
            new = dev([-7] * B)
            kvq.kvq_pages_compact(codes, scales, table, dl, dev(np.concatenate([[0], np.cumsum(drafted)])),
                                  torch.from_numpy(keep.view(np.int64)).cuda(), new, ws, L, kind, page_refs=dr)
            assert kvq.kvq_workspace_status(ws) == 0
            left = [m.compact(b, drafted[b], kept[b]) for b in range(B)]
            assert new.cpu().tolist() == left
            kvq.kvq_pages_resize(table, dl, dr, dev(range(B)), new, ws, L)
            assert m.resize(list(range(B)), left)
            equal()
            cut = [int(x) // 3 // page_size * page_size for x in m.lens]   # whole pages: rows may grow again
            kvq.kvq_pages_resize(table, dl, dr, dev(range(B)), dev(cut), ws, L)
            assert kvq.kvq_workspace_status(ws) == 0 and m.resize(list(range(B)), cut)
            equal()
