"""Forms of kvq_tree that the other tests leave out: more drafted tokens than the decode kernels take at once, masks of
several words over the latent row, more sequences than the flash kernel's table holds, and other scales.  Tolerances as
in test_tree_gpu.py."""
import random

import pytest
import torch

from block_quantized_bit_gb300 import kvq

from plain64 import tree64
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,mla,path,kind", [(4, 2, 64, False, 0, "q8_0"), (8, 2, 128, False, 1, "fp8_e4m3"),
                                                    (16, 1, 576, True, 2, "fp8_e4m3"), (16, 1, 576, True, 1, "q8_0")])
def test_more_drafts_than_the_decode_kernels_take_at_once(hq, hkv, d, mla, path, kind):
    drafted = [256, 200, 0, 255, 256, 31, 256, 120]            # 1374: chunks of 1024 and 350
    ctx = [50, 300, 20, 0, 17, 90, 33, 5]
    c = Case(hq, hkv, d, kind, ctx, drafted, words=4, mla=mla, mask="any", seed=d)
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    c.check(out, tensor=path == 2)


@pytest.mark.parametrize("words", [2, 3, 4])
@pytest.mark.parametrize("hq,path", [(128, 0), (64, 2), (128, 1)])
def test_masks_of_several_words_over_latent_rows(hq, path, words):
    n = 64 * words
    c = Case(hq, 1, 576, "fp8_e4m3", [0, 300, 15, 0], [n, n - 1, 17, 40], words=words, mla=True, masked=0.15, mask="any",
             seed=words)
    c.mask[c.start[3]:c.start[3] + 20] = 0                     # nothing before them either: zeros
    c.mask[c.start[0] + 3] = 0
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == 0
    assert (out[c.start[3]:c.start[3] + 20] == 0).all() and (out[c.start[0] + 3] == 0).all()
    c.check(out, tensor=path != 1)


@pytest.mark.parametrize("batch", [2048, 2049])
def test_sequences_up_to_and_past_the_flash_kernels_table(batch):
    r = random.Random(batch)
    c = Case(4, 2, 128, "fp8_e4m3", [r.randint(0, 60) for _ in range(batch)], [r.randint(0, 3) for _ in range(batch)],
             seed=batch)
    out, ws = c.run()
    assert kvq.kvq_workspace_status(ws) == 0
    c.check(out, tensor=batch <= 2048)


@pytest.mark.parametrize("scale", [0.03, 0.5, 1.7])
@pytest.mark.parametrize("hq,hkv,d,mla,path", [(8, 2, 128, False, 0), (16, 2, 256, False, 0), (4, 2, 64, False, 0),
                                               (128, 1, 576, True, 0)])
def test_other_scales(hq, hkv, d, mla, path, scale):
    c = Case(hq, hkv, d, "fp8_e4m3", [0, 500, 33], [7, 20, 64], mla=mla, seed=3)
    out = torch.full((c.total, hq, c.v_dim), float("nan"), device="cuda")
    ws = kvq.alloc_tree_workspace(c.L, len(c.lens), c.total, hq, c.table.shape[1], path)
    kvq.kvq_tree(c.q, c.codes, c.scales, c.table, c.dl, c.ds, c.mask, out, ws, c.L, c.kind, scale, path)
    assert kvq.kvq_workspace_status(ws) == 0
    ref = torch.zeros(out.shape, dtype=torch.float64, device="cuda")
    ref, mag = tree64(c.q, c.codes, c.scales, c.kind, c.table, c.lens, c.start, c.mask, c.v_dim, mla, scale, ref)
    n = c.start[-1]
    # the score's part of the tolerance grows with the scale
    rel = 2.0 ** -8 + 2 * (1.5e-4 + (2.2e-3 if mla else 1e-3) * max(1.0, scale))
    assert ((out[:n].double() - ref[:n]).abs() <= rel * mag[:n] + 1e-6).all()
    assert torch.isnan(out[n:]).all()
