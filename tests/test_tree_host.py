"""Host-side refusals of kvq_tree (no GPU needed)."""
import ctypes

import pytest
import torch

from block_quantized_bit_gb300 import build_lib, kvq

FAKE = 0x10000  # an aligned host address that must never be dereferenced: validation fails first
P = ctypes.c_void_p
EINVAL, EKIND, EHEADDIM, EALIGN, EWORKSPACE, EUNSUPPORTED = -1, -2, -3, -4, -5, -8


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return kvq.lib()


def L(**kw):
    base = dict(num_pages=10, page_size=16, num_kv_heads=2, head_dim=128, v_dim=128, mla=False)
    base.update(kw)
    return kvq.Layout(**base)


def tree(lib, lay, q=FAKE, pool=FAKE, scales=FAKE, table=FAKE, maxp=8, lens=FAKE, start=FAKE, mask=FAKE, words=1, total=6,
         batch=2, hq=8, scale=1.0, out=FAKE, od=0, ws=FAKE, wb=None, kind=1, path=0):
    if wb is None:
        wb = lib.kvq_tree_workspace_bytes(ctypes.byref(lay.c()), batch, total, hq, maxp, path)
    return lib.kvq_tree(P(q), P(pool), P(scales), P(table), maxp, P(lens), P(start), P(mask), words, total, batch, hq,
                        ctypes.c_float(scale), P(out), od, P(ws), wb, ctypes.byref(lay.c()), kind, path, None)


MLA = dict(num_kv_heads=1, head_dim=576, v_dim=512, mla=True)


def test_refusals(lib):
    assert tree(lib, L(num_kv_heads=0)) == EINVAL
    assert tree(lib, L(head_dim=100, v_dim=100)) == EHEADDIM
    assert tree(lib, L(), kind=9) == EKIND
    assert tree(lib, L(), od=2) == EINVAL
    assert tree(lib, L(), hq=7) == EINVAL
    assert tree(lib, L(), batch=-1) == EINVAL and tree(lib, L(), total=-1) == EINVAL and tree(lib, L(), maxp=0) == EINVAL
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert tree(lib, L(), scale=s) == EINVAL
    assert tree(lib, L(), words=0) == EINVAL
    assert tree(lib, L(), words=5) == EUNSUPPORTED
    assert tree(lib, L(), path=3) == EINVAL and tree(lib, L(), path=-1) == EINVAL
    assert tree(lib, L(page_size=32)) == EUNSUPPORTED
    assert tree(lib, L(head_dim=96, v_dim=96)) == EUNSUPPORTED
    assert tree(lib, L(head_dim=64, v_dim=64), path=2) == EUNSUPPORTED
    assert tree(lib, L(**MLA), hq=65, path=2) == EUNSUPPORTED
    assert tree(lib, L(), maxp=1 << 28) == EINVAL
    assert tree(lib, L(), wb=256) == EWORKSPACE
    assert tree(lib, L(), batch=2049, path=2) == EUNSUPPORTED
    for name in ("q", "pool", "scales", "table", "lens", "start", "mask", "out", "ws"):
        assert tree(lib, L(), **{name: 0}) == EINVAL
        assert tree(lib, L(), **{name: FAKE + 2}) == EALIGN
    assert tree(lib, L(), mask=FAKE + 4) == EALIGN


def test_workspace_sizes(lib):
    size = lambda lay, *a: lib.kvq_tree_workspace_bytes(ctypes.byref(lay.c()), *a)  # noqa: E731
    assert size(L(), 2, 6, 7, 8, 0) == 0 and size(L(), 2, 6, 8, 0, 0) == 0 and size(L(), 2, 6, 8, 8, 3) == 0
    assert size(L(page_size=32), 2, 6, 8, 8, 0) == 0
    assert size(L(head_dim=64, v_dim=64), 2, 6, 8, 8, 2) == 0
    assert size(L(head_dim=64, v_dim=64), 2, 6, 8, 8, 0) > 0
    assert size(L(**MLA), 2, 6, 128, 8, 0) > 0
    assert size(L(), 4096, 6, 8, 8, 2) == 0 and size(L(), 4096, 6, 8, 8, 0) > 0   # the flash kernel's table ends at 2048


def test_the_binding_checks_what_it_marshals():
    lay = L()
    pool, scales = kvq.alloc_pool(lay, "cpu")
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(6, 8, 128, dtype=torch.bfloat16)
    good = dict(q=q, pool=pool, scales=scales, block_table=i(16).view(2, 8), seq_lens=i(2), q_start=i(3),
                tree_mask=torch.zeros(6, 1, dtype=torch.int64), out=torch.zeros(6, 8, 128),
                workspace=torch.zeros(64, dtype=torch.uint8), layout=lay, kind="q8_0")
    bad = [dict(q=q[:, :, :64]), dict(out=torch.zeros(6, 8, 64)), dict(q_start=i(2)), dict(scales=None),
           dict(tree_mask=torch.zeros(5, 1, dtype=torch.int64)), dict(seq_lens=i(3)),
           dict(q=torch.zeros(6, 16, 128, dtype=torch.bfloat16)[:, ::2]), dict(pool=pool[:4]), {}]
    for b in bad:
        with pytest.raises(ValueError):
            kvq.kvq_tree(**{**good, **b})
    for b in (dict(q=q.float()), dict(out=torch.zeros(6, 8, 128, dtype=torch.float16)), dict(seq_lens=i(2).long()),
              dict(tree_mask=i(6).view(6, 1))):
        with pytest.raises(TypeError):
            kvq.kvq_tree(**{**good, **b})
