"""Host-side refusals of the page calls (no GPU needed): each returns its status before any launch."""
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


def copy(lib, lay, pool=FAKE, scales=FAKE, src=FAKE, dst=FAKE, n=3, kind=1):
    return lib.kvq_pages_copy(P(pool), P(scales), P(src), P(dst), n, ctypes.byref(lay.c()), kind, None)


def test_copy_refusals(lib):
    assert copy(lib, L(), kind=7) == EKIND
    assert copy(lib, L(head_dim=48, v_dim=48)) == EHEADDIM
    assert copy(lib, L(), n=-1) == EINVAL
    assert copy(lib, L(), src=0) == EINVAL
    assert copy(lib, L(), scales=0) == EINVAL
    assert copy(lib, L(), pool=FAKE + 8) == EALIGN
    assert copy(lib, L(), dst=FAKE + 2) == EALIGN
    assert copy(lib, L(page_size=2, num_kv_heads=1, head_dim=32, v_dim=32)) == EUNSUPPORTED  # 8 bytes of scales
    assert copy(lib, L(), n=0) == 0


def fork(lib, lay, table=FAKE, lens=FAKE, refs=FAKE, src=FAKE, dst=FAKE, n=2, cs=FAKE, cd=FAKE, ws=FAKE, wb=None, batch=4,
         maxp=8):
    if wb is None:
        wb = lib.kvq_pages_workspace_bytes(ctypes.byref(lay.c()), n, maxp)
    return lib.kvq_pages_fork(P(table), maxp, P(lens), batch, P(refs), P(src), P(dst), n, P(cs), P(cd), P(ws), wb,
                              ctypes.byref(lay.c()), None)


def resize(lib, lay, table=FAKE, lens=FAKE, refs=FAKE, seqs=FAKE, new=FAKE, n=2, ws=FAKE, wb=None, batch=4, maxp=8):
    if wb is None:
        wb = lib.kvq_pages_workspace_bytes(ctypes.byref(lay.c()), n, maxp)
    return lib.kvq_pages_resize(P(table), maxp, P(lens), batch, P(refs), P(seqs), P(new), n, P(ws), wb,
                                ctypes.byref(lay.c()), None)


@pytest.mark.parametrize("call", [fork, resize])
def test_fork_and_resize_refusals(lib, call):
    assert call(lib, L(num_kv_heads=0)) == EINVAL
    assert call(lib, L(), n=-1) == EINVAL
    assert call(lib, L(), batch=-1) == EINVAL
    assert call(lib, L(), maxp=0) == EINVAL
    assert call(lib, L(), maxp=1 << 28) == EINVAL            # 2^32 tokens per row
    assert call(lib, L(num_pages=(1 << 26) + 1)) == EUNSUPPORTED
    assert call(lib, L(), wb=255) == EWORKSPACE
    assert call(lib, L(), ws=0) == EINVAL
    assert call(lib, L(), ws=FAKE + 8) == EALIGN
    for name in ("table", "lens", "refs"):
        assert call(lib, L(), **{name: 0}) == EINVAL
        assert call(lib, L(), **{name: FAKE + 2}) == EALIGN
    for name in ("src", "dst", "cs", "cd") if call is fork else ("seqs", "new"):
        assert call(lib, L(), **{name: 0}) == EINVAL
        assert call(lib, L(), **{name: FAKE + 1}) == EALIGN


def compact(lib, lay, pool=FAKE, scales=FAKE, table=FAKE, lens=FAKE, start=FAKE, keep=FAKE, words=1, batch=2, new=FAKE,
            refs=0, ws=FAKE, wb=256, kind=1, maxp=8):
    return lib.kvq_pages_compact(P(pool), P(scales), P(table), maxp, P(lens), P(start), P(keep), words, batch, P(new),
                                 P(refs), P(ws), wb, ctypes.byref(lay.c()), kind, None)


def test_compact_refusals(lib):
    assert compact(lib, L(), kind=0) == EKIND
    assert compact(lib, L(), words=0) == EINVAL
    assert compact(lib, L(), words=5) == EUNSUPPORTED
    assert compact(lib, L(), batch=-1) == EINVAL
    assert compact(lib, L(), maxp=0) == EINVAL
    assert compact(lib, L(), wb=128) == EWORKSPACE
    assert compact(lib, L(num_kv_heads=40000)) == EUNSUPPORTED
    for name in ("pool", "scales", "table", "lens", "start", "keep", "new", "ws"):
        assert compact(lib, L(), **{name: 0}) == EINVAL
        assert compact(lib, L(), **{name: FAKE + 2}) == EALIGN
    assert compact(lib, L(), keep=FAKE + 4) == EALIGN
    assert compact(lib, L(), refs=FAKE + 2) == EALIGN


def test_workspace_sizes(lib):
    size = lambda lay, n, maxp: lib.kvq_pages_workspace_bytes(ctypes.byref(lay.c()), n, maxp)  # noqa: E731
    assert size(L(), -1, 8) == 0 and size(L(), 2, 0) == 0 and size(L(head_dim=31, v_dim=31), 2, 8) == 0
    assert size(L(num_pages=1 << 26), 2, 8) > 0 and size(L(num_pages=(1 << 26) + 1), 2, 8) == 0
    assert size(L(), 64, 100) >= 256 + 64 * 100 * 4


def test_the_binding_checks_what_it_marshals():
    """Lists of different lengths, other types, strided and host tensors never reach the library."""
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    lay, ws = L(), torch.zeros(4096, dtype=torch.uint8)
    pool, scales = kvq.alloc_pool(lay, "cpu")
    with pytest.raises(ValueError):
        kvq.kvq_pages_copy(pool, scales, i(2), i(3), lay, "q8_0")
    with pytest.raises(ValueError):
        kvq.kvq_pages_copy(pool, None, i(2), i(2), lay, "q8_0")                     # a scaled kind without scales
    with pytest.raises(ValueError):
        kvq.kvq_pages_copy(pool[:9], scales, i(2), i(2), lay, "q8_0")               # nine of ten pages
    with pytest.raises(ValueError):
        kvq.kvq_pages_copy(pool, scales, i(2), i(2), lay, "q8_0")                   # host tensors
    with pytest.raises(ValueError):
        kvq.kvq_pages_resize(i(8).view(2, 4), i(2), i(9), i(1), i(1), ws, lay)      # nine counts, ten pages
    with pytest.raises(ValueError):
        kvq.kvq_pages_fork(i(8).view(2, 4), i(2), i(10), i(1), i(1), i(2), i(1), ws, lay)
    with pytest.raises(ValueError):
        kvq.kvq_pages_compact(ws, ws, i(8).view(2, 4), i(2), i(2), torch.zeros(2, 1, dtype=torch.int64), i(2), ws, lay,
                              "q8_0")
    with pytest.raises(TypeError):
        kvq.kvq_pages_resize(i(8).view(2, 4), i(2), i(10), i(1).long(), i(1), ws, lay)
    with pytest.raises(ValueError):
        kvq.kvq_pages_resize(i(8).view(4, 2).t(), i(2), i(10), i(1), i(1), ws, lay)
