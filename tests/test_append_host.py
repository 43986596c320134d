"""Refusals of kvq_append and of the kind fp8_e4m3_page, checked before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from block_quantized_bit_gb300 import build_lib, kvq

OK, EINVAL, EKIND, EALIGN, EWORKSPACE, EUNSUPPORTED = 0, -1, -2, -4, -5, -8
FAKE = 0x10000  # an aligned host address that must never be dereferenced: validation fails first
PAGE = kvq.KVQ_FP8_E4M3_PAGE


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return kvq.lib()


def layout(num_pages=10, page_size=16, hkv=2, d=128, dv=None, mla=False):
    return kvq.Layout(num_pages, page_size, hkv, d, d if dv is None else dv, mla)


def append(lib, lay=None, kind=1, q=FAKE, k=FAKE, v=FAKE, out=2 * FAKE, pool=FAKE, scales=FAKE, table=FAKE, maxp=4, lens=FAKE,
           start=FAKE, positions=None, total=8, batch=2, hq=8, rope=(FAKE, 100, 64, 0, 0), strides=None, ws=FAKE, wb=256):
    r = None if rope is None else ctypes.byref(kvq.kvq_rope(*rope))
    s = None if strides is None else ctypes.byref(kvq.kvq_prompt_strides(*strides))
    return lib.kvq_append(pool, scales, q, k, v, table, maxp, lens, start, positions, total, batch, hq, out, r, s, ws, wb,
                          ctypes.byref((lay or layout()).c()), kind, None)


def reaches_the_device(status):
    """Every check passed: what is left is the device check."""
    return status in (-6, -7)


def test_append_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("calls that pass validation would launch")
    assert lib.kvq_append_workspace_bytes() == 256
    for kind in (1, 2, 3, 4, PAGE):
        assert reaches_the_device(append(lib, kind=kind))
    for kind in (0, 5, 7, -1):
        assert append(lib, kind=kind) == EKIND
    assert append(lib, layout(d=100)) == -3
    # sizes
    assert append(lib, total=-1) == EINVAL and append(lib, batch=-1) == EINVAL and append(lib, maxp=0) == EINVAL
    assert append(lib, maxp=1 << 27) == EINVAL                 # lengths pass 32 bits
    assert append(lib, hq=-1) == EINVAL
    # queries come with an output and a number of heads, or not at all
    assert append(lib, q=None) == EINVAL and append(lib, out=None) == EINVAL and append(lib, hq=0) == EINVAL
    assert append(lib, q=None, out=None) == EINVAL
    assert reaches_the_device(append(lib, q=None, out=None, hq=0))
    assert reaches_the_device(append(lib, out=FAKE))           # in place
    assert append(lib, out=FAKE, strides=[1024, 128, 256, 128, 256, 128, 2048, 128]) == EINVAL
    # pointers
    for name in ("pool", "scales", "k", "v", "table", "lens", "start", "ws"):
        assert append(lib, **{name: None}) == EINVAL, name
    assert reaches_the_device(append(lib, kind=3, scales=None))
    for name in ("pool", "scales", "q", "k", "v", "out", "ws"):
        assert append(lib, **{name: FAKE + 8}) == EALIGN, name
    for name in ("table", "lens", "start", "positions"):
        assert append(lib, **{name: FAKE + 2}) == EALIGN, name
    assert append(lib, wb=255) == EWORKSPACE
    # the latent row has no v; a page's scale is not for it
    mla = layout(hkv=1, d=576, dv=512, mla=True)
    assert append(lib, mla) == EINVAL and reaches_the_device(append(lib, mla, v=None))
    assert append(lib, mla, v=None, kind=PAGE) == EUNSUPPORTED
    for lay in (layout(page_size=32), layout(d=96), layout(d=32), layout(d=512)):
        assert append(lib, lay, kind=PAGE, rope=None) == EUNSUPPORTED
    assert reaches_the_device(append(lib, layout(page_size=5), rope=None))
    assert append(lib, layout(d=2080), rope=None) == EUNSUPPORTED


def test_append_refuses_rotations_it_cannot_do(lib):
    if torch.cuda.is_available():
        pytest.skip("calls that pass validation would launch")
    for bad in ((None, 100, 64, 0, 0), (FAKE, 0, 64, 0, 0), (FAKE, 100, 0, 0, 0), (FAKE, 100, 24, 0, 0),
                (FAKE, 100, 64, -8, 0), (FAKE, 100, 64, 4, 0), (FAKE, 100, 128, 8, 0), (FAKE, 100, 144, 0, 0),
                (FAKE, 100, 64, 72, 0), (FAKE, 100, 64, 0, 2), (FAKE, 100, 1 << 30, 1 << 30, 0)):
        assert append(lib, rope=bad) == EINVAL, bad
    assert append(lib, rope=(FAKE + 8, 100, 64, 0, 0)) == EALIGN
    assert reaches_the_device(append(lib, rope=(FAKE, 1, 16, 112, 1))) and reaches_the_device(append(lib, rope=None))


def test_append_refuses_strides_that_are_not_rows(lib):
    if torch.cuda.is_available():
        pytest.skip("calls that pass validation would launch")
    good = [1536, 128, 1536, 128, 1536, 128, 1024, 128]
    assert reaches_the_device(append(lib, strides=good))
    for i in range(8):
        for bad in (0, -128, 100, 1 << 39):
            assert append(lib, strides=good[:i] + [bad] + good[i + 1:]) == EINVAL, (i, bad)
    # a stride says nothing along a dimension of one
    assert reaches_the_device(append(lib, total=1, strides=[1, 128, 5, 128, 7, 128, 3, 128]))


def test_kind_with_a_scale_per_page(lib):
    lay = layout(hkv=2, d=128)
    assert kvq.kvq_bytes_per_token_ex(lay, "fp8_e4m3_page") == 2 * 2 * 128 + 2 * 2 * 4 / 16
    assert kvq.kvq_num_pages_ex(lay, "fp8_e4m3_page", 10 ** 9) == 10 ** 9 // (2 * 2 * (16 * 128 + 4))
    assert kvq.alloc_pool(lay, "cpu", "fp8_e4m3_page")[1].shape == (10, 2, 2)
    # workspaces: by kind; the others keep theirs
    ref = ctypes.byref(lay.c())
    dec = lambda kind, *a, o=None: lib.kvq_decode_workspace_bytes_kind(ref, kind, *a, o)  # noqa: E731
    ext = lambda kind, *a, o=None: lib.kvq_extend_workspace_bytes_kind(ref, kind, *a, o)  # noqa: E731
    assert dec(1, 4, 8, 10) == lib.kvq_decode_workspace_bytes(ref, 4, 8, 10)
    assert ext(1, 4, 20, 8, 10) == lib.kvq_extend_workspace_bytes_ex(ref, 20, 8, 10, None)
    assert dec(PAGE, 4, 8, 10) > 256 and ext(PAGE, 4, 20, 8, 10) > 256
    assert dec(PAGE, 4, 7, 10) == 0 and dec(5, 4, 8, 10) == 0 and dec(PAGE, -1, 8, 10) == 0 and ext(PAGE, 4, -1, 8, 10) == 0
    assert dec(PAGE, 4, 8, 10, o=ctypes.byref(kvq.kvq_decode_options(0, 1))) == 0
    assert ext(PAGE, 4, 20, 8, 10, o=ctypes.byref(kvq.kvq_extend_options(0, 1))) == 0
    for bad in (layout(page_size=32), layout(d=96), layout(hkv=1, d=576, dv=512, mla=True)):
        assert lib.kvq_decode_workspace_bytes_kind(ctypes.byref(bad.c()), PAGE, 4, 8, 10, None) == 0


def decode(lib, lay=None, hq=8, scales=FAKE, ws=FAKE, wb=1 << 30, opts=None, kind=PAGE, sm=1.0, od=0, batch=2, maxp=10):
    return lib.kvq_decode_ex(FAKE, FAKE, scales, FAKE, maxp, FAKE, batch, hq, ctypes.c_float(sm), FAKE, od, ws, wb,
                             ctypes.byref((lay or layout()).c()), kind, opts, None)


def extend(lib, lay=None, hq=8, scales=FAKE, ws=FAKE, wb=1 << 30, opts=None, kind=PAGE, sm=1.0, od=0, batch=2, start=FAKE):
    return lib.kvq_extend_ex(FAKE, FAKE, scales, FAKE, 10, FAKE, start, 5, batch, hq, ctypes.c_float(sm), FAKE, od, ws, wb,
                             ctypes.byref((lay or layout()).c()), kind, opts, None)


def test_attention_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("calls that pass validation would launch")
    for call in (decode, extend):
        assert reaches_the_device(call(lib))
        assert call(lib, hq=7) == EINVAL and call(lib, scales=None) == EINVAL and call(lib, ws=None) == EINVAL
        assert call(lib, sm=float("nan")) == EINVAL and call(lib, od=2) == EINVAL and call(lib, batch=-1) == EINVAL
        assert call(lib, wb=256) == EWORKSPACE and call(lib, ws=FAKE + 8) == EALIGN and call(lib, scales=FAKE + 4) == EALIGN
        for lay in (layout(page_size=32), layout(d=96), layout(hkv=1, d=576, dv=512, mla=True)):
            assert call(lib, lay) == EUNSUPPORTED
    assert extend(lib, sm=0.0) == EINVAL and extend(lib, start=None) == EINVAL and extend(lib, batch=2049) == EUNSUPPORTED
    assert decode(lib, maxp=1 << 27) == EINVAL
    for o in ((1, 0), (0, 1), (0, 2)):
        assert decode(lib, opts=ctypes.byref(kvq.kvq_decode_options(*o))) == EUNSUPPORTED
    assert decode(lib, opts=ctypes.byref(kvq.kvq_decode_options(0, 3))) == EINVAL
    for o in ((1, 0), (2, 0), (0, 1)):
        assert extend(lib, opts=ctypes.byref(kvq.kvq_extend_options(*o))) == EUNSUPPORTED


def test_calls_that_do_not_take_a_scale_per_page(lib):
    ref = ctypes.byref(layout().c())
    F = ctypes.c_float(1.0)
    assert lib.kvq_store(FAKE, FAKE, FAKE, FAKE, FAKE, 4, ref, PAGE, None) == EKIND
    assert lib.kvq_store_unscaled(FAKE, FAKE, FAKE, FAKE, 4, ref, PAGE, None) == EKIND
    assert lib.kvq_decode_sparse(FAKE, FAKE, FAKE, FAKE, 10, FAKE, FAKE, 16, 2, 8, F, FAKE, 0, FAKE, 1 << 30, ref, PAGE,
                                 None) == EKIND
    assert lib.kvq_tree(FAKE, FAKE, FAKE, FAKE, 10, FAKE, FAKE, FAKE, 1, 5, 2, 8, F, FAKE, 0, FAKE, 1 << 30, ref, PAGE, 0,
                        None) == EKIND
    assert lib.kvq_pages_compact(FAKE, FAKE, FAKE, 10, FAKE, FAKE, FAKE, 1, 2, FAKE, None, FAKE, 256, ref, PAGE, None) == EKIND


def test_binding_refuses_what_it_can_see():
    lay = layout()
    codes, scales = kvq.alloc_pool(lay, "cpu", "fp8_e4m3_page")
    rows = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    start, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    call = lambda **o: kvq.kvq_append(**{**dict(pool=codes, scales=scales, k=rows, v=rows, block_table=table, seq_lens=lens,  # noqa: E731
                                                q_start=start, workspace=ws, layout=lay, kind="fp8_e4m3_page"), **o})
    with pytest.raises(ValueError, match="current CUDA device"):
        call()
    with pytest.raises(ValueError, match="q_start"):
        call(q_start=start[:2])
    with pytest.raises(TypeError, match="seq_lens"):
        call(seq_lens=lens.long())
    with pytest.raises(ValueError, match="block_table"):
        call(block_table=table[:, 0])
