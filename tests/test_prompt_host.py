"""Host-side refusals of kvq_prompt (no GPU needed)."""
import ctypes

import pytest
import torch

from block_quantized_bit_gb300 import build_lib, kvq

FAKE = 0x10000  # an aligned host address that must never be dereferenced: validation fails first
P = ctypes.c_void_p
EINVAL, EHEADDIM, EALIGN, EWORKSPACE, EUNSUPPORTED = -1, -3, -4, -5, -8


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return kvq.lib()


def prompt(lib, q=FAKE, k=FAKE, v=FAKE, start=FAKE, total=9, batch=2, hq=8, hkv=2, d=128, scale=1.0, out=FAKE, od=0,
           strides=None, ws=FAKE, wb=256):
    return lib.kvq_prompt(P(q), P(k), P(v), P(start), total, batch, hq, hkv, d, ctypes.c_float(scale), P(out), od,
                          None if strides is None else ctypes.byref(kvq.kvq_prompt_strides(*strides)), P(ws), wb, None)


def test_refusals(lib):
    assert prompt(lib, od=2) == EINVAL
    assert prompt(lib, total=-1) == EINVAL and prompt(lib, batch=-1) == EINVAL
    assert prompt(lib, hq=0) == EINVAL and prompt(lib, hkv=0) == EINVAL and prompt(lib, hq=7) == EINVAL
    assert prompt(lib, d=0) == EHEADDIM and prompt(lib, d=100) == EHEADDIM
    assert prompt(lib, d=96) == EUNSUPPORTED and prompt(lib, batch=2049) == EUNSUPPORTED
    assert prompt(lib, total=2 ** 31 - 1) == EUNSUPPORTED and prompt(lib, total=2 ** 30, hq=1 << 10) == EUNSUPPORTED
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert prompt(lib, scale=s) == EINVAL
    assert prompt(lib, wb=255) == EWORKSPACE
    for name in ("q", "k", "v", "start", "out", "ws"):
        assert prompt(lib, **{name: 0}) == EINVAL
        assert prompt(lib, **{name: FAKE + 2}) == EALIGN


def test_stride_refusals(lib):
    good = [8 * 128, 128, 2 * 128, 128, 2 * 128, 128, 8 * 128, 128]
    for i in range(8):
        for bad in (0, -8, 12, 1 << 39):
            assert prompt(lib, strides=good[:i] + [bad] + good[i + 1:]) == EINVAL
    assert prompt(lib, strides=good, wb=0) == EWORKSPACE      # the strides themselves are fine
    # along a dimension of one a stride says nothing
    assert prompt(lib, strides=good[:2] + [256, 1, 256, 3] + good[6:], hkv=1, wb=0) == EWORKSPACE
    assert prompt(lib, strides=[1, 128, 5, 128, 7, 128, 3, 128], total=1, wb=0) == EWORKSPACE


def test_the_binding_checks_what_it_marshals():
    q, k = torch.zeros(9, 8, 128, dtype=torch.bfloat16), torch.zeros(9, 2, 128, dtype=torch.bfloat16)
    good = dict(q=q, k=k, v=k, q_start=torch.zeros(3, dtype=torch.int32), out=torch.zeros(9, 8, 128),
                workspace=torch.zeros(256, dtype=torch.uint8))
    for bad in (dict(q=q[:, 0]), dict(v=k[:8]), dict(k=k[:8], v=k[:8]), dict(out=torch.zeros(9, 8, 64)),
                dict(k=k[:, :, :64], v=k[:, :, :64]), dict(q_start=torch.zeros(0, dtype=torch.int32)),
                dict(q=torch.zeros(9, 8, 256, dtype=torch.bfloat16)[:, :, ::2]), {}):
        with pytest.raises(ValueError):
            kvq.kvq_prompt(**{**good, **bad})
    for bad in (dict(q=q.half()), dict(k=k.float(), v=k.float()), dict(out=torch.zeros(9, 8, 128, dtype=torch.float16)),
                dict(q_start=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            kvq.kvq_prompt(**{**good, **bad})
