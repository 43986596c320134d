"""Sizes of kvq_tree past the kernels' 32-bit counts (no GPU needed)."""
import ctypes

import pytest

from test_tree_host import EUNSUPPORTED, L, MLA, lib, tree  # noqa: F401 (lib: the fixture)

PAGES = (2 ** 31 - 128) // 16   # of the longest row that is taken


@pytest.mark.parametrize("lay", [L(num_kv_heads=1), L(head_dim=64, v_dim=64), L(**MLA)])
@pytest.mark.parametrize("path", [0, 1])
def test_rows_whose_rounded_length_passes_32_bits_are_refused(lib, lay, path):  # noqa: F811
    size = lambda maxp: lib.kvq_tree_workspace_bytes(ctypes.byref(lay.c()), 1, 6, 8, maxp, path)  # noqa: E731
    for maxp in (PAGES + 1, (2 ** 31 - 1) // 16):
        assert size(maxp) == 0
        assert tree(lib, lay, batch=1, maxp=maxp, wb=1 << 62, path=path) == EUNSUPPORTED
    assert size(PAGES) > 0
    if lib.kvq_device_check() != 0:
        assert tree(lib, lay, batch=1, maxp=PAGES, wb=1 << 62, path=path) == lib.kvq_device_check()


def test_the_flash_kernels_bounds_are_the_documented_ones(lib):  # noqa: F811
    lay = L()   # two kv heads
    size = lambda batch, total, hq, maxp, path: lib.kvq_tree_workspace_bytes(  # noqa: E731
        ctypes.byref(lay.c()), batch, total, hq, maxp, path)
    for batch, total, hq, maxp, fits in ((2048, 100, 8, 4 * 54252, True), (2048, 100, 8, 4 * 54253, False),
                                         (1, 249999999, 8, 8, True), (1, 250000000, 8, 8, False), (2049, 100, 8, 8, False)):
        assert (batch <= 2048 and batch * (2 * (hq // 2) + 1) * 2 * (maxp / 4 + 1) < 2e9 and total * hq < 2e9) == fits
        assert (size(batch, total, hq, maxp, 2) > 0) == fits
        assert size(batch, total, hq, maxp, 0) > 0
