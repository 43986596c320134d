"""Sizes of kvq_pages_fork and kvq_pages_resize that no launch can have are refused before any (no GPU needed)."""
import ctypes

import pytest

from test_pages_host import EUNSUPPORTED, L, fork, lib, resize  # noqa: F401 (lib: the fixture)

COLS = 65535 * 2048   # columns of a row: a grid's y dimension times a CTA's columns
LIST = 2 ** 31 - 1 - 8192


def layout():
    return L(page_size=1)


@pytest.mark.parametrize("call", [fork, resize])
def test_rows_and_lists_past_a_grid_are_refused(lib, call):  # noqa: F811
    for kw in (dict(maxp=COLS + 1), dict(maxp=2 ** 31 - 1), dict(n=LIST + 1), dict(n=2 ** 31 - 1)):
        assert call(lib, layout(), wb=1 << 62, **kw) == EUNSUPPORTED, kw
    if lib.kvq_device_check() != 0:   # the largest that are taken get as far as the device, which is not there
        for kw in (dict(maxp=COLS), dict(n=LIST)):
            assert call(lib, layout(), wb=1 << 62, **kw) == lib.kvq_device_check(), kw


def test_their_workspaces_have_no_size(lib):  # noqa: F811
    size = lambda n, maxp: lib.kvq_pages_workspace_bytes(ctypes.byref(layout().c()), n, maxp)  # noqa: E731
    assert size(2, COLS) >= 2 * COLS * 4 and size(2, COLS + 1) == 0
    assert size(LIST, 1) >= LIST * 28 and size(LIST + 1, 1) == 0
