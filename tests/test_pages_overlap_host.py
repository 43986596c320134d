"""kvq_pages_compact refuses a result that overlaps what the call still reads (no GPU needed)."""
import pytest

from test_pages_host import EINVAL, L, compact, lib  # noqa: F401 (lib: the fixture)

BATCH, MAXP, WORDS, PAGES = 6, 8, 2, 10
AT = dict(table=0x10000, lens=0x20000, start=0x30000, keep=0x40000, refs=0x50000)
BYTES = dict(table=BATCH * MAXP * 4, lens=BATCH * 4, start=(BATCH + 1) * 4, keep=BATCH * WORDS * 8, refs=PAGES * 4)


def call(lib, new, **kw):  # noqa: F811
    return compact(lib, L(num_pages=PAGES), batch=BATCH, words=WORDS, maxp=MAXP, new=new, **{**AT, **kw})


@pytest.mark.parametrize("name", list(AT))
def test_new_lens_may_not_overlap_an_input(lib, name):  # noqa: F811
    at, end = AT[name], AT[name] + BYTES[name]
    for new in (at, at + 4, end - 4, at - BATCH * 4 + 4):
        assert call(lib, new) == EINVAL, hex(new)
    # right before and right behind: nothing to refuse (the call then gets as far as the device, which is not there)
    if lib.kvq_device_check() != 0:
        for new in (at - BATCH * 4, end):
            assert call(lib, new) == lib.kvq_device_check(), hex(new)


def test_without_counts_there_is_nothing_to_overlap(lib):  # noqa: F811
    if lib.kvq_device_check() != 0:
        assert call(lib, 0x50000, refs=0) == lib.kvq_device_check()
