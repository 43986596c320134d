"""kvq_pages_resize and kvq_pages_fork over counts that are wrong."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from test_pages_gpu import dev, layout

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["taken", "released"])
def test_a_free_page_that_a_row_lists_is_taken_and_released_at_once(first):
    """Row 1 lists pages that nobody counted; one call lets row 0 take the same pages and frees row 1.  Whichever entry
    runs first (thousands of empty ones lie between the two), the pages are row 0's afterwards, counted once, and the
    wrong counts are reported."""
    k, filler = 40, 5000
    L = layout("d32", 64)
    table = torch.full((filler + 2, k), -1, dtype=torch.int32)
    table[1] = torch.arange(k, dtype=torch.int32)
    table = table.cuda()
    lens = torch.zeros(filler + 2, dtype=torch.int32).cuda()
    lens[1] = k * 16
    refs = torch.zeros(64, dtype=torch.int32).cuda()
    ends = (0, 1) if first == "taken" else (1, 0)
    seqs = [ends[0]] + list(range(2, filler + 2)) + [ends[1]]
    new = torch.zeros(filler + 2, dtype=torch.int32).cuda()
    new[0 if first == "taken" else -1] = k * 16
    ws = kvq.alloc_pages_workspace(L, filler + 2, k)
    kvq.kvq_pages_resize(table, lens, refs, dev(seqs), new, ws, L)
    assert kvq.kvq_workspace_status(ws) == -1
    assert table[0].tolist() == list(range(k)) and (table[1:] == -1).all()
    assert lens[0] == k * 16 and int(lens.sum()) == k * 16
    assert refs.tolist() == [1] * k + [0] * (64 - k)


@pytest.mark.parametrize("first", ["taken", "released"])
def test_a_fork_takes_a_free_page_that_a_replaced_row_lists(first):
    """Row 1's last page goes to a copy for row 2 on page 0, which row 0, itself replaced, lists with a count of 0."""
    filler = 5000
    L = layout("d32", 8)
    table = torch.full((filler + 4, 2), -1, dtype=torch.int32).cuda()
    lens = torch.zeros(filler + 4, dtype=torch.int32).cuda()
    table[0, 0], lens[0] = 0, 16
    table[1, 0], lens[1] = 5, 7
    refs = dev([0, 0, 0, 0, 0, 1, 0, 0])
    take, drop = (1, 2), (3, 0)                      # (parent, child); row 3 is empty
    ends = (take, drop) if first == "taken" else (drop, take)
    pairs = [ends[0]] + [(3, 4 + i) for i in range(filler)] + [ends[1]]
    cs, cd = dev([77] * len(pairs)), dev([77] * len(pairs))
    ws = kvq.alloc_pages_workspace(L, len(pairs), 2)
    kvq.kvq_pages_fork(table, lens, refs, dev([p[0] for p in pairs]), dev([p[1] for p in pairs]), cs, cd, ws, L)
    assert kvq.kvq_workspace_status(ws) == -1
    assert refs.tolist() == [1, 0, 0, 0, 0, 1, 0, 0]
    assert table[2].tolist() == [0, -1] and table[1].tolist() == [5, -1] and (table[0] == -1).all()
    at = 0 if first == "taken" else len(pairs) - 1
    assert (cs[at], cd[at]) == (5, 0) and lens[2] == 7
