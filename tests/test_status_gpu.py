"""The status word of a call that found several things wrong: the gravest one stays, whichever was written last."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from test_pages_gpu import dev, layout
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


def word(ws):
    return int(ws[:4].view(torch.int32))


def tree_words(d, path):
    """Status words of a call with a bad sequence, with a bad page, and with both."""
    got = []
    for sequence, page in ((True, False), (False, True), (True, True)):
        c = Case(4, 2, d, "fp8_e4m3", [5, 20], [9, 4], seed=3)
        if sequence:
            c.dl[0] = 3                              # fewer tokens than drafted ones
        if page:
            c.table[1, 0] = c.L.num_pages
        _, ws = c.run(path)
        assert kvq.kvq_workspace_status(ws) == -1
        got.append(word(ws))
    return got


@pytest.mark.parametrize("d,path", [(128, 0), (128, 1), (64, 0)])
def test_of_two_reports_the_graver_stays(d, path):
    sequence, page, both = tree_words(d, path)
    assert 0 < page < sequence == both


def test_nothing_is_graver_than_a_wait_that_was_given_up():
    """Its outputs are not valid at all, while the other reports only name what was skipped or refused."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kvq.kvq_wait_probe(ws)
    assert kvq.kvq_workspace_status(ws) == -9
    words = tree_words(128, 0)
    L = layout("d32", 4)
    table, lens, refs = dev([[-1, -1]]), dev([0]), dev([1, 1, 1, 1])
    pws = kvq.alloc_pages_workspace(L, 1, 2)
    for seqs, new, status in (([0], [20], -10), ([1], [20], -1)):
        kvq.kvq_pages_resize(table, lens, refs, dev(seqs), dev(new), pws, L)
        assert kvq.kvq_workspace_status(pws) == status
        words.append(word(pws))
    assert all(0 < w < word(ws) for w in words)
