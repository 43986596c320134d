"""kvq_pages_resize whose entries ask for more pages in all than 32 bits count: refused, and nothing is changed."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from test_pages_gpu import layout

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [4096, 8192, 8193])       # 2^31, 2^32 and 2^32 + 2^19 pages asked for
def test_a_demand_past_32_bits_finds_too_few_pages(rows):
    cols, pages = 1 << 19, 600000
    L = layout("d32", pages)
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[:50] = 2
    held = refs.clone()
    new = torch.full((rows,), cols * 16, dtype=torch.int32, device="cuda")
    ws = kvq.alloc_pages_workspace(L, rows, cols)
    kvq.kvq_pages_resize(table, lens, refs, torch.arange(rows, dtype=torch.int32, device="cuda"), new, ws, L)
    assert kvq.kvq_workspace_status(ws) == -10
    assert torch.equal(refs, held) and int(lens.abs().sum()) == 0
    for part in table.split(512):
        assert (part == -1).all()
