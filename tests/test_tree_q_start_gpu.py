"""kvq_tree where single entries of q_start are wrong: the sequences that they spoil are skipped and reported, and the
others, whose contexts are cut into several segments, come out as if the spoilt ones were not there."""
import pytest

from block_quantized_bit_gb300 import kvq

from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,path", [(8, 2, 128, 0), (16, 2, 256, 0), (4, 2, 64, 0), (8, 2, 128, 1)])
@pytest.mark.parametrize("ctx,drafted,wrong,skipped", [
    ([30, 40, 9000], [2, 2, 4], {1: 20}, (0, 1)),              # past the end, behind it a valid long sequence
    ([9000, 40, 50, 7000], [3, 3, 2, 3], {2: -1}, (1, 2)),     # negative, valid ones on both sides
    ([8000, 40, 9000], [5, 2, 4], {2: 0}, (1, 2)),             # falls back to the start: sequence 2 has 11 drafts of 4
])
def test_a_wrong_entry_spoils_only_its_neighbours(ctx, drafted, wrong, skipped, hq, hkv, d, path):
    c = Case(hq, hkv, d, "fp8_e4m3", ctx, drafted, seed=d + len(ctx))
    for at, x in wrong.items():
        c.ds[at] = x
    if wrong == {2: 0}:
        c.dl[2] = 10                                           # fewer tokens than the 11 drafts it now claims
    out, ws = c.run(path)
    assert kvq.kvq_workspace_status(ws) == -1
    c.check(out, tensor=path == 0 and d != 64, skipped=skipped)
