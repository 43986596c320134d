"""kvq_tree and kvq_prompt where running maxima move late, more than once, and for different rows at different keys: O
and the row sums are then rescaled inside a segment.  Tolerances as in test_tree_gpu.py and test_prompt_gpu.py: the keys
planted here are a row's own q times at most 24, so sum |q_i k_i| stays below 64 (|q|^2 is about 1, at most 1.7 of the
rows drawn here)."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq

from test_prompt_gpu import check, inputs, run
from test_tree_gpu import PAGE, Case

pytestmark = pytest.mark.gpu

STEPS = (11.0, 17.5, 24.0)   # scores that a row meets one after the other; 8 log2 units are 5.55


@pytest.mark.parametrize("kind", ["fp8_e4m3", "q8_0"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 256)])
def test_rows_of_drafts_rescale_at_their_own_tiles(hq, hkv, d, kind):
    ctx, drafted = [24000, 31000, 27001], [16, 11, 24]
    c = Case(hq, hkv, d, kind, ctx, drafted, seed=d)
    g, tile = hq // hkv, 128 if d == 128 else 64
    units = sum(-(-n * g // 128) * hkv * -(-x // tile) for n, x in zip(drafted, c.lens))
    assert units > 6 * torch.cuda.get_device_properties(0).multi_processor_count
    k, v, slots = [], [], []
    gen = torch.Generator(device="cuda").manual_seed(1)
    for b, n in enumerate(drafted):
        rows = n * g
        for step, size in enumerate(STEPS):
            for r in range(rows):
                # a key of its own for each row and step, the steps in three thirds of the context: every tile or two
                # moves another row's maximum, and a segment has six tiles and more
                p = int(ctx[b] * (step + (r + 0.5) / rows) / 3)
                row = c.start[b] + r // g
                heads = [h * g + r % g for h in range(hkv)]
                q = c.q[row, heads].float()
                k.append(q * (size / q.square().sum(-1, keepdim=True)))
                v.append(torch.randn(hkv, d, generator=gen, device="cuda"))
                slots.append(int(c.table[b, p // PAGE]) * PAGE + p % PAGE)
    kvq.kvq_store(c.codes, c.scales, torch.stack(k).to(torch.bfloat16), torch.stack(v).to(torch.bfloat16),
                  torch.tensor(slots, dtype=torch.int64).cuda(), c.L, kind)
    assert float(c.q[:c.start[-1]].float().square().sum(-1).max()) < 1.7
    for dtype in (torch.float32, torch.bfloat16):
        out, ws = c.run(dtype=dtype)
        assert kvq.kvq_workspace_status(ws) == 0
        c.check(out, dtype)
        again, _ = c.run(dtype=dtype)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 64), (8, 2, 256), (3, 1, 128)])
def test_rows_of_prompts_rescale_at_their_own_tiles(hq, hkv, d):
    lens = [2500, 700, 1300]
    q, k, v, start = inputs(lens, hq, hkv, d, seed=d + hq)
    g, scale = hq // hkv, d ** -0.5
    for b, n in enumerate(lens):
        for step, size in enumerate(STEPS):
            for i in range(40):
                # row n - 1 - i of the sequence meets its keys in rising order, each in another key tile
                p, row = start[b] + int(n * (0.1 + 0.25 * step) + i * 5), start[b] + n - 1 - i
                x = q[row, [h * g + i % g for h in range(hkv)]].float()
                k[p] = (x * (size / (scale * x.square().sum(-1, keepdim=True)))).to(torch.bfloat16)
    out, ws = run(q, k, v, start)
    assert kvq.kvq_workspace_status(ws) == 0
    check(out, q, k, v, start)
    again, _ = run(q, k, v, start)
    assert torch.equal(out.view(torch.int32), again.view(torch.int32))
