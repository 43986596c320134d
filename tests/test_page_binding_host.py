"""What the binding refuses of attention calls over fp8_e4m3_page before the library sees them (no GPU needed: the tensors'
device stands in for the current one)."""
import pytest
import torch

from block_quantized_bit_gb300 import kvq


@pytest.fixture
def call(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)

    def refuse(*a):
        raise AssertionError("reached the library")

    class Library:
        kvq_decode_ex = kvq_extend = kvq_decode_noalloc = staticmethod(refuse)

    monkeypatch.setattr(kvq, "lib", lambda: Library)
    monkeypatch.setattr(kvq, "_stream", lambda s: 0)
    lay = kvq.Layout(6, 16, 2, 128, 128)
    codes, scales = kvq.alloc_pool(lay, "cpu", "fp8_e4m3_page")
    base = dict(q=torch.zeros(3, 4, 128, dtype=torch.bfloat16), pool=codes, scales=scales,
                block_table=torch.zeros(3, 2, dtype=torch.int32), seq_lens=torch.zeros(3, dtype=torch.int32),
                out=torch.zeros(3, 4, 128), workspace=torch.zeros(4096, dtype=torch.uint8), layout=lay, kind="fp8_e4m3_page")
    start = torch.zeros(4, dtype=torch.int32)
    return {"decode": lambda **o: kvq.kvq_decode(**{**base, **o}),
            "extend": lambda **o: kvq.kvq_extend(**{**base, "q_start": start, **o}),
            "noalloc": lambda **o: kvq.kvq_decode_noalloc(**{k: v for k, v in {**base, **o}.items() if k != "workspace"})}


@pytest.mark.parametrize("which", ["decode", "extend", "noalloc"])
def test_wrong_tensors(call, which):
    f = call[which]
    with pytest.raises(AssertionError, match="reached"):
        f()
    with pytest.raises(TypeError, match="q must be"):
        f(q=torch.zeros(3, 4, 128))
    with pytest.raises(ValueError, match="q must be contiguous"):
        f(q=torch.zeros(4, 3, 128, dtype=torch.bfloat16).transpose(0, 1))
    with pytest.raises(TypeError, match="block_table"):
        f(block_table=torch.zeros(3, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="block_table"):
        f(block_table=torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="seq_lens"):
        f(seq_lens=torch.zeros(3))
    with pytest.raises(ValueError, match="q and out"):
        f(out=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError, match="q and out"):
        f(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), out=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError, match="out must be contiguous"):
        f(out=torch.zeros(4, 3, 128).transpose(0, 1))
    with pytest.raises(TypeError, match="scales"):
        f(scales=None)
    with pytest.raises(ValueError, match="pool"):
        f(pool=torch.zeros(100, dtype=torch.uint8))


def test_rows_and_sequences_that_do_not_agree(call):
    rows = dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16), out=torch.zeros(2, 4, 128))
    with pytest.raises(ValueError, match="one row"):
        call["decode"](**rows)
    with pytest.raises(ValueError, match="one row"):
        call["noalloc"](**rows)
    with pytest.raises(ValueError, match="q_start"):
        call["extend"](q_start=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="q_start"):
        call["extend"](q_start=torch.zeros(4, dtype=torch.int64))
