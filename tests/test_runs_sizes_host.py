"""Sizes that do not fit the C calls' 32-bit arguments are refused by the
wrappers of the several-sequence operators: ctypes would drop their upper bits
without a word.  No GPU needed."""
import pytest

from prefill_kv_shared_gb300 import binding

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("run", [(1 << 32, 0, 0), ((1 << 32) + 4, 0, 0), (4, 1 << 32, 0), (4, 0, 1 << 31),
                                 (4, 0, (1 << 32) + 7), (4, -(1 << 33), 0), (1 << 70, 0, 0)])
def test_run_fields(run):
    with pytest.raises(ValueError, match="32 bits"):
        binding.AttnRuns([(1, 0, 0), run], 8, 2, 64)


@pytest.mark.parametrize("heads", [((1 << 32) + 8, 2, 64), (8, (1 << 32) + 2, 64), (8, 2, (1 << 32) + 64)])
def test_heads(heads):
    with pytest.raises(ValueError, match="32 bits"):
        binding.AttnRuns([(1, 0, 0)], *heads)


@pytest.mark.parametrize("rows,vocab", [((1 << 32) + 3, 1), (1 << 31, 1), (1, (1 << 32) + 5), (1, 1 << 31)])
def test_rows_and_vocabulary(rows, vocab):
    logits = torch.zeros(1, 1, dtype=torch.bfloat16).expand(rows, vocab)  # no memory behind it
    if vocab > 1:
        logits = torch.empty(0, dtype=torch.bfloat16, device="meta").new_empty(rows, vocab)
    with pytest.raises(ValueError, match="32 bits"):
        binding.logprobs(logits)


def test_mask_words():
    runs = object.__new__(binding.AttnRuns)  # the sizes are looked at before anything else
    runs.n_rows = 1
    mask = torch.empty(1, (1 << 32) + 1, dtype=torch.int64, device="meta")
    with pytest.raises(ValueError, match="words"):
        binding.attention_tree(None, None, None, runs, mask, None)
