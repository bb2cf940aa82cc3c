"""VocabOps.device_error over its two error words: neither is lost."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import VocabOps


@pytest.mark.parametrize("first", [0, L.LMLOSS_ERR_BAD_PARENT])
@pytest.mark.parametrize("second", [0, L.LMLOSS_ERR_RANGE])
def test_both_words_are_read(monkeypatch, first, second):
    words = {"a": first, "b": second}

    def read(handle):
        code, words[handle] = words[handle], 0
        return code
    monkeypatch.setattr(L, "lmloss_vocab_get_device_error", read)
    ops = VocabOps.__new__(VocabOps)
    ops.handle, ops.scores_handle = "a", "b"
    got = [ops.device_error() for _ in range(3)]
    ops.handle = ops.scores_handle = None
    assert [c for c in got if c] == [c for c in (first, second) if c] and got[2] == 0


@pytest.mark.gpu
def test_errors_of_two_operators():
    import __graft_entry__
    __graft_entry__.build()
    ops = VocabOps(0, max_tokens=0, max_rows=0)
    ops.embedding_forward(torch.randn(5, 8, device="cuda"), torch.tensor([5], device="cuda"))
    ops.quantize_table(torch.full((3, 32), float("inf"), device="cuda"))
    assert {ops.device_error(), ops.device_error()} == {L.LMLOSS_ERR_BAD_TARGET, L.LMLOSS_ERR_RANGE}
    assert ops.device_error() == 0
    ops.close()
