"""The parts of lse that the gradient of log-probabilities takes: what is refused, on the host.  No GPU needed."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import VocabOps
from tests.test_vocab_logprobs_abi import BAD, OK, _grad, lib, ops  # noqa: F401


@pytest.mark.parametrize("kw,expect", [
    ({"row_max": 0x60000, "log_sum": 0x70000}, OK), ({"row_max": 0x60000}, BAD), ({"log_sum": 0x70000}, BAD),
    ({"lse": None, "row_max": 0x60000, "log_sum": 0x70000}, OK), ({"lse": None, "log_sum": 0x70000}, BAD),
])
def test_both_parts_or_neither(lib, kw, expect):  # noqa: F811
    assert L.lmloss_logprobs_check_grad_args(_grad(**kw)) == expect


def test_wrapper_refuses(ops, monkeypatch):  # noqa: F811
    monkeypatch.setattr("lm_head_vocab_gb300.vocab._raw_stream", lambda index: 0)
    z, lse = torch.zeros(3, 40), torch.zeros(3)
    for error, kw in [(ValueError, dict()), (ValueError, dict(row_max=lse)), (ValueError, dict(log_sum=lse)),
                      (ValueError, dict(lse=lse, row_max=lse)), (ValueError, dict(row_max=lse[:2], log_sum=lse)),
                      (TypeError, dict(row_max=lse.half(), log_sum=lse)), (TypeError, dict(row_max=lse, log_sum=lse.double()))]:
        with pytest.raises(error):
            VocabOps.token_logprobs_backward(ops, z, **kw)


def test_they_are_made_on_request(ops, monkeypatch):  # noqa: F811
    monkeypatch.setattr("lm_head_vocab_gb300.vocab._raw_stream", lambda index: 0)
    seen = []
    monkeypatch.setattr(VocabOps, "_logprobs", staticmethod(lambda handle, a, raw: seen.append((a.row_max_out, a.log_sum_out)) or OK), raising=False)
    monkeypatch.setattr(VocabOps, "scores_handle", None, raising=False)
    r = ops.token_logprobs(torch.zeros(3, 40))
    assert r.row_max is None and r.log_sum is None and seen == [(None, None)]
    r = ops.token_logprobs(torch.zeros(3, 40), for_gradient=True)
    assert seen[1] == (r.row_max.data_ptr(), r.log_sum.data_ptr()) and r.row_max.shape == r.log_sum.shape == (3,)
