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


# rows of 2-byte logits 208 elements apart, 100 used
@pytest.mark.parametrize("columns,expect", [
    (100, OK), (104, OK), (108, OK), (99, BAD), (109, BAD), (1, BAD), (208, BAD), (416, BAD), (208 + 100, OK), (208 + 108, OK),
    (208 + 99, BAD), (-100, OK), (-108, OK), (-99, BAD), (-109, BAD), (-208 - 104, OK), (3 * 208, OK), (-3 * 208, OK),
])
def test_gradient_beside_the_logits(lib, columns, expect):  # noqa: F811
    assert L.lmloss_logprobs_check_grad_args(_grad(logits=0x10000, ld=208, ld_grad=208, grad_out=0x10000 + 2 * columns)) == expect
    if abs(columns) < 2 * 208:
        assert L.lmloss_logprobs_check_grad_args(_grad(logits=0x10000, ld=208, ld_grad=200, grad_out=0x10000 + 2 * columns)) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V,wide", [(torch.bfloat16, 3001, 6002), (torch.bfloat16, 3000, 6008), (torch.float32, 1000, 2001)])
def test_halves_of_one_tensor(dtype, V, wide):
    import __graft_entry__
    __graft_entry__.build()
    h = VocabOps(0, max_tokens=0, max_rows=64)
    both = torch.randn(9, wide, device="cuda").to(dtype)
    z, d = both[:, :V], both[:, wide - V:]
    tokens, g = torch.randint(0, V, (9, 3), device="cuda"), torch.randn(9, 3, device="cuda")
    r = h.token_logprobs(z, tokens, for_gradient=True)
    alone = z.clone()
    want = h.token_logprobs_backward(alone, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum)
    h.token_logprobs_backward(z, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum, grad=d)
    assert torch.equal(d, want) and torch.equal(z, alone)
    h.close()
