"""What VocabOps checks before it calls the library, on the host: the calls stop before any kernel."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import VocabOps


@pytest.fixture(scope="module")
def ops():
    L.build()
    L.load()
    h = VocabOps.__new__(VocabOps)      # no handle: tensors on the host, the library's own checks only
    h.device, h._index, h.handle, h.workspace_bytes = torch.device("cpu"), -1, None, 0
    return h


def test_views_that_stand_for_other_values_are_refused(ops):
    # a conjugated or negated view holds the bytes of what it was made from
    x = torch.randn(6, 4, dtype=torch.complex64)
    plain = torch.empty(6, 4, dtype=torch.complex64)
    for t, o in ((x.conj(), plain), (plain, x.conj()), (x.conj().imag, torch.empty(6, 4)), (x.real, x.conj().imag)):
        assert t.is_conj() or t.is_neg() or o.is_conj() or o.is_neg()
        with pytest.raises(ValueError, match="conjugate"):
            ops._describe(t, o, 0, 6, 6)
    ops._describe(x.conj(), x.conj(), 0, 6, 6)                   # moved as they are
    ops._describe(x, plain, 0, 6, 6)
    with pytest.raises(ValueError, match="conjugate"):
        ops.embedding_forward(torch.view_as_complex(torch.randn(6, 4, 2)).conj().imag, torch.zeros(3, dtype=torch.int64))


def test_a_workspace_that_is_too_small_is_named(ops):
    a = L.lmloss_embedding_args(ids=0x10000, T=5000, V=10, D=16, table=0x20000, ld_table=16, rows=0x30000, ld_rows=16, scale=1.0)
    need = L.lmloss_embedding_workspace(a)
    e = ops._refused(L.LMLOSS_ERR_INVALID_ARG, "here", a, L.lmloss_embedding_check_args, L.lmloss_embedding_workspace)
    assert e.status == L.LMLOSS_ERR_INVALID_ARG and f"{need} bytes" in str(e) and "0 there" in str(e) and "max_tokens" in str(e)
    # other reasons, and other errors, are left as they are
    a.scale = float("nan")
    e = ops._refused(L.LMLOSS_ERR_INVALID_ARG, "here", a, L.lmloss_embedding_check_args, L.lmloss_embedding_workspace)
    assert e.status == L.LMLOSS_ERR_INVALID_ARG and "bytes" not in str(e)
    a.scale = 1.0
    e = ops._refused(L.LMLOSS_ERR_CUDA, "here", a, L.lmloss_embedding_check_args, L.lmloss_embedding_workspace)
    assert e.status == L.LMLOSS_ERR_CUDA and "bytes" not in str(e)


def test_positions_without_one_row_stride_are_a_value_error(ops, monkeypatch):
    monkeypatch.setattr("lm_head_vocab_gb300.vocab._raw_stream", lambda index: 0)
    ids = torch.zeros(2, 4, dtype=torch.int64)
    whole = torch.randn(2, 5, 8)
    with pytest.raises(ValueError, match="one row stride"):
        ops.embedding_backward(whole[:, :-1], ids, torch.zeros(9, 8))
    with pytest.raises(ValueError, match="one row stride"):
        ops.embedding_forward(torch.randn(9, 8), ids, out=whole[:, :-1])


@pytest.mark.gpu
def test_a_call_past_the_handle_says_so():
    import __graft_entry__
    __graft_entry__.build()
    h = VocabOps(0, max_tokens=2000, max_dim=64, max_rows=2, max_vocab=1000)
    with pytest.raises(L.LMLossError, match="bytes of workspace needed"):
        h.embedding_backward(torch.zeros(200000, 64, device="cuda"), torch.zeros(200000, device="cuda").long(), num_embeddings=3)
    with pytest.raises(L.LMLossError, match="bytes of workspace needed"):
        h.beam_step(torch.zeros(64, 100000, device="cuda"), torch.zeros(16, 4, device="cuda"), num_candidates=64)
    with pytest.raises(L.LMLossError, match=r"invalid argument \(status 1\)"):
        h.beam_step(torch.zeros(2, 100, device="cuda"), torch.zeros(1, 2, device="cuda"), eos_token=100)
    h.close()
