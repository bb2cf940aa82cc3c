"""What a VocabOps of given maxima allocates, on the host: the operators that it is made for pay for themselves alone.
And on the GPU, that the others' workspace comes with the first call that needs it."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import VocabOps


@pytest.fixture
def made(monkeypatch):
    """The workspaces asked for, over handles that are none."""
    L.build()
    sizes = []
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(L, "lmloss_vocab_create", lambda device, bytes_: sizes.append(bytes_) or None)
    return sizes


def _needed(max_tokens, max_dim, max_rows, max_vocab):
    need = 0
    if max_tokens:
        need = L.lmloss_embedding_workspace(L.lmloss_embedding_args(T=max_tokens, V=max_vocab, D=max_dim, ld_table=max_dim,
                                                                    ld_rows=max_dim, scale=1.0))
    if max_rows:
        need = max(need, L.lmloss_beam_workspace(L.lmloss_beam_args(B=max_rows, K=1, M=L.LMLOSS_MAX_BEAMS, V=max_vocab, ld=max_vocab,
                                                                    dtype=L.LMLOSS_FP32, eos_token=-1)))
    return need


@pytest.mark.parametrize("max_tokens,max_dim,max_rows,max_vocab", [
    (1 << 16, 8192, 1024, 1 << 18), (0, 8192, 8, 1 << 18), (1024, 1 << 20, 1024, 1 << 18), (0, (1 << 20) + 1, 1024, 1 << 18),
    (1024, 1 << 30, 1024, 1000), (0, 64, 1 << 24, 1000), (0, 64, 0, 1000), (0, 0, 4, 1000)])
def test_constructor_takes_what_beams_and_embeddings_need(made, max_tokens, max_dim, max_rows, max_vocab):
    ops = VocabOps(0, max_tokens=max_tokens, max_dim=max_dim, max_rows=max_rows, max_vocab=max_vocab)
    assert made == [_needed(max_tokens, max_dim, max_rows, max_vocab), 0]
    assert (ops.logprobs_workspace_bytes > 0) == (max_rows > 0) and ops.scores_workspace_bytes >= ops.logprobs_workspace_bytes


def test_a_closed_handle_makes_no_calls(made):
    ops = VocabOps(0, max_tokens=0, max_rows=4)
    ops.close()
    a = L.lmloss_logprobs_args(logits=0x10000, T=1, V=1, ld=1, temperature=1.0)
    with pytest.raises(L.LMLossError):
        ops._with_workspace(L.LMLOSS_ERR_INVALID_ARG, ops._logprobs, a, 0, "here", L.lmloss_logprobs_check_args,
                            L.lmloss_logprobs_workspace, 1000)


def test_the_first_call_that_needs_it_asks_once(made, monkeypatch):
    asked, calls = [], []
    monkeypatch.setattr(L, "lmloss_vocab_reserve", lambda handle, bytes_: asked.append(bytes_) or L.LMLOSS_OK)

    def call(handle, args, raw):
        calls.append(1)
        return L.LMLOSS_OK if len(calls) == 1 else L.LMLOSS_ERR_INVALID_ARG
    ops = VocabOps(0, max_tokens=0, max_rows=4)
    a = L.lmloss_logprobs_args(logits=0x10000, T=1, V=1, ld=1, temperature=1.0)
    rest = (call, a, 0, "here", L.lmloss_logprobs_check_args, L.lmloss_logprobs_workspace, ops.logprobs_workspace_bytes)
    with pytest.raises(L.LMLossError):                       # another error asks for nothing
        ops._with_workspace(L.LMLOSS_ERR_CUDA, *rest)
    b = L.lmloss_logprobs_args(logits=0x10000, T=1, V=1, ld=1, temperature=0.0)
    with pytest.raises(L.LMLossError):                       # nor do arguments that no workspace would help
        ops._with_workspace(L.LMLOSS_ERR_INVALID_ARG, call, b, *rest[2:])
    assert not asked and not calls
    ops._with_workspace(L.LMLOSS_ERR_INVALID_ARG, *rest)
    with pytest.raises(L.LMLossError):
        ops._with_workspace(L.LMLOSS_ERR_INVALID_ARG, *rest)
    assert asked == [ops.logprobs_workspace_bytes] and calls == [1]


def test_reserve_refuses(made):
    assert L.lmloss_vocab_reserve(None, 1) == L.LMLOSS_ERR_INVALID_ARG


@pytest.mark.gpu
def test_memory_comes_with_the_first_call_that_needs_it():
    import __graft_entry__
    __graft_entry__.build()
    torch.zeros(1, device="cuda")
    VocabOps(0, max_tokens=0, max_rows=8).close()
    before = torch.cuda.mem_get_info()[0]
    ops = VocabOps(0, max_tokens=1024, max_dim=1 << 20, max_rows=1024)
    assert before - torch.cuda.mem_get_info()[0] < 200 << 20   # not the 4.3 GB of 1024 rows of 2^20 fp32 columns
    t = ops.quantize_table(torch.randn(100, 64, device="cuda"))
    ops.table4_lookup(t, torch.arange(9, device="cuda"))
    ops.table4_logits(t, torch.randn(4, 64, device="cuda"))
    assert not ops._reserved
    z = torch.randn(2, 100000, device="cuda")
    r = ops.token_logprobs(z, num_top=5)
    assert 0 < ops._reserved < 3 << 20 and torch.equal(r.top_tokens, z.sort(dim=1, descending=True, stable=True)[1][:, :5])
    assert before - torch.cuda.mem_get_info()[0] < 200 << 20
    ops.close()
    small = VocabOps(0, max_tokens=0, max_dim=64, max_rows=64, max_vocab=1000)
    y = small.table4_logits(t, torch.randn(40, 64, device="cuda"))
    assert y.shape == (40, 100) and small._reserved == small.scores_workspace_bytes
    small.close()


@pytest.mark.gpu
def test_the_first_call_may_be_captured():
    import __graft_entry__
    __graft_entry__.build()
    a = VocabOps(0, max_tokens=0, max_dim=512, max_rows=64, max_vocab=100000)
    b = VocabOps(0, max_tokens=0, max_dim=512, max_rows=64, max_vocab=100000)
    t = b.quantize_table(torch.randn(2000, 512, device="cuda"))
    x, z = torch.randn(40, 512, device="cuda"), torch.randn(3, 100000, device="cuda")
    tokens = torch.randint(0, 2000, (3, 2), device="cuda")
    b.table4_logits(t, x), b.token_logprobs(z, tokens, num_top=9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, r = a.table4_logits(t, x), a.token_logprobs(z, tokens, num_top=9)
    for seed in range(2):
        x.normal_()
        z.normal_()
        graph.replay()
        torch.cuda.synchronize()
        q, s = b.table4_logits(t, x), b.token_logprobs(z, tokens, num_top=9)
        assert torch.equal(p, q) and torch.equal(r.logp, s.logp) and torch.equal(r.top_tokens, s.top_tokens)
    assert a.device_error() == 0
    a.close(), b.close()


@pytest.mark.gpu
def test_a_graph_keeps_the_workspace_that_it_was_captured_with():
    import __graft_entry__
    __graft_entry__.build()
    handle = L.lmloss_vocab_create(0, 0)
    z = torch.randn(2, 100000, device="cuda")
    lse, again = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")

    def call(out):
        a = L.lmloss_logprobs_args(z.data_ptr(), 2, 100000, 100000, L.LMLOSS_FP32, temperature=1.0, lse_out=out.data_ptr())
        return L.lmloss_logprobs_forward(handle, a, torch.cuda.current_stream().cuda_stream)
    assert call(lse) == L.LMLOSS_ERR_INVALID_ARG             # no workspace yet
    a = L.lmloss_logprobs_args(T=2, V=100000, ld=100000, temperature=1.0)
    assert L.lmloss_vocab_reserve(handle, L.lmloss_logprobs_workspace(a)) == L.LMLOSS_OK
    assert call(lse) == L.LMLOSS_OK
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert call(lse) == L.LMLOSS_OK
    assert L.lmloss_vocab_reserve(handle, 1 << 20) == L.LMLOSS_OK and L.lmloss_vocab_reserve(handle, 0) == L.LMLOSS_OK
    fill = torch.full((1 << 22,), 7.0, device="cuda")        # what another allocation would put in its place
    z.normal_()
    graph.replay()
    assert call(again) == L.LMLOSS_OK
    torch.cuda.synchronize()
    assert torch.equal(lse, again) and bool((fill == 7.0).all())
    assert torch.allclose(lse.double(), torch.logsumexp(z.double(), 1), atol=1e-5)
    assert L.lmloss_vocab_destroy(handle) == L.LMLOSS_OK
