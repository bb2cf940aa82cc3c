"""What workspace the logits of 4-bit tables ask of a handle: none for a decoding step's few rows, what the header says for
more, and a call that lacks it is refused before it writes anything."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L

pytestmark = pytest.mark.gpu

BF, H, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def big():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_dim=8192, max_rows=512)
    yield h
    h.close()


def raw_logits(handle, big, t, x, out):
    a = L.lmloss_table4_logits_args(big._table4(t), x.data_ptr(), len(x), x.stride(0), out.data_ptr(), out.stride(0),
                                    {BF: 0, F: 1, H: 2}[x.dtype], {BF: 0, F: 1, H: 2}[out.dtype], 1.0)
    return L.lmloss_table4_logits(handle, a, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("group,scales,zeros", [(32, F, True), (64, BF, False), (128, H, True)])
@pytest.mark.parametrize("D", [1, 100, 1001, 4096, 6144])
def test_few_rows_need_none(big, group, scales, zeros, D):
    w = torch.randn(300, D, device="cuda")
    t = big.quantize_table(w, group_size=group, zeros=zeros, scale_dtype=scales)
    handle = L.lmloss_vocab_create(0, 0)
    try:
        for T, x, o in ((1, BF, BF), (8, BF, BF), (8, H, H), (1, F, F), (4, F, F), (4, BF, F), (4, F, BF)):
            rows = torch.randn(T, D, device="cuda").to(x)
            out = torch.empty(T, 300, device="cuda", dtype=o)
            assert raw_logits(handle, big, t, rows, out) == L.LMLOSS_OK
            assert torch.equal(out, big.table4_logits(t, rows, out_dtype=o))
        assert L.lmloss_vocab_get_device_error(handle) == 0
    finally:
        L.lmloss_vocab_destroy(handle)


@pytest.mark.parametrize("x,T", [(BF, 9), (F, 5), (BF, 128), (F, 64), (BF, 129), (H, 1500)])
def test_more_rows_need_what_is_said(big, x, T):
    D = 700
    t = big.quantize_table(torch.randn(300, D, device="cuda"), group_size=64)
    a = L.lmloss_table4_logits_args(T=T)
    a.table.V, a.table.D, a.table.group = 300, D, 64
    need = L.lmloss_table4_logits_workspace(a)
    rows = torch.randn(T, D, device="cuda").to(x)
    out = torch.full((T, 300), 5.0, device="cuda", dtype=x)
    small, enough = L.lmloss_vocab_create(0, 0), L.lmloss_vocab_create(0, need)
    try:
        assert raw_logits(small, big, t, rows, out) == L.LMLOSS_ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert bool((out == 5.0).all())                      # nothing was launched
        assert raw_logits(enough, big, t, rows, out) == L.LMLOSS_OK
        assert torch.equal(out, big.table4_logits(t, rows))
    finally:
        L.lmloss_vocab_destroy(small)
        L.lmloss_vocab_destroy(enough)


@pytest.mark.parametrize("x", [BF, F])
def test_a_wrapper_past_its_maxima_says_so(big, x):
    # up to the handle's rows, whatever the type; one block of operand rows more is refused
    from lm_head_vocab_gb300 import VocabOps
    D, most = 8192, 256
    h = VocabOps(0, max_tokens=0, max_dim=D, max_rows=most, max_vocab=1000)
    t = h.quantize_table(torch.randn(100, D, device="cuda"))
    rows = torch.randn(most + 300, D, device="cuda").to(x)
    assert torch.equal(h.table4_logits(t, rows[:most]), big.table4_logits(t, rows[:most]))
    past = most + 1 if x is F else 2 * most + 1              # a pair is two operand rows
    with pytest.raises(L.LMLossError, match="bytes of workspace needed"):
        h.table4_logits(t, rows[:past])
    assert h.device_error() == 0
    h.close()


@pytest.mark.parametrize("x", [BF, H, F])
@pytest.mark.parametrize("T", [2, 8, 16, 40, 100, 300])
def test_a_row_by_its_place_alone(big, x, T):
    # the other rows' values do not matter, nor what the workspace held
    t = big.quantize_table(torch.randn(700, 512, device="cuda"), group_size=64, zeros=True)
    rows = torch.randn(T, 512, device="cuda").to(x)
    want = big.table4_logits(t, rows, out_dtype=F)
    for keep in {0, T // 2, T - 1}:
        others = (torch.randn(T, 512, device="cuda") * 100).to(x)
        others[keep] = rows[keep]
        assert torch.equal(big.table4_logits(t, others, out_dtype=F)[keep], want[keep])
