"""The gradient's workspace on the host: what lmloss_embedding_workspace gives for a handle's
largest call has to serve every smaller one.  No GPU needed."""
import pytest

import lm_head_vocab_gb300._lib as L

TYPES = (L.LMLOSS_BF16, L.LMLOSS_FP16, L.LMLOSS_FP32)


@pytest.fixture(scope="module", autouse=True)
def lib():
    L.build()
    return L.load()


def need(T, D, rows=L.LMLOSS_BF16, table=L.LMLOSS_BF16, V=1000):
    return L.lmloss_embedding_workspace(L.lmloss_embedding_args(
        T=T, V=V, D=D, ld_table=D, ld_rows=D, scale=1.0, rows_dtype=rows, table_dtype=table))


def layout(T, D, rows):
    """What a call lays out, from its description: positions and keys twice, digit counts, the
    windows' list and their two fp32 parts, each from a 256-byte boundary."""
    vecs, tpr = (D + 7) // 8, 8
    while tpr < 128 and tpr < vecs:
        tpr *= 2
    ranges, window = -(-vecs // tpr), 32
    while window > 8:
        groups = -(-T // window) * ranges
        if groups >= 600 and groups * tpr // 128 >= (600 if rows == L.LMLOSS_FP32 else 300):
            break
        window //= 2
    windows = -(-T // window)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    return 4 * up(4 * T) + up(4 * 256 * -(-T // 2048)) + up(4 * windows) + up(4 * 2 * windows * 8 * vecs)


WIDTHS = (1, 8, 9, 40, 64, 127, 128, 256, 512, 777, 1000, 1024, 1025, 2048, 3000, 4096, 4097, 8192)
COUNTS = tuple(sorted({1, 1025, 2049, 4097, 65536, 131073} | {m * w + d for m in (60, 75, 150, 299, 300, 599, 600, 1200, 2400, 4800)
                                                             for w in (8, 16, 32) for d in (-1, 0, 1)}))


def test_a_larger_call_needs_no_less():
    for i, D in enumerate(WIDTHS):
        for j, T in enumerate(COUNTS):
            here = need(T, D)
            assert {need(T, D, r, t, V) for r in TYPES for t in TYPES for V in (1, 1 << 20)} == {here}
            if i:
                assert here >= need(T, WIDTHS[i - 1])
            if j:
                assert here >= need(COUNTS[j - 1], D)


@pytest.mark.parametrize("T,D", [(4800, 4096), (8192, 2048), (32768, 1024), (65536, 256), (65536, 128), (20000, 512),
                                 (2048, 8192), (4097, 1001), (131073, 8)])
def test_a_handle_serves_what_is_within_its_maxima(T, D):
    size = need(T, D)
    for rows in TYPES:
        for t in COUNTS + (T,):
            for d in WIDTHS + (D,):
                if t <= T and d <= D:
                    assert layout(t, d, rows) <= size, (t, d, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("most,D,T,dtype", [(4800, 1024, 4096, "bfloat16"), (20000, 512, 19000, "bfloat16"),
                                            (20000, 256, 20000, "float32")])
def test_smaller_calls_and_other_types_on_a_gpu(most, D, T, dtype):
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    ops = VocabOps(0, max_tokens=most, max_dim=max(D, 512), max_rows=0)
    g = torch.Generator(device="cuda").manual_seed(T)
    V = 300
    ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    rows = torch.randint(-4, 5, (T, D), device="cuda", generator=g).to(getattr(torch, dtype))
    total = ops.embedding_backward(rows, ids, torch.empty(V, D, device="cuda"))
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, rows.double())
    assert torch.equal(total.double(), want) and ops.device_error() == 0      # whole numbers: exact
    ops.close()


def test_few_positions_need_none():
    assert need(0, 8192) == need(1, 1) == need(1024, 8192) == 0 < need(1025, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 1000, 1024])
def test_few_positions_without_a_workspace(T):
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import LMLossError, VocabOps
    ops = VocabOps(0, max_tokens=0, max_rows=0)
    assert ops.workspace_bytes == 0
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(0, 40, (T,), device="cuda", generator=g)
    rows = torch.randint(-4, 5, (T, 33), device="cuda", generator=g).float()
    total = ops.embedding_backward(rows, ids, num_embeddings=40)
    assert torch.equal(total, torch.zeros(40, 33, device="cuda").index_add_(0, ids, rows))
    # (the exception is not kept: it would hold this call's tensors)
    with pytest.raises(LMLossError, match=f"status {L.LMLOSS_ERR_INVALID_ARG}"):
        ops.embedding_backward(torch.zeros(1025, 33, device="cuda"), torch.zeros(1025, device="cuda").long(), num_embeddings=40)
    ops.close()
