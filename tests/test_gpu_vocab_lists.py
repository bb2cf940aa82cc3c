"""Sequences whose rows are cut into more parts than a block has threads: the last block picks from
several lists a thread, and by rounds where more candidates tie than it can hold."""
import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_ranks import BF, F, H, check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_rows=64)
    yield h
    h.close()


SHAPES = [(16, 16, 151936), (20, 40, 128256), (64, 64, 262144)]


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("K,M,V", SHAPES)
def test_more_lists_than_threads(ops, dtype, K, M, V):
    z, s, n, fin = inputs(1, K, V, dtype, K)
    check(ops, z, s, M, 0.0, n)
    check(ops, z, s, M, 0.7, n, fin, 17)
    # the best candidates all in one row's last columns, then one in each row
    z[K - 1, -M:] = torch.linspace(30, 31, M, device="cuda").to(dtype)
    check(ops, z, s, M, 0.0, n)
    z[:, V // 3] = 40.0
    check(ops, z, s, M, 1.0, n)


@pytest.mark.parametrize("K,M,V", SHAPES)
@pytest.mark.parametrize("levels", [1, 3])
def test_more_ties_than_are_held(ops, K, M, V, levels):
    # rows with the same bits and beams with the same score: equal candidates by beam, then by token
    g = torch.Generator(device="cuda").manual_seed(V)
    row = torch.randint(0, levels, (V,), device="cuda", generator=g).to(BF)
    z, s = row.expand(K, V).contiguous(), torch.full((1, K), -3.0, device="cuda")
    r = ops.beam_step(z, s, num_candidates=M)
    top = np.nonzero(row.float().cpu().numpy() == levels - 1)[0]
    assert len(top) > M and ops.device_error() == 0
    assert r.parents[0].tolist() == [0] * M and r.tokens[0].tolist() == top[:M].tolist()
    # the same ties in the later beams only, beside ended ones that are better and worse
    s[0, :K // 2] = -100.0
    fin = torch.zeros(1, K, dtype=torch.uint8, device="cuda")
    fin[0, 0] = fin[0, K - 1] = 1
    s[0, 0], s[0, K - 1] = -0.5, -99.0
    lengths = torch.full((1, K), 7, device="cuda", dtype=torch.int32)
    lengths[0, 0] = lengths[0, K - 1] = 8
    r = ops.beam_step(z, s, num_candidates=M, finished=fin, eos_token=5, lengths=lengths, length_penalty=0.6)
    assert r.parents[0].tolist() == [0] + [K // 2] * (M - 1)
    assert r.tokens[0].tolist() == [5] + top[:M - 1].tolist()
    assert r.finished[0].tolist() == [1] + [int(t == 5) for t in top[:M - 1]]
    assert r.lengths[0].tolist() == [8] * M and ops.device_error() == 0
