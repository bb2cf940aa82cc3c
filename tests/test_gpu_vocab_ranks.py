"""The order of candidates whose scores are divided by a power of their length, on the GPU.

Tolerance, from the arithmetic: scores are off by what a row's logsumexp is off (an exponential
within 2^-22, its argument within 2^-23 relative of up to 64, a chain of at most 40 fp32
additions: under 2^-16 in all), and a power of a length by less than 1e-7 relative where the
penalty is at most 16.  Two candidates may trade places where their true ranks differ by less than
that of either: a difference of scores is divided by the same power as the scores are.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, H, F = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_rows=512)
    yield h
    h.close()


def check(ops, z, s, M, alpha, lengths, finished=None, eos=-1, may=None):
    """Each candidate is one of the row's best, in an order that its exact ranks allow."""
    B, K = s.shape
    V = z.shape[1]
    mask = None
    if may is not None:                                   # [B * K or 1, V] truth values
        bits = torch.zeros(may.shape[0], (V + 31) // 32 * 32, dtype=torch.int64, device="cuda")
        bits[:, :V] = may
        word = (bits.view(may.shape[0], -1, 32) << torch.arange(32, device="cuda")).sum(2)
        mask = torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()
    r = ops.beam_step(z, s, num_candidates=M, lengths=lengths, length_penalty=alpha, finished=finished, eos_token=eos,
                      token_mask=mask)
    assert ops.device_error() == 0
    fin = torch.zeros(B, K, dtype=torch.bool) if finished is None else finished.bool().cpu()
    zd = z.double().cpu().view(B, K, V)
    score = s.double().cpu()[:, :, None] + zd - torch.logsumexp(zd, 2, keepdim=True)
    if may is not None:
        score = torch.where(may.cpu().expand(B * K, V).view(B, K, V), score, -INF)
    if finished is not None:
        stay = torch.full((B, K, V), -INF, dtype=torch.float64)
        stay[:, :, eos] = s.double().cpu()
        score = torch.where(fin[:, :, None], stay, score)
    steps = (lengths.cpu() + (~fin).int()).clamp(min=1).double()
    norm = (steps ** alpha).clamp(max=torch.finfo(torch.float64).max)
    rank = (score / norm[:, :, None]).flatten(1)
    slack = ((2.0 ** -16 + score.abs() * 1e-7) / norm[:, :, None]).flatten(1)
    place = r.parents.cpu().long() * V + r.tokens.cpu()
    for b in range(B):
        n = min(M, int((rank[b] > -INF).sum()))
        got = place[b, :n]
        assert len(set(got.tolist())) == n
        low, high = rank[b] - slack[b], rank[b] + slack[b]
        # none of the chosen could come after a later one, none that was left out before the last
        for m in range(n - 1):
            assert (high[got[m]] >= low[got[m + 1:]]).all(), (b, m)
        out = torch.ones_like(rank[b], dtype=torch.bool)
        out[got] = False
        assert n == 0 or not out.any() or low[out].max() <= high[got].min(), b
        # within a row the order is exact
        for k in range(K):
            mine = got[got // V == k]
            kept = score[b, k].sort(descending=True, stable=True)[1][:len(mine)]
            if not fin[b, k]:
                assert mine.remainder(V).tolist() == kept.tolist()
        assert (r.tokens[b, n:] == -100).all()
    return r


def inputs(B, K, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B * K, V, device="cuda", generator=g) * 3
    s = -40 * torch.rand(B, K, device="cuda", generator=g)
    n = torch.randint(1, 4000, (B, K), device="cuda", generator=g, dtype=torch.int32)
    fin = (torch.rand(B, K, device="cuda", generator=g) < 0.3).to(torch.uint8)
    return z.to(dtype), s, n, fin


def test_powers_past_the_range_of_fp32(ops):
    # 4097^10.7 = 4.5e38: the long beam's rank is -1.333e-36, the short one's -1.317e-36, the better one
    V = 1000
    z = torch.full((2, V), -60.0, device="cuda")
    z[:, 7] = 0.0                                          # one token of probability 1 in each
    s = torch.tensor([[-600.0, -350.0]], device="cuda")
    n = torch.tensor([[4096, 3899]], device="cuda", dtype=torch.int32)
    r = check(ops, z, s, 1, 10.7, n)
    assert r.parents.tolist() == [[1]] and r.tokens.tolist() == [[7]]


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("alpha", [0.3, 1.0, 2.5, 7.9, 8.4, 9.1, 10.7, 12.0, 16.0])
def test_order_of_normalised_scores(ops, dtype, alpha):
    z, s, n, fin = inputs(3, 5, 2500, dtype, int(alpha * 10))
    check(ops, z, s, 10, alpha, n)
    check(ops, z, s, 10, alpha, n, fin, 17)
    g = torch.Generator(device="cuda").manual_seed(1)
    may = torch.rand(15, 2500, device="cuda", generator=g) < 0.1
    may[4] = False                                         # nothing may follow one beam
    check(ops, z, s, 10, alpha, n, fin, 17, may)
    check(ops, z, s, 10, alpha, n, None, -1, may[:1])


@pytest.mark.parametrize("alpha", [85.0, 1e4])
def test_powers_past_the_range_of_fp64(ops, alpha):
    z, s, n, _ = inputs(1, 1, 2500, F, 3)
    check(ops, z, s, 20, alpha, n + 4000)
