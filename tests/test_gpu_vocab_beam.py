"""Beam search's step and the reordering of beam states on the GPU, against fp64 on
the host.

Tolerance of a row's logsumexp, from the arithmetic: each exponential is within
2^-22 (ex2.approx) and its argument, a logit times log2 e less the row's largest,
within 2^-23 relative of fp32 rounding and of log2 e's own (E = the mean |argument|
under the softmax); a chain of at most 40 fp32 additions per slice; the result
rounded to fp32.  Scores are the sum of that with exact terms, rounded to fp32.
Candidates of one row are ordered exactly; candidates of different rows whose true
scores are closer than twice that tolerance may trade places.
"""
import itertools

import numpy as np
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
    h = VocabOps(0, max_tokens=0, max_rows=1024)
    yield h
    h.close()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def reference(logits, scores, M, finished, eos, lengths, alpha, mask):
    """Per sequence: the sorted candidates (rank key, k, v, score), and each row's lse and tolerance."""
    z = logits.double().cpu().numpy()
    sc = scores.double().cpu().numpy()
    B, K = sc.shape
    V = z.shape[1]
    fin = np.zeros((B, K), bool) if finished is None else finished.cpu().numpy().astype(bool)
    ln = None if lengths is None else lengths.cpu().numpy().astype(np.float64)
    may = None
    if mask is not None:
        may = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :V].astype(bool)
        may = np.broadcast_to(may, (B * K, V))
    with np.errstate(all="ignore"):
        top = z.max(1, keepdims=True)
        e = np.exp(z - np.where(np.isfinite(top), top, 0))
        tot = e.sum(1, keepdims=True)
        lse = (np.where(np.isfinite(top), top, 0) + np.log(tot))[:, 0]
        lse[np.isnan(z).any(1) | (z == INF).any(1)] = np.nan
        arg = np.where(e > 0, (np.where(np.isfinite(top), top, 0) - z) * 1.4426950408889634, 0)
        E = (e / tot * np.abs(arg)).sum(1)
        tol = 2.0 ** -22 + 40 * 2.0 ** -24 + 2.0 ** -23 * (E + 1)
        tol[~np.isfinite(tol)] = 0
    lists = []
    for b in range(B):
        c = []
        for k in range(K):
            r = b * K + k
            norm = 1.0 if ln is None else max(1.0, ln[b, k] + (not fin[b, k])) ** alpha
            if fin[b, k]:
                if np.isfinite(sc[b, k]):
                    c.append((sc[b, k] / norm, k, eos, sc[b, k]))
                continue
            if not np.isfinite(sc[b, k]) or not np.isfinite(lse[r]):
                continue
            ok = np.isfinite(z[r])
            if may is not None:
                ok = ok & may[r]
            v = np.nonzero(ok)[0]
            v = v[np.lexsort((v, -z[r, v]))][:M]
            c += [((sc[b, k] + z[r, x] - lse[r]) / norm, k, int(x), sc[b, k] + z[r, x] - lse[r]) for x in v]
        c.sort(key=lambda t: (-t[0], t[1], t[2]))
        lists.append(c)
    return lists, lse.reshape(B, K), tol.reshape(B, K), fin, ln


def check(ops, logits, scores, *, M, finished=None, eos=-1, lengths=None, alpha=0.0, mask=None):
    r = ops.beam_step(logits, scores, num_candidates=M, finished=finished, eos_token=eos, lengths=lengths,
                      length_penalty=alpha, token_mask=mask)
    assert ops.device_error() == 0
    lists, lse, tol, fin, ln = reference(logits, scores, M, finished, eos, lengths, alpha, mask)
    B, K = scores.shape
    S, P, T, L = (x.cpu().numpy() for x in (r.scores, r.parents, r.tokens, r.lse))
    fo = r.finished.cpu().numpy()
    lo = None if lengths is None else r.lengths.cpu().numpy()
    for b in range(B):
        for k in range(K):
            if fin[b, k]:
                assert L[b, k] == 0
            elif np.isnan(lse[b, k]):
                assert np.isnan(L[b, k])
            elif np.isinf(lse[b, k]):
                assert L[b, k] == lse[b, k]
            else:
                assert abs(L[b, k] - lse[b, k]) <= tol[b, k] + 2.0 ** -24 * abs(lse[b, k]), (b, k, L[b, k], lse[b, k])
        c = lists[b]
        by = {(k, v): (key, s) for key, k, v, s in c}
        n = min(M, len(c))
        got = [(int(P[b, m]), int(T[b, m])) for m in range(n)]
        assert len(set(got)) == n
        t = 2 * tol[b].max()
        for m in range(n):
            key, s = by[got[m]]                 # a candidate of the reference
            k = got[m][0]
            assert abs(S[b, m] - s) <= (0 if fin[b, k] else tol[b, k]) + 2.0 ** -24 * abs(s) + 1e-45, (b, m, S[b, m], s)
            assert abs(key - c[m][0]) <= t
            if not any(abs(c[m][0] - x[0]) <= t and x[1] != c[m][1] for x in c):
                assert got[m] == (c[m][1], c[m][2]), (b, m, got[m], c[m])
            assert fo[b, m] == (fin[b, k] or got[m][1] == eos)
            if lo is not None:
                assert lo[b, m] == ln[b, k] + (not fin[b, k])
        for k in range(K):                      # within a row: exact, ties by the lower token
            assert [v for kk, v in got if kk == k] == [v for _, kk, v, _ in c if kk == k][:sum(kk == k for kk, _ in got)]
        for m in range(n, M):                   # nothing left
            assert S[b, m] == -INF and T[b, m] == -100 and P[b, m] == m % K and fo[b, m] == 0
            if lo is not None:
                assert lo[b, m] == ln[b, m % K]
    return r


def inputs(B, K, V, dtype, seed, std=3.0):
    g = gen(seed)
    z = torch.randn(B * K, V, device="cuda", generator=g) * std
    z[:, :: max(1, V // 7)] += 5
    scores = -10 * torch.rand(B, K, device="cuda", generator=g)
    return z.to(dtype), scores


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("B,K,M,V", [
    (1, 1, 1, 1), (1, 1, 3, 2), (2, 3, 5, 31), (1, 1, 64, 40), (3, 4, 4, 1000), (2, 5, 10, 2047), (1, 4, 8, 2048),
    (2, 2, 64, 2049), (1, 3, 33, 4099), (1, 64, 64, 515), (2, 8, 16, 32003), (5, 7, 14, 16384), (1, 1, 64, 128256),
    (40, 8, 16, 17000)])
def test_step(ops, dtype, B, K, M, V):
    z, s = inputs(B, K, V, dtype, V + M)
    check(ops, z, s, M=M)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,K,M,V", [(3, 4, 8, 1000), (2, 6, 12, 9001), (1, 2, 5, 70)])
@pytest.mark.parametrize("per_row", [False, True])
def test_masks_lengths_and_finished(ops, dtype, B, K, M, V, per_row):
    g = gen(V)
    z, s = inputs(B, K, V, dtype, V)
    fin = (torch.rand(B, K, device="cuda", generator=g) < 0.3).to(torch.uint8)
    ln = torch.randint(0, 50, (B, K), device="cuda", generator=g, dtype=torch.int32)
    words = (V + 31) // 32
    mask = torch.randint(-2 ** 31, 2 ** 31, (B * K if per_row else 1, words), device="cuda", generator=g).int()
    if per_row:
        mask[0] = 0                                   # nothing may follow beam 0
        mask[1] = 0
        mask[1, (V - 1) // 32] = torch.tensor(1 << ((V - 1) % 32), device="cuda").int()   # only the last token
    for alpha in (0.0, 0.6, 1.0, 2.5):
        check(ops, z, s, M=M, finished=fin, eos=V // 2, lengths=ln, alpha=alpha, mask=mask)
    check(ops, z, s, M=M, mask=mask)
    check(ops, z, s, M=M, finished=fin, eos=0)
    check(ops, z, s, M=M, finished=torch.ones_like(fin), eos=V - 1)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("V", [40007, 40008])
@pytest.mark.parametrize("kind", ["lowest", "late", "few", "one late"])
def test_masks_over_long_rows(ops, dtype, V, kind):
    """The allowed logits lie far below the others, or come long after the first ones: rows that
    one block reads alone, in several tiles."""
    B, K, M = 57, 8, 12
    z, s = inputs(B, K, V, dtype, V)
    c = torch.arange(V, device="cuda")
    if kind == "lowest":
        may = (z < -6) & (c % 8 != 3)
    elif kind == "late":
        may = ((c > V - 500) & (c % 2 == 0)).expand(B * K, V)
    elif kind == "few":
        may = ((c % 997 == 0) & (c > 9000)).expand(B * K, V)
    else:
        may = (c == V - 2).expand(B * K, V).clone()
        may[::3, 5] = True
        may[1::5] = False
    words = (V + 31) // 32
    bits = torch.zeros(B * K, words * 32, device="cuda", dtype=torch.int64)
    bits[:, :V] = may
    word = (bits.view(B * K, words, 32) << torch.arange(32, device="cuda")).sum(2)
    mask = torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()
    check(ops, z, s, M=M, mask=mask)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("V", [7, 513, 2048, 16384, 40000])
@pytest.mark.parametrize("M", [1, 8, 64])
@pytest.mark.parametrize("kind", ["constant", "few", "up", "down", "one_thread", "zeros"])
def test_orders_and_ties(ops, dtype, V, M, kind):
    # every candidate equal; a few levels; the best ones side by side; signed zeros
    g = gen(V + M)
    v = torch.arange(V, device="cuda", dtype=torch.float32)
    if kind == "constant":
        row = torch.full((V,), 1.25, device="cuda")
    elif kind == "few":
        row = torch.randint(0, 3, (V,), device="cuda", generator=g).float()
    elif kind == "up":
        row = v / V * 8
    elif kind == "down":
        row = -v / V * 8
    elif kind == "one_thread":       # the best ones a block's stride apart
        row = torch.where(v % 2048 < 8, 5.0, 0.0) + torch.where(v % 1024 < 4, 2.0, 0.0)
    else:
        row = torch.where(v % 3 == 0, -0.0, 0.0)
    z = torch.stack([row, row.flip(0), row]).to(dtype)
    check(ops, z, torch.tensor([[-1.0, -1.5, -3.0]], device="cuda"), M=M)
    # beams that are the same in everything: by beam, then by token
    same = torch.stack([row, row]).to(dtype)
    r = check(ops, same, torch.full((1, 2), -2.0, device="cuda"), M=M)
    full = torch.cat([same[0], same[1]]).double().cpu().numpy()
    order = np.lexsort((np.arange(2 * V), -full))[:M]
    n = len(order)
    assert r.parents[0, :n].tolist() == (order // V).tolist() and r.tokens[0, :n].tolist() == (order % V).tolist()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [100, 5000])
def test_rows_without_candidates(ops, dtype, V):
    B, K, M = 4, 4, 6
    z, s = inputs(B, K, V, dtype, 11)
    z[0] = -INF                       # no token at all
    z[1, 3:] = -INF                   # three tokens
    z[2, 5] = float("nan")            # a row out
    z[3, 7] = INF                     # a row out
    z[4:8] = -INF                     # a sequence without a way on
    z[8:12] = float("nan")
    s[3, 1:] = -INF                   # only one beam alive
    z[12, 1:] = -INF                  # ... with one token
    check(ops, z, s, M=M)
    lowest = torch.finfo(dtype).min
    z[5, :9] = lowest                 # the type's lowest value is a logit like another
    z[6] = lowest
    check(ops, z, s, M=M)
    s[0, 0] = float("nan")
    s[1] = -INF
    check(ops, z, s, M=M)


@pytest.mark.parametrize("dtype", [BF, H, F])
def test_strides_and_alignment(ops, dtype):
    B, K, V, M = 2, 3, 3001, 7
    z, s = inputs(B, K, V, dtype, 5)
    want = check(ops, z, s, M=M)
    for pad, off in ((0, 1), (7, 0), (7, 3), (1095, 0), (0, 8)):
        buf = torch.full((off + B * K * (V + pad) + 16,), INF, device="cuda", dtype=dtype)   # must not be read into a row
        view = buf[off:off + B * K * (V + pad)].view(B * K, V + pad)[:, :V]
        view.copy_(z)
        r = ops.beam_step(view, s, num_candidates=M)
        for a, b in ((r.scores, want.scores), (r.tokens, want.tokens), (r.parents, want.parents), (r.lse, want.lse)):
            assert torch.equal(a, b)          # the same bits wherever a row starts


def test_row_offsets_past_32_bits(ops):
    K, V, ld = 4, 1000, 1 << 30
    buf = torch.empty(3 * ld + V, device="cuda", dtype=BF)
    view = buf.as_strided((K, V), (ld, 1))
    z, s = inputs(1, K, V, BF, 3)
    view.copy_(z)
    want = ops.beam_step(z, s)
    r = ops.beam_step(view, s)
    assert torch.equal(r.scores, want.scores) and torch.equal(r.tokens, want.tokens)
    assert torch.equal(r.parents, want.parents)


def test_many_rows_and_repeats(ops):
    z, s = inputs(64, 16, 5003, BF, 21)
    a = check(ops, z, s, M=32)
    for _ in range(3):
        b = ops.beam_step(z, s, num_candidates=32)
        for x, y in ((a.scores, b.scores), (a.tokens, b.tokens), (a.parents, b.parents), (a.lse, b.lse)):
            assert torch.equal(x, y)


def test_no_sequences(ops):
    r = ops.beam_step(torch.empty(0, 50, device="cuda"), torch.empty(0, 4, device="cuda"), num_candidates=3)
    assert r.scores.shape == (0, 3) and r.lse.shape == (0, 4)


# ------------------------------------------------------------------ reorder
def expected(t, parents, dim):
    B, Ko = parents.shape
    K = t.shape[dim] // B
    rows = (parents.long() + torch.arange(B, device="cuda")[:, None] * K).flatten()
    return t.index_select(dim, rows)


def parents_of(B, K, Ko, kind, g):
    if kind == "identity":
        return torch.arange(Ko, device="cuda", dtype=torch.int32).repeat(B, 1) % K
    if kind == "same":
        return torch.full((B, Ko), K - 1, device="cuda", dtype=torch.int32)
    if kind == "cycle":
        return ((torch.arange(Ko, device="cuda", dtype=torch.int32) + 1) % K).repeat(B, 1)
    return torch.randint(0, K, (B, Ko), device="cuda", generator=g, dtype=torch.int32)


@pytest.mark.parametrize("kind", ["identity", "same", "cycle", "random"])
@pytest.mark.parametrize("B,K,Ko", [(1, 1, 1), (3, 4, 4), (2, 5, 3), (2, 3, 8), (1, 64, 64), (7, 16, 16)])
def test_reorder(ops, kind, B, K, Ko):
    g = gen(B * 100 + K)
    parents = parents_of(B, K, Ko, kind, g)
    N = B * K
    kv = torch.randn(2, N, 3, 20, 24, device="cuda", generator=g).to(BF)
    for t, dim in ((kv, 1), (kv[:, :, :, :7], 1), (kv[:, :, 1:, 2:9, 3:20], 1), (kv[:, :, :, ::3], 1),
                   (torch.randint(0, 99, (N, 513), device="cuda", generator=g)[:, :211], 0),
                   (torch.randn(N, 33, device="cuda", generator=g), 0), (torch.randn(N, device="cuda", generator=g), 0),
                   (torch.randint(0, 2, (N, 5), device="cuda", generator=g).bool(), 0),
                   (torch.randint(0, 99, (N, 301), device="cuda", generator=g).to(torch.uint8)[:, 1:], 0),
                   (torch.randn(N, 2, 4096, device="cuda", generator=g, dtype=torch.float64), 0),
                   (torch.randn(5, N, device="cuda", generator=g).t(), 0), (torch.randn(5, N, device="cuda", generator=g), -1)):
        want = expected(t, parents, dim)
        keep = t.clone()
        got, = ops.beam_reorder([t], parents, dim=dim)
        assert torch.equal(got, want) and torch.equal(t, keep)
        if Ko == K:
            hold = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
            ops.beam_reorder([t], parents, out=[hold], dim=dim)
            assert torch.equal(hold, want)
            same, = ops.beam_reorder([t], parents, out="inplace", dim=dim)
            assert same is t and torch.equal(t, want)
    assert ops.device_error() == 0


def test_reorder_leaves_the_rest_alone(ops):
    g = gen(2)
    B, K = 3, 4
    parents = parents_of(B, K, K, "random", g)
    for inplace in (False, True):
        src = torch.randn(B * K, 2, 50, 16, device="cuda", generator=g)
        dst = src if inplace else torch.randn(B * K, 2, 50, 16, device="cuda", generator=g)
        before, want = dst.clone(), expected(src[:, :, 3:41, :15], parents, 0)
        ops.beam_reorder([src[:, :, 3:41, :15]], parents, out=[dst[:, :, 3:41, :15]])
        assert torch.equal(dst[:, :, 3:41, :15], want)
        inside = torch.zeros_like(dst, dtype=torch.bool)
        inside[:, :, 3:41, :15] = True
        assert torch.equal(dst[~inside], before[~inside])


def test_reorder_many_states_at_once(ops):
    g = gen(4)
    B, K = 2, 6
    parents = parents_of(B, K, K, "random", g)
    states = [torch.randn(B * K, n, device="cuda", generator=g) for n in (1, 2, 3, 4, 5, 8, 16, 31, 64, 129, 1000, 4096)] * 2
    states = [t.clone() for t in states] + [torch.empty(B * K, 0, device="cuda")]
    want = [expected(t, parents, 0) for t in states]
    got = ops.beam_reorder(states, parents)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ops.beam_reorder(states, parents, out="inplace")
    assert all(torch.equal(a, b) for a, b in zip(states, want))


@pytest.mark.parametrize("inplace", [False, True])
def test_bad_parents(ops, inplace):
    x = torch.arange(12.0, device="cuda").view(6, 2)
    p = torch.tensor([[2, -1, 0], [3, 1, 2 ** 31 - 1]], device="cuda", dtype=torch.int32)
    out = x if inplace else torch.full_like(x, -7.0)
    old = out.clone()
    src = x.clone()
    ops.beam_reorder([x], p, out=[out])
    assert ops.device_error() == 8 and ops.device_error() == 0
    assert torch.equal(out[0], src[2]) and torch.equal(out[2], src[0]) and torch.equal(out[4], src[4])
    assert torch.equal(out[1], old[1]) and torch.equal(out[3], old[3]) and torch.equal(out[5], old[5])


@pytest.mark.parametrize("inplace", [False, True])
def test_reorder_offsets_past_32_bits(ops, inplace):
    B, K = 1, 3
    t = torch.zeros(B * K, 3 << 29, device="cuda", dtype=BF)          # rows of 3 GB
    view = t[:, ::1]
    marks = torch.randn(K, 64, device="cuda", generator=gen(1)).to(BF)
    t[:, -64:] = marks
    p = torch.tensor([[2, 0, 1]], device="cuda", dtype=torch.int32)
    got, = ops.beam_reorder([view], p, out="inplace" if inplace else None)
    assert torch.equal(got[:, -64:], marks[p[0].long()])
    assert not got[:, :-64].view(torch.int32).any().item()


def test_other_stream_and_graph(ops):
    g = gen(8)
    B, K, V = 3, 4, 3001
    z, s = inputs(B, K, V, BF, 8)
    kv = torch.randn(B * K, 2, 9, 16, device="cuda", generator=g)
    want = ops.beam_step(z, s)
    moved, = ops.beam_reorder([kv], want.parents)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r = ops.beam_step(z, s, stream=st)
    q, = ops.beam_reorder([kv], r.parents, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(r.tokens, want.tokens) and torch.equal(r.scores, want.scores) and torch.equal(q, moved)
    out = torch.empty_like(kv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ops.beam_step(z, s)
        ops.beam_reorder([kv], r.parents, out=[out])
    graph.replay()
    assert torch.equal(r.tokens, want.tokens) and torch.equal(r.scores, want.scores) and torch.equal(out, moved)
    z2, s2 = inputs(B, K, V, BF, 9)
    z.copy_(z2)
    s.copy_(s2)
    kv.normal_(generator=g)
    graph.replay()
    want = ops.beam_step(z, s)
    moved, = ops.beam_reorder([kv], want.parents)
    assert torch.equal(r.tokens, want.tokens) and torch.equal(r.scores, want.scores) and torch.equal(out, moved)


def test_refusals(ops):
    from lm_head_vocab_gb300 import LMLossError
    z, s = inputs(2, 3, 100, BF, 1)
    ok = torch.zeros(2, 3, dtype=torch.uint8, device="cuda")
    for kw, err in (({"num_candidates": 0}, ValueError), ({"num_candidates": 65}, ValueError),
                    ({"finished": ok}, LMLossError), ({"finished": ok.bool(), "eos_token": 1}, TypeError),
                    ({"finished": ok[:1], "eos_token": 1}, ValueError), ({"eos_token": 100}, LMLossError),
                    ({"length_penalty": 0.5}, LMLossError), ({"length_penalty": -1.0}, LMLossError),
                    ({"lengths": ok}, TypeError), ({"lengths": ok.int()[:, :2]}, ValueError),
                    ({"token_mask": torch.zeros(6, 3, device="cuda", dtype=torch.int32)}, ValueError),
                    ({"token_mask": torch.zeros(2, 4, device="cuda", dtype=torch.int32)}, ValueError),
                    ({"token_mask": torch.zeros(1, 4, device="cuda", dtype=torch.int64)}, TypeError)):
        with pytest.raises(err):
            ops.beam_step(z, s, **kw)
    with pytest.raises(TypeError):
        ops.beam_step(z.double(), s)
    with pytest.raises(TypeError):
        ops.beam_step(z, s.double())
    with pytest.raises(ValueError):
        ops.beam_step(z[:5], s)
    with pytest.raises(ValueError):
        ops.beam_step(z.cpu(), s)
    with pytest.raises(ValueError):
        ops.beam_step(torch.randn(100, 6, device="cuda").t(), s)
    from lm_head_vocab_gb300 import VocabOps
    small = VocabOps(0, max_tokens=0, max_rows=1, max_vocab=100)
    with pytest.raises(LMLossError) as e:                    # more rows than the handle's workspace
        small.beam_step(z, s, num_candidates=64)
    assert e.value.status == 1
    small.beam_step(z[:1], s[:1, :1], num_candidates=64)
    small.close()
    x = torch.randn(6, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for states, parents, kw, err in (
            ([x], p.long(), {}, TypeError), ([x], p[0], {}, ValueError), ([x[:5]], p, {}, ValueError),
            ([x], p.cpu(), {}, ValueError), ([x.cpu()], p, {}, ValueError), ([x, x[:4]], p, {}, ValueError),
            ([x], p, {"out": [x[:, :4]]}, ValueError), ([x], p, {"out": [x.double()]}, TypeError),
            ([x], p, {"out": []}, ValueError), ([x], p, {"out": "there"}, ValueError),
            ([x], p[:, :2].contiguous(), {"out": "inplace"}, ValueError),
            ([x[:, :4]], p, {"out": [x[:, 2:6]]}, LMLossError),
            ([x[:, :1].expand(6, 8)], p, {"out": "inplace"}, ValueError),
            ([torch.randn(6, 8, 8, 8, 8, 8, device="cuda")[:, ::2, ::2, ::2, ::2]], p, {}, ValueError)):
        with pytest.raises(err):
            ops.beam_reorder(states, parents, **kw)
    # a broadcast state may be read
    got, = ops.beam_reorder([x[:, :1].expand(6, 8)], p)
    assert torch.equal(got, expected(x[:, :1].expand(6, 8), p, 0))


def test_every_parent_map_of_three_beams_in_place(ops):
    maps = torch.tensor(list(itertools.product(range(3), repeat=3)), device="cuda", dtype=torch.int32)
    x = torch.randn(len(maps) * 3, 37, device="cuda", generator=gen(1))
    want = expected(x, maps, 0)
    ops.beam_reorder([x], maps, out="inplace")
    assert torch.equal(x, want)
