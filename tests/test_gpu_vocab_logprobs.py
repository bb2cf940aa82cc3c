"""Token log-probabilities with entropy and alternatives, and their gradient, on the GPU against fp64.

Tolerances, from the arithmetic (eps = 2^-24, u the exponents in base 2, E = sum p |u|):
a row's sum of exponentials has a relative error of at most
  2^-22 (ex2.approx) + 3 eps ln2 E (difference, product and factor rounded)
  + 100 eps (additions: 16 in a tile, a tile after another, the trees)
  + 4 eps R (a running sum's rescaling, R raises of the maximum at most: a tile each)
which is lse's absolute error, but for its own rounding; and the sum of u 2^u, all of one sign,
the same and 2 eps.  H = ln s - ln2 e / s has that error once, and twice times L = sum p (m - y).
Log-probabilities are subtracted in fp64 and rounded.  Alternatives are in the exact order.

The gradient: p = ex2(d log2 e), d = y - lse from two fused operations: relative 2^-22 + 4 eps (|d| + |lse|)
(lse is an input, its rounding is no error; 1 / tau's pair leaves 2 eps); the sums of n given gradients
(n + 8) eps of their magnitudes; each product and sum 4 eps; the type's rounding; below 2^-126 (fp16: half its
smallest step) flushed.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, H, F = torch.bfloat16, torch.float16, torch.float32
INF, EPS = float("inf"), 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_rows=64)
    yield h
    h.close()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def allowed(mask, T, V):
    if mask is None:
        return np.ones((T, V), bool)
    bits = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :V].astype(bool)
    return np.broadcast_to(bits, (T, V))


def reference(logits, mask, tau):
    z = logits.double().cpu().numpy()
    may = allowed(mask, *z.shape)
    tau = float(np.float32(tau))
    with np.errstate(all="ignore"):
        y = np.where(may, z / tau, -INF)
        m = np.where(np.isnan(y), -INF, y).max(1)
        none = m == -INF
        none &= ~np.isnan(y).any(1)
        d = y - np.where(np.isfinite(m), m, 0)[:, None]
        e = np.exp(d)
        s = e.sum(1)
        lse = np.where(none, -INF, np.where(np.isfinite(m), m, 0) + np.log(s))
        lse[(np.isnan(y) | (y == INF)).any(1)] = np.nan
        p = e / s[:, None]
        L = np.where(p > 0, -p * d, 0).sum(1)
        ent = np.where(none, 0, np.log(s) + L)
        ent[np.isnan(lse)] = np.nan
    return z, may, y, lse, ent, L, none


def tolerance(L, T, V):
    R = 2 + V // 1024
    return 2.0 ** -22 + 3 * EPS * np.nan_to_num(L) + (100 + 4 * R) * EPS


def near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    # a result past fp32's range rounds to infinity (logits of 3e38 at a temperature of 1/2)
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.copysign(INF, want), want)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), f"{what}: infinities and NaN"
    err = np.abs(got[fine] - want[fine])
    tol = np.broadcast_to(tol, want.shape)[fine]
    assert (err <= tol).all(), f"{what}: {err.max()} over {tol[err.argmax()] if err.size else 0}"


def check(ops, logits, tokens=None, M=0, tau=1.0, mask=None, **kw):
    r = ops.token_logprobs(logits, tokens, num_top=M, temperature=tau, token_mask=mask, **kw)
    assert ops.device_error() == 0
    z, may, y, lse, ent, L, none = reference(logits, mask, tau)
    T, V = z.shape
    tol = tolerance(L, T, V)
    near(r.lse.cpu(), lse, tol + EPS * np.abs(np.nan_to_num(lse)), "lse")
    if r.entropy is not None:
        near(r.entropy.cpu(), ent, tol * (1 + 2 * np.nan_to_num(L)) + 2 * EPS * np.nan_to_num(np.abs(ent)), "entropy")
    if tokens is not None:
        t = tokens.cpu().numpy().reshape(T, -1)
        with np.errstate(all="ignore"):
            want = np.take_along_axis(y, np.maximum(t, 0), 1) - lse[:, None]
        want = np.where(none[:, None], -INF, want)
        want = np.where(t == -100, 0, want)
        near(r.logp.cpu().numpy().reshape(T, -1), want, tol[:, None] + EPS * np.abs(np.nan_to_num(want)), "logp")
        assert r.logp.shape == tokens.shape
    if M:
        top, at = r.top_logp.cpu().numpy(), r.top_tokens.cpu().numpy()
        for i in range(T):
            v = np.nonzero(may[i] & np.isfinite(z[i]))[0] if np.isfinite(lse[i]) else np.zeros(0, int)
            v = v[np.lexsort((v, -z[i, v]))][:M]
            assert at[i].tolist() == v.tolist() + [-100] * (M - len(v)), f"row {i}"
            want = np.concatenate([y[i, v] - lse[i], np.full(M - len(v), -INF)])
            near(top[i], want, tol[i] + EPS * np.abs(np.nan_to_num(want)), "alternatives")
    return r


def make(T, V, dtype, seed, std=3.0):
    return (torch.randn(T, V, device="cuda", generator=gen(seed)) * std).to(dtype)


def some_tokens(T, n, V, seed, dtype=torch.int64):
    t = torch.randint(0, V, (T, n), device="cuda", generator=gen(seed))
    t[torch.rand(T, n, device="cuda", generator=gen(seed + 1)) < 0.1] = -100
    return t.to(dtype)


def random_mask(rows, V, seed, density=2):
    m = torch.randint(-2 ** 31, 2 ** 31, (rows, (V + 31) // 32), device="cuda", generator=gen(seed))
    for i in range(density - 1):
        m &= torch.randint(-2 ** 31, 2 ** 31, m.shape, device="cuda", generator=gen(seed + 50 + i))
    return m.int()


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("T,V,n,M", [(1, 1, 1, 1), (1, 2, 3, 5), (3, 7, 1, 64), (2, 33, 0, 4), (1, 128256, 4, 20),
                                     (5, 32003, 2, 5), (33, 4099, 5, 1), (7, 70001, 1, 0), (700, 1000, 1, 3),
                                     (64, 20011, 3, 33)])
def test_against_fp64(ops, dtype, T, V, n, M):
    z = make(T, V, dtype, T + V)
    check(ops, z, some_tokens(T, n, V, 5), M, tau=0.8)


@pytest.mark.parametrize("tau", [1.0, 0.05, 3.0, 2.0 ** -20, 2.0 ** 20])
def test_temperatures(ops, tau):
    check(ops, make(6, 5003, F, 3), some_tokens(6, 3, 5003, 4, torch.int32), 7, tau=tau)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("T,V", [(1, 128256), (9, 4099), (300, 3001)])
@pytest.mark.parametrize("rows,density", [("one", 1), ("all", 2), ("all", 6)])
def test_masks(ops, dtype, T, V, rows, density):
    mask = random_mask(T if rows == "all" else 1, V, 9, density)
    if T > 2:
        if rows == "all":
            mask[T // 2] = 0                                 # nothing
            mask[1] = 0
            mask[1, (V - 1) // 32] = 1 << ((V - 1) % 32)     # the last column alone
            mask[2] = -1
    z = make(T, V, dtype, 11)
    # what stands in masked columns has no effect
    may = torch.from_numpy(allowed(mask, T, V).copy()).cuda()
    odd = torch.where(torch.arange(V, device="cuda") % 3 == 0, float("nan"), INF)
    z = torch.where(may, z, odd.to(dtype)[None])
    check(ops, z, some_tokens(T, 6, V, 13), 9, mask=mask, tau=1.7)


@pytest.mark.parametrize("dtype", [BF, H, F])
def test_rows_of_lowest_values_infinities_and_nan(ops, dtype):
    V = 9001
    low = torch.finfo(dtype).min
    z = make(12, V, dtype, 17)
    z[0] = -INF
    z[1] = low
    z[2, 5:] = low
    z[3, 5:] = -INF
    z[4, 100] = float("nan")
    z[5, 8000] = INF
    z[6] = 0
    z[7, ::2] = -INF
    z[8] = low
    z[8, 77] = low / 2
    z[9, 0], z[9, 1] = torch.finfo(dtype).max, torch.finfo(dtype).max
    z[10, :] = -0.0
    z[10, 40] = 0.0
    check(ops, z, some_tokens(12, 4, V, 19), 10)
    check(ops, z, some_tokens(12, 4, V, 19), 10, tau=0.5)


def test_equal_and_sorted_rows(ops):
    V = 66000
    z = torch.zeros(6, V, device="cuda")
    z[1] = torch.arange(V, device="cuda") / 4096            # the largest last
    z[2] = -torch.arange(V, device="cuda") / 4096
    z[3, V - 70:] = 1.0
    z[4] = torch.arange(V, device="cuda") % 7
    z[5] = (torch.arange(V, device="cuda") // 512).float()
    for t in (F, BF):
        check(ops, z.to(t), None, 64)
        check(ops, z.to(t).repeat(120, 1)[:700], None, 64)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("shift,extra", [(0, 0), (1, 0), (3, 5), (7, 1)])
def test_strides_and_alignment(ops, dtype, shift, extra):
    T, V = 5, 10007
    flat = torch.full((shift + T * (V + extra) + 64,), float("nan"), device="cuda", dtype=dtype)
    z = flat[shift:shift + T * (V + extra)].view(T, V + extra)[:, :V]
    z.copy_(make(T, V, dtype, 23))
    check(ops, z, some_tokens(T, 3, V, 29), 12)
    same = ops.token_logprobs(z.contiguous(), num_top=12)
    r = ops.token_logprobs(z, num_top=12)
    for a, b in ((r.lse, same.lse), (r.entropy, same.entropy), (r.top_logp, same.top_logp), (r.top_tokens, same.top_tokens)):
        assert torch.equal(a, b)                             # bits depend on columns, not addresses


def test_outputs_left_out_and_one_dimension(ops):
    z = make(4, 3000, BF, 31)
    t = torch.tensor([1, -100, 2999, 0], device="cuda")
    r = check(ops, z, t, 3)
    a = ops.token_logprobs(z, t, entropy=False, num_top=3)
    assert a.entropy is None and torch.equal(a.lse, r.lse) and torch.equal(a.logp, r.logp)
    b = ops.token_logprobs(z)
    assert b.logp is None and b.top_logp is None and torch.equal(b.entropy, r.entropy)
    e = ops.token_logprobs(z[:0], t[:0], num_top=2)
    assert e.logp.shape == (0,) and e.top_tokens.shape == (0, 2)


def test_bad_tokens(ops):
    import lm_head_vocab_gb300._lib as L
    z = make(3, 50, F, 37)
    t = torch.tensor([[1, 50], [-1, 2], [2 ** 40, -100]], device="cuda")
    r = ops.token_logprobs(z, t)
    assert ops.device_error() == L.LMLOSS_ERR_BAD_TARGET and ops.device_error() == 0
    assert torch.isnan(r.logp).tolist() == [[False, True], [True, False], [True, False]]
    g = ops.token_logprobs_backward(z, r.lse, t, torch.ones(3, 2, device="cuda"))
    assert ops.device_error() == L.LMLOSS_ERR_BAD_TARGET
    ok = torch.tensor([[1, -100], [-100, 2], [-100, -100]], device="cuda")
    assert torch.equal(g, ops.token_logprobs_backward(z, r.lse, ok, torch.ones(3, 2, device="cuda")))


def test_many_rows(ops):
    # more rows than one launch counts
    T, V = 70001, 40
    z = make(T, V, H, 41)
    check(ops, z, some_tokens(T, 1, V, 43), 2)


# ------------------------------------------------------------------ gradient
def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check_grad(ops, z, tokens, g, ge=None, tau=1.0, mask=None, out=None):
    r = ops.token_logprobs(z, tokens, temperature=tau, token_mask=mask)
    z0 = z.clone()
    d = ops.token_logprobs_backward(z, r.lse, tokens, g, entropy=r.entropy if ge is not None else None, grad_entropy=ge,
                                    temperature=tau, token_mask=mask, grad=out)
    assert ops.device_error() == 0 and d.dtype == z.dtype
    t64, (T, V) = float(np.float32(tau)), z.shape
    may = torch.from_numpy(allowed(mask, T, V).copy()).cuda()
    y = torch.where(may, z0.double() / t64, -INF)
    lse, ent = r.lse.double()[:, None], r.entropy.double()[:, None]
    none = lse == -INF
    p = torch.where(none, 0.0, torch.exp(y - lse))
    n = 0 if tokens is None else tokens.numel() // max(T, 1)
    tk = torch.zeros(T, 0, dtype=torch.int64, device="cuda") if tokens is None else tokens.view(T, n).long()
    gg = torch.zeros(T, 0, device="cuda").double() if tokens is None else g.view(T, n).double()
    gg = torch.where((tk == -100) | none, 0.0, gg)
    dd = torch.where(p > 0, y - lse, 0.0)
    e = 0.0 if ge is None else ge.double()[:, None]
    by = gg.sum(1, keepdim=True) + e * (dd + ent)
    at = torch.zeros_like(p).scatter_add_(1, tk.clamp(min=0), gg)
    at_abs = torch.zeros_like(p).scatter_add_(1, tk.clamp(min=0), gg.abs())
    want = torch.where(may, (at - p * by) / t64, 0.0)
    e_abs = 0.0 if ge is None else ge.double().abs()[:, None]
    terms = gg.abs().sum(1, keepdim=True) + e_abs * (dd.abs() + ent.abs())
    rel = 2.0 ** -22 + 4 * EPS * (dd.abs() + torch.where(none, 0.0, lse.abs()))
    tol = (p * by.abs() * rel + p * terms * (n + 12) * EPS + at_abs * (n + 4) * EPS) / t64 + want.abs() * 4 * EPS
    tol += want.abs() * half_step(z.dtype) + {F: 2.0 ** -125, BF: 2.0 ** -125, H: 2.0 ** -25}[z.dtype] * (1 + terms / t64)
    nan = torch.isnan(lse)
    assert torch.equal(torch.isnan(d), (nan & may).expand(T, V))
    err = torch.where(nan, 0.0, (d.double() - want).abs())
    assert bool((err <= torch.where(nan, INF, tol)).all()), f"{(err / tol).nan_to_num().max().item()}"
    assert not d[~may].any()
    return r, d


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("T,V,n", [(1, 1, 1), (3, 5, 9), (2, 128256, 1), (50, 4099, 16), (300, 1000, 3), (4, 9000, 0)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient(ops, dtype, T, V, n, entropy):
    z = make(T, V, dtype, 51 + T)
    tokens = some_tokens(T, n, V, 53) if n else None
    if n > 4:
        tokens[:, 3] = tokens[:, 0]                          # the same token twice, thrice
        tokens[:, 4] = tokens[:, 0]
    g = torch.randn(T, n, device="cuda", generator=gen(55)) if n else None
    ge = torch.randn(T, device="cuda", generator=gen(57)) if entropy else None
    check_grad(ops, z, tokens, g, ge, tau=0.7)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("shift,extra,gshift,gextra", [(0, 0, 1, 0), (3, 0, 3, 0), (1, 7, 5, 3), (0, 1, 0, 1)])
def test_gradient_strides(ops, dtype, shift, extra, gshift, gextra):
    T, V = 6, 3001
    def place(s, x):
        flat = torch.full((s + T * (V + x) + 64,), 7.0, device="cuda", dtype=dtype)
        return flat, flat[s:s + T * (V + x)].view(T, V + x)[:, :V]
    _, z = place(shift, extra)
    z.copy_(make(T, V, dtype, 61))
    flat, out = place(gshift, gextra)
    tokens, g = some_tokens(T, 4, V, 63), torch.randn(T, 4, device="cuda", generator=gen(65))
    ge = torch.randn(T, device="cuda", generator=gen(66))
    _, d = check_grad(ops, z, tokens, g, ge, out=out)
    out.fill_(7.0)
    assert bool((flat == 7.0).all())                         # nothing beside the rows was written
    r = ops.token_logprobs(z, tokens)
    new = ops.token_logprobs_backward(z, r.lse, tokens, g, entropy=r.entropy, grad_entropy=ge)
    there = ops.token_logprobs_backward(z, r.lse, tokens, g, entropy=r.entropy, grad_entropy=ge, grad="inplace")
    assert there.data_ptr() == z.data_ptr() and torch.equal(there, new)


@pytest.mark.parametrize("dtype", [BF, F])
def test_gradient_masks_and_odd_rows(ops, dtype):
    T, V = 9, 5003
    mask = random_mask(T, V, 71)
    mask[3] = 0
    z = make(T, V, dtype, 73)
    z[0, ::2] = -INF
    z[1] = torch.finfo(dtype).min
    z[4, :] = float("nan")
    mask[4, 0] = 1
    tokens, g = some_tokens(T, 5, V, 75), torch.randn(T, 5, device="cuda", generator=gen(76))
    check_grad(ops, z, tokens, g, torch.randn(T, device="cuda", generator=gen(77)), mask=mask, tau=2.0)
    check_grad(ops, z, tokens, g, torch.randn(T, device="cuda", generator=gen(77)), mask=random_mask(1, V, 79))


def test_gradient_against_differences(ops):
    # d/dz of sum g logp + sum gH H by central differences of the fp64 formula, at a few places of each row
    T, V, tau = 3, 40, 1.5
    z = make(T, V, F, 81, std=1.0)
    tokens = torch.randint(0, V, (T, 4), device="cuda", generator=gen(82))
    tokens[:, 1] = tokens[:, 0]
    g, ge = torch.randn(T, 4, device="cuda", generator=gen(83)), torch.randn(T, device="cuda", generator=gen(84))
    r = ops.token_logprobs(z, tokens, temperature=tau)
    d = ops.token_logprobs_backward(z, r.lse, tokens, g, entropy=r.entropy, grad_entropy=ge, temperature=tau)

    def value(x):
        lp = torch.log_softmax(x / tau, 1)
        return (lp.gather(1, tokens) * g.double()).sum(1) - (lp.exp() * lp).sum(1) * ge.double()
    h = 1e-4
    for v in range(V):
        step = torch.zeros(T, V, dtype=torch.float64, device="cuda")
        step[:, v] = h
        want = (value(z.double() + step) - value(z.double() - step)) / (2 * h)
        # the difference's own error: h^2 / 6 of a third derivative below 100, and 1e-15 / h
        assert bool(((d[:, v].double() - want).abs() < 1e-6 + 2e-6 * want.abs()).all())


def test_gradient_with_many_tokens(ops):
    T, V, n = 2, 3000, 1024
    z = make(T, V, F, 91)
    check_grad(ops, z, some_tokens(T, n, V, 93), torch.randn(T, n, device="cuda", generator=gen(95)))


# ------------------------------------------------------- streams and graphs
def test_captured_and_replayed(ops):
    T, V, n = 3, 128256, 2
    z = make(T, V, BF, 101)
    t = some_tokens(T, n, V, 103)
    g, ge = torch.randn(T, n, device="cuda"), torch.randn(T, device="cuda")
    ops.token_logprobs(z, t, num_top=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ops.token_logprobs(z, t, num_top=5)
        d = ops.token_logprobs_backward(z, r.lse, t, g, entropy=r.entropy, grad_entropy=ge)
    for seed in (104, 105):
        z.copy_(make(T, V, BF, seed))
        graph.replay()
        torch.cuda.synchronize()
        e = ops.token_logprobs(z, t, num_top=5)
        f = ops.token_logprobs_backward(z, e.lse, t, g, entropy=e.entropy, grad_entropy=ge)
        for a, b in ((r.logp, e.logp), (r.lse, e.lse), (r.entropy, e.entropy), (r.top_logp, e.top_logp),
                     (r.top_tokens, e.top_tokens), (d, f)):
            assert torch.equal(a, b)


def test_on_a_stream_of_the_callers(ops):
    z, t = make(4, 50000, BF, 111), some_tokens(4, 2, 50000, 113)
    want = ops.token_logprobs(z, t, num_top=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = ops.token_logprobs(z, t, num_top=4, stream=s)
    d = ops.token_logprobs_backward(z, r.lse, t, torch.ones_like(r.logp), stream=s)
    s.synchronize()
    assert torch.equal(r.logp, want.logp) and torch.equal(r.top_tokens, want.top_tokens)
    assert torch.equal(d, ops.token_logprobs_backward(z, want.lse, t, torch.ones_like(want.logp)))


def test_offsets_past_32_bits(ops):
    # 2.6e9 logits: the last rows are those of the same rows alone
    T, V, far = 20000, 128256, 300
    z = torch.empty(T, V, device="cuda", dtype=BF)
    z.normal_(0.0, 2.0, generator=gen(103))
    tokens = torch.randint(0, V, (T, 3), device="cuda", generator=gen(104))
    r = ops.token_logprobs(z, tokens, num_top=5)
    e = ops.token_logprobs(z[-far:], tokens[-far:], num_top=5)
    for a, b in ((r.logp, e.logp), (r.lse, e.lse), (r.entropy, e.entropy), (r.top_logp, e.top_logp)):
        # (a row alone is cut into other parts: a few steps of fp32)
        assert bool(((a[-far:] - b).abs() <= 2.0 ** -19 * b.abs().clamp(min=1)).all())
    assert torch.equal(r.top_tokens[-far:], e.top_tokens)
    g, ge = torch.randn(T, 3, device="cuda", generator=gen(105)), torch.randn(T, device="cuda", generator=gen(106))
    want = ops.token_logprobs_backward(z[-far:], r.lse[-far:], tokens[-far:], g[-far:], entropy=r.entropy[-far:], grad_entropy=ge[-far:])
    got = ops.token_logprobs_backward(z, r.lse, tokens, g, entropy=r.entropy, grad_entropy=ge, grad="inplace")
    assert torch.equal(got[-far:], want)
    assert ops.device_error() == 0
