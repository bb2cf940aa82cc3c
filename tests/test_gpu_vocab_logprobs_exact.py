"""The gradient of token log-probabilities on the GPU against that of the logits' own softmax in fp64, not of an
lse that fp32 has rounded.

Tolerances: with d = ln p and E = 2^-24, p = ex2(d log2 e) has a relative error of at most 2^-22 (ex2) + 5 E |d| (z - m, its two
products with 1 / tau and the change to base 2 rounded) + E ln s (its rounding) + t, t being ln s's own error, `tolerance` of
test_gpu_vocab_logprobs.py.  H's is t (4 + 2 L), as in test_gpu_vocab_logprobs_range.py.  The n given gradients' sum
(n + 12) E of their magnitudes, a token's own (n + 4) E; the type's rounding; below 2^-126 (fp16: half its smallest step)
flushed.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_logprobs import BF, EPS, F, H, INF, allowed, gen, half_step, make, ops, random_mask, some_tokens, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


def check(ops, z, tokens, g, ge=None, tau=1.0, mask=None, out=None, lse=None):  # noqa: F811
    z0 = z.clone()
    r = ops.token_logprobs(z, tokens, temperature=tau, token_mask=mask, for_gradient=True)
    d = ops.token_logprobs_backward(z, lse, tokens, g, row_max=r.row_max, log_sum=r.log_sum,
                                    entropy=r.entropy if ge is not None else None, grad_entropy=ge, temperature=tau,
                                    token_mask=mask, grad=out)
    assert ops.device_error() == 0 and d.dtype == z.dtype
    (T, V), t64 = z.shape, float(np.float32(tau))
    may = torch.from_numpy(allowed(mask, T, V).copy()).cuda()
    x = torch.where(may, z0.double(), -INF)
    m = x.amax(1, keepdim=True)
    none = m == -INF
    assert torch.equal(r.row_max.double(), m[:, 0])
    x = (x - torch.where(none, 0.0, m)) / t64
    log_s = torch.logsumexp(x, 1, keepdim=True)
    dd = x - torch.where(none, 0.0, log_s)
    p = torch.exp(dd)
    dd = torch.where(p > 0, dd, 0.0)
    L = -(p * dd).sum(1, keepdim=True)
    ent = L
    t = torch.from_numpy(tolerance((torch.where(p > 0, -p * torch.where(p > 0, x, 0.0), 0.0)).sum(1, keepdim=True).cpu().numpy(), T, V)).cuda()
    assert bool(((r.log_sum.double()[:, None] - log_s).abs() <= t + EPS * log_s)[~none].all())
    assert bool((r.log_sum[none[:, 0]] == -INF).all())
    n = tokens.numel() // T
    tk, gg = tokens.view(T, n).long(), torch.where((tokens.view(T, n) == -100) | none, 0.0, g.view(T, n).double())
    e = torch.zeros(T, 1, device="cuda").double() if ge is None else torch.where(none, 0.0, ge.double()[:, None])
    at = torch.zeros_like(p).scatter_add_(1, tk.clamp(min=0), gg)
    at_abs = torch.zeros_like(p).scatter_add_(1, tk.clamp(min=0), gg.abs())
    by = gg.sum(1, keepdim=True) + e * (dd + ent)
    want = torch.where(may, (at - p * by) / t64, 0.0)
    terms = gg.abs().sum(1, keepdim=True) + e.abs() * (dd.abs() + ent)
    rel = 2.0 ** -22 + 5 * EPS * dd.abs() + EPS * torch.where(none, 0.0, log_s) + t
    tol = (p * by.abs() * rel + p * terms * (n + 12) * EPS + at_abs * (n + 4) * EPS) / t64 + want.abs() * 4 * EPS
    tol += p * e.abs() * (dd.abs() * 5 * EPS + EPS * torch.where(none, 0.0, log_s) + 2 * t + t * (4 + 2 * L)) / t64
    tol += want.abs() * half_step(z.dtype) + {F: 2.0 ** -125, BF: 2.0 ** -125, H: 2.0 ** -25}[z.dtype] * (1 + terms / t64)
    # a result past the type's range
    most = torch.finfo(z.dtype).max
    want = torch.where(want.abs() > most, torch.copysign(torch.full_like(want, INF), want), want)
    err = torch.where(want.isinf(), torch.where((d.double() == want) | (d.double().abs() >= most * 0.99), 0.0, INF), (d.double() - want).abs())
    assert bool((err <= tol).all()), f"{(err / tol).nan_to_num().max().item()}"
    assert not d[~may].any() and not d[none[:, 0]].any()
    return r, d


def grads(T, n, seed, entropy=True):
    g = torch.randn(T, n, device="cuda", generator=gen(seed))
    return g, torch.randn(T, device="cuda", generator=gen(seed + 1)) if entropy else None


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("tau", [1.0, 0.7, 0.01, 1e-3, 1e-6, 2.0 ** -20, 50.0])
@pytest.mark.parametrize("entropy", [False, True])
def test_temperatures(ops, dtype, tau, entropy):  # noqa: F811
    for T, V, n in ((7, 5003, 3), (1, 70000, 2), (300, 1000, 1)):
        z = make(T, V, F, 300 + T, std=2.0)
        z[:, V // 2] = 25 + torch.arange(T, device="cuda") / T * 3    # one logit far above the others
        z[0, V // 3] = z[0, V // 2]
        tokens = some_tokens(T, n, V, 301)
        tokens[:, 0] = V // 2
        g, ge = grads(T, n, 303, entropy)
        check(ops, z.to(dtype), tokens, g, ge, tau)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_rows_at_the_types_ends(ops, dtype, tau):  # noqa: F811
    # an lse past fp32's range is no row without candidates
    T, V = 8, 3001
    info = torch.finfo(dtype)
    z = make(T, V, dtype, 310)
    z[0] = info.min
    z[1, 4:] = info.min
    z[2] = info.max
    z[3] = -INF
    z[4] = info.min
    z[4, 100] = -INF
    z[5] = info.max
    z[5, ::2] = info.min
    z[6, 1:] = -INF
    g, ge = grads(T, 4, 311)
    tokens = some_tokens(T, 4, V, 313)
    tokens[:, 0] = 0
    check(ops, z, tokens, g, ge, tau)


@pytest.mark.parametrize("dtype", [BF, F])
def test_additive_masks_and_large_logits(ops, dtype):  # noqa: F811
    T, V = 5, 9001
    for i, fill in enumerate((-1e4, -1e9, -1e10, -1e20, 1e10, 1e20)):
        z = make(T, V, dtype, 320 + i)
        z[:, ::3] = fill
        z[1] = fill
        z[2, : V // 2] = fill
        g, ge = grads(T, 3, 321)
        for tau in (1.0, 1e-6):
            check(ops, z, some_tokens(T, 3, V, 323), g, ge, tau)
            check(ops, z, some_tokens(T, 3, V, 323), g, ge, tau, random_mask(T, V, 325))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("shift,extra,gshift,gextra", [(0, 0, 1, 0), (3, 1, 0, 8), (1, 7, 5, 3)])
def test_strides_and_in_place(ops, dtype, shift, extra, gshift, gextra):  # noqa: F811
    T, V = 6, 3001

    def place(s, x):
        return torch.full((s + T * (V + x) + 64,), 7.0, device="cuda", dtype=dtype)[s:s + T * (V + x)].view(T, V + x)[:, :V]
    z, out = place(shift, extra), place(gshift, gextra)
    z.copy_(make(T, V, dtype, 330))
    tokens, (g, ge) = some_tokens(T, 4, V, 331), grads(T, 4, 333)
    mask = random_mask(T, V, 335)
    r, d = check(ops, z, tokens, g, ge, 0.02, mask, out)
    there = ops.token_logprobs_backward(z, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum, entropy=r.entropy,
                                        grad_entropy=ge, temperature=0.02, token_mask=mask, grad="inplace")
    assert there.data_ptr() == z.data_ptr() and torch.equal(there, d)


def test_lse_is_not_looked_at_beside_them(ops):  # noqa: F811
    z, tokens, (g, ge) = make(4, 1000, F, 340), some_tokens(4, 2, 1000, 341), grads(4, 2, 343)
    _, a = check(ops, z, tokens, g, ge)
    _, b = check(ops, z, tokens, g, ge, lse=torch.full((4,), float("nan"), device="cuda"))
    assert torch.equal(a, b)


def test_captured_on_another_stream(ops):  # noqa: F811
    T, V = 3, 70000
    z, tokens, (g, ge) = make(T, V, BF, 350), some_tokens(T, 2, V, 351), grads(T, 2, 353)
    check(ops, z, tokens, g, ge, 1e-3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ops.token_logprobs(z, tokens, temperature=1e-3, for_gradient=True)
        d = ops.token_logprobs_backward(z, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum, entropy=r.entropy,
                                        grad_entropy=ge, temperature=1e-3)
    z.copy_(make(T, V, BF, 355))
    graph.replay()
    torch.cuda.synchronize()
    _, want = check(ops, z, tokens, g, ge, 1e-3)
    assert torch.equal(d, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = ops.token_logprobs(z, tokens, temperature=1e-3, for_gradient=True, stream=s)
    d = ops.token_logprobs_backward(z, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum, entropy=r.entropy, grad_entropy=ge,
                                    temperature=1e-3, stream=s)
    s.synchronize()
    assert torch.equal(d, want)


@pytest.mark.parametrize("dtype", [BF, H, F])
def test_rows_with_nan_and_infinities(ops, dtype):  # noqa: F811
    # such a row's gradient is NaN where columns are allowed, and disturbs no other
    T, V = 8, 5003
    z, tokens, (g, ge) = make(T, V, dtype, 360), some_tokens(T, 3, V, 361), grads(T, 3, 363)
    mask = random_mask(T, V, 365)
    mask[6] = 0
    may = torch.from_numpy(allowed(mask, T, V).copy()).cuda()
    clean, want = check(ops, z, tokens, g, ge, 0.1, mask)
    at = [int(may[i].nonzero()[9]) for i in range(6)]
    z[1, at[1]] = float("nan")
    z[2, at[2]] = INF
    z[4] = float("nan")
    z[5, at[5]] = INF
    z[5, ::2] = -INF
    z[3][~may[3]] = float("nan")                             # nothing that counts
    z[0][~may[0]] = INF
    for m in (None, mask):
        r = ops.token_logprobs(z, tokens, temperature=0.1, token_mask=m, for_gradient=True)
        d = ops.token_logprobs_backward(z, None, tokens, g, row_max=r.row_max, log_sum=r.log_sum, entropy=r.entropy,
                                        grad_entropy=ge, temperature=0.1, token_mask=m)
        ok = torch.ones(V, dtype=torch.bool, device="cuda")
        for i in (1, 2, 4, 5):
            inside = ok if m is None else may[i]
            assert bool(d[i][inside].isnan().all()) and not d[i][~inside].any()
        assert bool(r.log_sum[[1, 2, 4, 5]].isnan().all())
    assert torch.equal(d[[0, 3, 6, 7]], want[[0, 3, 6, 7]])
    assert ops.device_error() == 0
