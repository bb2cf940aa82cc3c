"""Token log-probabilities of finite logits of any size, on the GPU against fp64: what additive masks leave
(-1e4 to -1e30), rows of such values alone, large logits and low temperatures.

Tolerances as in test_gpu_vocab_logprobs.py, with two additions.  A row's sums go about the maximum's fp32
value in base 2, which is off by at most 2 (above that, about the maximum itself): every exponent u of the sum of u 2^u
is at most 2 larger in size, so H's error of twice tol L becomes twice tol (L + 2 ln 2), below tol (2 L + 3).
Where sums go about the maximum itself, a thread adds up a part's columns one after another: V / 256 additions
at most, each of half a step, in place of the 100 and 4 V / 1024 counted there, which is no more.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_logprobs import BF, EPS, F, H, INF, gen, make, near, ops, random_mask, reference, some_tokens, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


def check(ops, z, tokens, M, tau=1.0, mask=None):  # noqa: F811
    r = ops.token_logprobs(z, tokens, num_top=M, temperature=tau, token_mask=mask)
    assert ops.device_error() == 0
    z64, may, y, lse, ent, L, none = reference(z, mask, tau)
    T, V = z64.shape
    tol = tolerance(L, T, V)
    near(r.lse.cpu(), lse, tol + EPS * np.abs(np.nan_to_num(lse)), "lse")
    near(r.entropy.cpu(), ent, tol * (4 + 2 * np.nan_to_num(L)) + 2 * EPS * np.nan_to_num(np.abs(ent)), "entropy")
    t = tokens.cpu().numpy()
    # (the difference to the maximum first: fp64 leaves 2^-53 of y, too much beside a tolerance of 1e-6 from y = 2^33 on)
    zmax = np.where(may, z64, -INF).max(1, keepdims=True)
    t64 = float(np.float32(tau))
    with np.errstate(all="ignore"):
        log_s = np.log(np.where(may, np.exp((z64 - zmax) / t64), 0).sum(1, keepdims=True))
        logp = np.where(may, (z64 - zmax) / t64 - log_s, -INF)
    want = np.where(t == -100, 0, np.take_along_axis(logp, np.maximum(t, 0), 1))
    # z / tau, the maximum's part of lse and lse itself, in fp64, are each off by 2^-53 of lse
    tol = tol + 2.0 ** -51 * np.abs(np.nan_to_num(lse))
    near(r.logp.cpu().numpy(), want, tol[:, None] + EPS * np.abs(np.nan_to_num(want)), "logp")
    at, top = r.top_tokens.cpu().numpy(), r.top_logp.cpu().numpy()
    for i in range(T):
        v = np.nonzero(may[i] & np.isfinite(z64[i]))[0]
        v = v[np.lexsort((v, -z64[i, v]))][:M]
        assert at[i].tolist() == v.tolist() + [-100] * (M - len(v)), f"row {i}"
        near(top[i, :len(v)], logp[i, v], tol[i] + EPS * np.abs(logp[i, v]), "alternatives")
    return r


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("tau", [1.0, 0.7, 1e-6, 2.0 ** -20])
@pytest.mark.parametrize("T,V", [(1, 128256), (6, 9001), (600, 3001)])
def test_additive_masks(ops, dtype, tau, T, V):  # noqa: F811
    # every size of what stands for "not allowed", beside ordinary logits: one column in three, whole threads'
    # first vectors, whole parts
    fills = (-1e4, -6e4) if dtype is H else (-1e4, -1e9, -3e9, -1e10, -1e12, -1e15, -1e20, -1e28)
    for i, fill in enumerate(fills):
        z = make(T, V, dtype, 200 + i)
        col = torch.arange(V, device="cuda")
        z[:, col % 3 == 1] = fill
        z[:, : V // 2] = fill
        z[:, 5] = 1.0
        if T > 4:
            z[1] = fill                                      # the whole row
            z[2, 1:] = fill                                  # all but one
            z[3, ::2] = -INF
            z[3, 1::2] = fill
        check(ops, z, some_tokens(T, 3, V, 210), 5, tau)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("T,V", [(1, 128256), (7, 9001), (300, 2000)])
@pytest.mark.parametrize("size", [1e3, 2e4, 6e4, 1e6, 3e8, 3e9, 1e10, 1e15, 1e20, 1e30])
def test_large_logits(ops, dtype, T, V, size):  # noqa: F811
    if dtype is H and size > 6e4:
        return
    z = make(T, V, F, 220)
    for tau in (1.0, 0.7, 1e-6):
        check(ops, (z * 2 + size).clamp(max=6.5e4 if dtype is H else 3e38).to(dtype), some_tokens(T, 3, V, 221), 5, tau)
        check(ops, (z * 2 - size).clamp(min=-6.5e4 if dtype is H else -3e38).to(dtype), some_tokens(T, 3, V, 222), 5, tau)
    check(ops, (z * (size / 40)).clamp(-6.5e4, 6.5e4).to(dtype), some_tokens(T, 3, V, 223), 5)


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("T", [1, 400])
def test_where_sums_change_over(ops, dtype, T):  # noqa: F811
    # maxima, threads and parts on both sides of where the maximum itself takes over from its fp32 value in base 2,
    # close to one another
    V = 20003
    for bits in (24, 25, 26, 27, 28, 30, 31, 32, 33):
        for tau in (1.0, 1e-6, 2.0 ** -20):
            edge = 2.0 ** bits * np.log(2) * float(np.float32(tau))
            if dtype is H and edge > 3e4:
                continue
            for sign in (1, -1):
                z = sign * edge + make(T, V, F, 230 + bits) * min(1.0, tau) * 2
                z[:, ::7] = sign * edge * (1 + 2.0 ** -7)
                z[:, 9000:] -= edge * 2.0 ** -6
                check(ops, z.to(dtype), some_tokens(T, 2, V, 231), 4, tau)


def test_masks_over_large_logits(ops):  # noqa: F811
    T, V = 9, 40007
    for size in (1e10, -1e10, 1e20):
        z = make(T, V, F, 240)
        z[:, ::2] += size
        mask = random_mask(T, V, 241)
        mask[3] = 0
        mask[4] = 0x55555555                                 # the large ones alone
        mask[5] = -0x55555556                                # the others alone
        check(ops, z, some_tokens(T, 4, V, 243), 6, 0.9, mask)
