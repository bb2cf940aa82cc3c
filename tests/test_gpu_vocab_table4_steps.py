"""Logits of 16-bit hidden rows with one column far above the others, as a decoding step's have: the column's products may
not cut off the others' sums.

Tolerance: a hidden value counts within 2^-35 of its row's largest; products are exact, and a group's sum loses 2^-23
of its magnitudes for each of group + 2 additions; the scaled sums 2^-24 for each of G + 4 operations, the factors
2^-23; the type's rounding.  A column that meets its zero point (q = z) adds no magnitude.
For fp32 results the rows are pairs: of the lower parts, below 2^-11 of a group's largest, sums are cut off at 2^-13 of
2^-11 of it in the unit of the table's numbers, for each of the group's products of 8 columns.
"""
import pytest
import torch

from tests.test_gpu_vocab_table4 import BF, EPS, F, H, gen, half_step, ops, parts, table  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("times", [300.0, 3000.0, 3e4])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 9, 16, 40, 100])
@pytest.mark.parametrize("group,D,scales,zeros", [(32, 1001, F, True), (64, 2048, H, True), (128, 4096, H, False)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (H, H), (H, BF), (BF, F), (H, F)])
def test_one_column_above_the_others(ops, times, T, group, D, scales, zeros, dtype, out):  # noqa: F811
    V, at = 300, D // 3
    t = table(ops, V, D, group, scales, zeros, seed=int(times) % 89)
    # two rows in three do not see the column: their number there is its zero point
    q = t.zeros[at // group] & 15 if zeros else torch.full((V,), 8, dtype=torch.uint8, device="cuda")
    q = torch.where(torch.arange(V, device="cuda") % 3 == 0, (q + 5) % 16, q)
    old = t.values[:, at // 2]
    t.values[:, at // 2] = (old & 0xf0 | q) if at % 2 == 0 else (old & 0x0f | q << 4)
    x = torch.randn(T, D, device="cuda", generator=gen(500 + T))
    x[:, at] = times * torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.37)
    x = x.to(dtype)
    n, s = parts(t)
    unseen = torch.arange(V, device="cuda") % 3 != 0
    assert not n[unseen, at].any() and bool(n[~unseen, at].all())
    G = (D + group - 1) // group
    w, xd = n * s, x.double()
    want, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    tol = mag * ((group + 2) * 2.0 ** -23 + 2.0 ** -23 + (G + 4) * EPS) + 2.0 ** -35 * xd.abs().amax(1, keepdim=True) * w.abs().sum(1)[None]
    if out is F:
        wide = torch.nn.functional.pad(xd.abs(), (0, G * group - D)).view(T, G, group).amax(2)
        tol += wide @ t.scales.double() * (group // 8) * 2.0 ** -24
    tol += want.abs() * half_step(out) * (1 + 2.0 ** -7) + (2.0 ** -25 if out is H else 2.0 ** -126)
    got = ops.table4_logits(t, x, out_dtype=out).double()
    err = torch.where(got.isinf() & (want.abs() > torch.finfo(out).max * 0.999), 0.0, (got - want).abs())
    assert bool((err <= tol).all()), f"{(err / tol).max().item()} of the tolerance"
    # what the type does not round away is as small as sums in fp32 of what the rows do see
    rest = (err - want.abs() * half_step(out) * (1 + 2.0 ** -7)).clamp(min=0)
    assert (rest[:, unseen] / mag[:, unseen]).max().item() < 2.0 ** -18
    assert ops.device_error() == 0
