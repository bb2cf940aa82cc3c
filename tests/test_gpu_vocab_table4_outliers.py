"""Logits of fp32 hidden rows with one column far above the others, as large models' have, against the bound that the
header states for a value x: 2^-23 of its group's largest + 2^-46 of its row's.

Beside it: the sums of the lower parts, below 2^-11 of the group's largest each, times whole numbers of at most 15 + z, lose
2^-23 of their magnitudes for each of group + 2 additions (the upper parts' are exact); the groups' scaled sums 2^-24
for each of G + 4 operations, and the factors at the end 2^-23.
"""
import pytest
import torch

from tests.test_gpu_vocab_table4 import EPS, F, H, gen, ops, parts, table  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("times", [300.0, 3000.0, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("T", [1, 3, 12, 40, 100])
@pytest.mark.parametrize("group,D,scales", [(32, 1001, F), (128, 4096, H)])
def test_one_column_above_the_others(ops, times, T, group, D, scales):  # noqa: F811
    V, at = 400, D // 3
    t = table(ops, V, D, group, scales, True, seed=int(times) % 97)
    # two rows in three do not see the column: their number there is its zero point
    q = t.zeros[at // group] & 15
    q = torch.where(torch.arange(V, device="cuda") % 3 == 0, (q + 5) % 16, q)
    old = t.values[:, at // 2]
    t.values[:, at // 2] = (old & 0xf0 | q) if at % 2 == 0 else (old & 0x0f | q << 4)
    x = torch.randn(T, D, device="cuda", generator=gen(400 + T))
    x[:, at] = times * torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.37)
    n, s = parts(t)
    unseen = torch.arange(V, device="cuda") % 3 != 0
    assert not n[unseen, at].any() and bool(n[~unseen, at].all())
    G = (D + group - 1) // group
    w, xd = n * s, x.double()
    wide = torch.nn.functional.pad(xd.abs(), (0, G * group - D)).view(T, G, group).amax(2)     # the groups' largest
    tops = wide.repeat_interleave(group, 1)[:, :D]
    scale = t.scales.double().t()                                                             # [V, G]
    want, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    bound = (2.0 ** -23 * tops + 2.0 ** -46 * xd.abs().amax(1, keepdim=True)) @ w.abs().t()
    bound += (wide * 2.0 ** -11) @ (scale * (15 + t.zeros.double().t())).t() * group * (group + 2) * 2.0 ** -23
    bound += mag * ((G + 4) * EPS + 2.0 ** -23) + want.abs() * EPS
    got = ops.table4_logits(t, x).double()
    err = (got - want).abs()
    assert bool((err <= bound).all()), f"{(err / bound).max().item()} of the bound"
    # and far inside it for the most part: a tenth of the values' part alone, as sums of many of either sign are
    values = (2.0 ** -23 * tops + 2.0 ** -46 * xd.abs().amax(1, keepdim=True)) @ w.abs().t() + mag * 2.0 ** -23
    assert (err[:, unseen] / values[:, unseen]).mean().item() < 0.1
    assert ops.device_error() == 0
