"""Gradients added to an fp32 table: what the header says of their rounding, bit for bit, on every
way of adding.

No sums are taken (one position a token with something in it), so a result is one of three fp32
values: the fused product and sum; the product rounded, then the sum; the same with subnormals taken
as 0 before and after the addition."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def flushed(x):
    return torch.where(x.abs() < 2.0 ** -126, 0.0, x)


@pytest.mark.parametrize("T", [100, 3000, 9000])
@pytest.mark.parametrize("D", [64, 33, 1000])
def test_added_to_an_fp32_table(T, D):
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    ops = VocabOps(0, max_tokens=9000, max_dim=1000, max_rows=0)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    V, scale = 20000, 1.7
    ids = torch.randperm(V, device="cuda", generator=g)[:T]
    ids[T // 2:T // 2 + 3] = ids[0]                       # one token of four positions, three of them zero
    old = torch.randn(V, D, device="cuda", generator=g) * torch.exp2(torch.randint(-148, 60, (V, D), device="cuda", generator=g).float())
    rows = torch.randn(T, D, device="cuda", generator=g) * torch.exp2(torch.randint(-140, 60, (T, D), device="cuda", generator=g).float())
    rows[T // 2:T // 2 + 3] = 0
    total = old.clone()
    ops.embedding_backward(rows, ids, total, scale=scale, accumulate=True)
    assert ops.device_error() == 0
    ops.close()
    at = torch.cat([ids[:T // 2], ids[T // 2 + 3:]])
    r, o, got = torch.cat([rows[:T // 2], rows[T // 2 + 3:]]).cpu(), old[at].cpu(), total[at].cpu()
    s = torch.tensor(scale)                               # fp32
    product = r * s
    ways = ((r.double() * s.double() + o.double()).float(), product + o, flushed(flushed(product) + flushed(o)))
    assert torch.stack([got == w for w in ways]).any(0).all()
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[ids] = False
    assert torch.equal(total[rest].view(torch.int32), old[rest].view(torch.int32))   # the others are left alone
