"""Embedding lookup and its gradient on the GPU, against fp64 on the host.

Tolerances, from the arithmetic.  The lookup rounds scale * w to fp32 (half a step,
2^-24 relative) and that to the result's type.  The gradient adds n rows in fp32
(each addition within 2^-24 of the partial sum, which the terms' magnitudes bound),
multiplies by the scale (2^-24), adds the old value with the product (2^-24 of the
result) and rounds to the result's type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, H, F = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=20000, max_dim=4200, max_rows=0)
    yield h
    h.close()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """spacing of the type's subnormals"""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(rows, cols, dtype, pad, off, g, std=1.0):
    """[rows, cols] view with `pad` more columns a row, `off` elements into its buffer."""
    buf = torch.empty(off + rows * (cols + pad) + 8, device="cuda", dtype=dtype).normal_(0, std, generator=g)
    return buf, buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def make_ids(T, V, kind, dtype, g, ignored=0.1):
    if kind == "same":
        ids = torch.full((T,), V // 2, device="cuda")
    elif kind == "all":
        ids = torch.arange(T, device="cuda") % V
    elif kind == "none":
        ids = torch.full((T,), -100, device="cuda")
    elif kind == "runs":      # runs whose lengths step over the sort windows' borders
        ids = torch.repeat_interleave(torch.arange(T, device="cuda"), torch.arange(T, device="cuda") % 70 + 1)[:T] % V
        ids = ids[torch.randperm(T, generator=g, device="cuda")]
    else:
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * np.log(V + 1)) - 1).long().clamp_(0, V - 1)
        ids[torch.rand(T, generator=g, device="cuda") < ignored] = -100
    return ids.to(dtype)


PAIRS = [(a, b) for a in (BF, H, F) for b in (BF, H, F)]


@pytest.mark.parametrize("wt,ot", PAIRS)
@pytest.mark.parametrize("T,V,D,pad,off", [(1, 1, 1, 0, 0), (5, 7, 8, 0, 0), (130, 33, 64, 8, 0), (257, 1000, 1001, 0, 0),
                                           (64, 50, 72, 0, 1), (33, 40, 4099, 5, 0), (3, 2000, 4096, 0, 0)])
def test_lookup(ops, wt, ot, T, V, D, pad, off):
    g = gen(T * 1000 + D)
    _, w = strided(V, D, wt, pad, off, g, 0.3)
    buf, out = strided(T, D, ot, pad, off, g)
    before = buf.clone()
    ids = make_ids(T, V, "text", torch.int64 if D % 2 else torch.int32, g)
    scale = 1.7
    r = ops.embedding_forward(w, ids, scale=scale, out=out)
    assert r is out
    ref = w.double().cpu()[ids.long().clamp(min=0).cpu()] * float(np.float32(scale))
    ref[ids.cpu() == -100] = 0
    tol = ref.abs() * (half_step(ot) * (1 + U) + U) + smallest(ot)
    assert ((out.double().cpu() - ref).abs() <= tol).all()
    assert (out[ids == -100] == 0).all()
    # nothing around the result was written
    inside = torch.zeros_like(before, dtype=torch.bool)
    inside[off:off + T * (D + pad)].view(T, D + pad)[:, :D] = True
    assert torch.equal(buf[~inside].view(torch.uint8), before[~inside].view(torch.uint8))
    # the same without a buffer of one's own
    assert torch.equal(ops.embedding_forward(w, ids, scale=scale, out_dtype=ot), out)
    assert ops.device_error() == 0


def test_lookup_shapes_and_empty(ops):
    w = torch.randn(10, 24, device="cuda", generator=gen(1))
    ids = torch.tensor([[1, 2, 3], [9, -100, 0]], device="cuda")
    r = ops.embedding_forward(w, ids)
    assert r.shape == (2, 3, 24) and torch.equal(r[0], w[1:4]) and (r[1, 1] == 0).all()
    assert ops.embedding_forward(w, ids[:0]).shape == (0, 3, 24)
    assert ops.embedding_forward(w, ids, out_dtype=BF).dtype == BF


@pytest.mark.parametrize("bad", [10, -1, -101, 2 ** 40, -2 ** 40])
def test_ids_outside_the_table(ops, bad):
    w = torch.randn(10, 24, device="cuda", generator=gen(1))
    ids = torch.tensor([3, bad, -100, 9], device="cuda")
    r = ops.embedding_forward(w, ids)
    assert torch.isnan(r[1]).all() and torch.equal(r[0], w[3]) and torch.equal(r[3], w[9]) and (r[2] == 0).all()
    assert ops.device_error() == 4
    assert ops.device_error() == 0
    g = ops.embedding_backward(torch.ones(4, 24, device="cuda"), ids, num_embeddings=10)
    assert ops.device_error() == 4
    ref = torch.zeros(10, 24, device="cuda")
    ref[3] = ref[9] = 1
    assert torch.equal(g, ref)


def reference(rows, ids, V, scale, old):
    """(value, bound without the last rounding) in fp64"""
    rows, ids = rows.double().cpu(), ids.long().cpu()
    ok = ids >= 0
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    s = torch.zeros(V, rows.shape[1], dtype=torch.float64).index_add_(0, ids[ok], rows[ok])
    m = torch.zeros(V, rows.shape[1], dtype=torch.float64).index_add_(0, ids[ok], rows[ok].abs())
    scale = float(np.float32(scale))
    tol = (n[:, None] + 1) * U * m * abs(scale)
    ref = s * scale
    if old is not None:
        ref = ref + old.double().cpu()
    return ref, tol + U * ref.abs(), n


@pytest.mark.parametrize("gt,ot", PAIRS)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,D,pad,off,kind", [
    (1, 1, 1, 0, 0, "text"), (33, 20, 8, 0, 0, "text"), (700, 90, 72, 8, 0, "runs"), (1111, 300, 129, 0, 0, "text"),
    (333, 40, 64, 0, 1, "same"), (2300, 5, 1032, 0, 0, "text")])
def test_gradient(ops, gt, ot, accumulate, T, V, D, pad, off, kind):
    g = gen(T + D)
    _, rows = strided(T, D, gt, pad, off, g)
    buf, total = strided(V, D, ot, pad, off, g)
    ids = make_ids(T, V, kind, torch.int32 if D % 2 else torch.int64, g)
    if not accumulate:
        total.fill_(float("nan"))     # what was there does not matter
    before = buf.clone()
    old = total.clone()
    scale = -0.37
    r = ops.embedding_backward(rows, ids, total, scale=scale, accumulate=accumulate)
    assert r is total and ops.device_error() == 0
    ref, tol, n = reference(rows, ids, V, scale, old if accumulate else None)
    err = (total.double().cpu() - ref).abs()
    bound = tol + half_step(ot) * (ref.abs() + tol) + smallest(ot)
    assert (err <= bound).all(), (err - bound).max()
    untouched = n == 0
    if accumulate:
        assert torch.equal(total[untouched.cuda()], old[untouched.cuda()])
    else:
        assert (total[untouched.cuda()] == 0).all()
    inside = torch.zeros_like(before, dtype=torch.bool)
    inside[off:off + V * (D + pad)].view(V, D + pad)[:, :D] = True
    assert torch.equal(buf[~inside].view(torch.uint8), before[~inside].view(torch.uint8))
    # the same bits again
    again = old.clone()
    ops.embedding_backward(rows, ids, again, scale=scale, accumulate=accumulate)
    assert torch.equal(again, total)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049, 4096,
                               4097, 6143, 6144, 6145, 8191, 16385, 20000])
@pytest.mark.parametrize("kind", ["same", "text", "all", "runs", "none"])
def test_gradient_lengths(ops, T, kind):
    g = gen(T)
    V, D = 3000, 40
    rows = torch.randn(T, D, device="cuda", generator=g)
    ids = make_ids(T, V, kind, torch.int64, g)
    total = ops.embedding_backward(rows, ids, num_embeddings=V)
    ref, tol, _ = reference(rows, ids, V, 1.0, None)
    assert ((total.double().cpu() - ref).abs() <= tol + U * (ref.abs() + tol)).all()
    # exact for whole numbers: every row counted once
    ones = torch.randint(-8, 9, (T, D), device="cuda", generator=g).float()
    total = ops.embedding_backward(ones, ids, num_embeddings=V)
    ref, _, _ = reference(ones, ids, V, 1.0, None)
    assert torch.equal(total.double().cpu(), ref)
    assert ops.device_error() == 0


@pytest.mark.parametrize("V", [1, 2, 255, 256, 257, 65535, 65536, 65537, 131072, 300001])
def test_gradient_vocabularies(ops, V):
    g = gen(V)
    T, D = 3000, 8
    rows = torch.randint(-8, 9, (T, D), device="cuda", generator=g).to(BF)
    ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    ids[:2] = torch.tensor([0, V - 1], device="cuda")
    ids[5::11] = -100
    total = ops.embedding_backward(rows, ids, torch.full((V, D), 7.0, device="cuda"))
    ref, _, _ = reference(rows, ids, V, 1.0, None)
    assert torch.equal(total.double().cpu(), ref)


def test_gradient_nothing_to_add(ops):
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    rows = torch.empty(0, 16, device="cuda")
    t = torch.full((9, 16), 3.0, device="cuda")
    assert torch.equal(ops.embedding_backward(rows, ids, t.clone(), accumulate=True), t)
    assert (ops.embedding_backward(rows, ids, t.clone()) == 0).all()


def test_non_finite_rows_stay_with_their_token(ops):
    ids = torch.tensor([4, 4, 2, -100, 1], device="cuda")
    rows = torch.ones(5, 16, device="cuda")
    rows[1, 3] = float("inf")
    rows[2, 5] = float("nan")
    rows[3] = float("nan")            # ignored: its gradient is not read into any sum
    t = ops.embedding_backward(rows, ids, num_embeddings=6)
    assert torch.isinf(t[4, 3]) and torch.isnan(t[2, 5])
    t[4, 3] = t[2, 5] = 0
    assert torch.isfinite(t).all() and (t[1] == 1).all() and t[4].sum() == 30


def test_adjoint_and_differences(ops):
    g = gen(3)
    T, V, D, scale = 700, 211, 96, 1.3
    w = torch.randn(V, D, device="cuda", generator=g)
    c = torch.randn(T, D, device="cuda", generator=g)
    ids = make_ids(T, V, "text", torch.int64, g)
    dw = ops.embedding_backward(c, ids, num_embeddings=V, scale=scale).double()
    # f(w) = sum(c * lookup(w)) is linear: <c, lookup(w)> = <dw, w>, and its slope along any direction is <dw, d>
    f = lambda x: (c.double() * ops.embedding_forward(x, ids, scale=scale).double()).sum().item()  # noqa: E731
    # each of the T D products carries the lookup's 2 fp32 roundings; each sum those of `reference`
    size = (c.abs().double() * ops.embedding_forward(w.abs(), ids, scale=scale).double()).sum().item()
    assert abs(f(w) - (dw * w.double()).sum().item()) <= (2 + T + 3) * U * size
    d = torch.zeros_like(w)
    d[ids[ids >= 0][0], 17] = 1.0
    step = 2.0 ** -6
    slope = (f(w + step * d) - f(w - step * d)) / (2 * step)
    v = ids[ids >= 0][0]
    n = int((ids == v).sum())
    # w +- step rounds to fp32, the lookup twice, on the terms of this one column
    terms = (c[ids == v, 17].abs().double() * (w[v, 17].abs().double() + 1) * scale).sum().item()
    assert abs(slope - dw[v, 17].item()) <= (6 * U * terms) / step + (n + 2) * U * terms + 1e-9 * size


def test_offsets_past_32_bits(ops):
    # a table of more than 2^31 elements and more than 2^32 bytes
    V, D = 600001, 4096
    w = torch.empty(V, D, device="cuda", dtype=H)
    last = torch.tensor([V - 1, 0, V - 2, V // 2], device="cuda")
    w[last] = torch.randn(4, D, device="cuda", generator=gen(5)).to(H)
    assert torch.equal(ops.embedding_forward(w, last), w[last])
    rows = torch.randn(4, D, device="cuda", generator=gen(6)).to(H)
    w.fill_(1.0)
    ops.embedding_backward(rows, last, w)
    assert torch.equal(w[last], rows)
    w[last] = 0
    assert not w.view(torch.int64).any().item()


def test_other_stream_and_graph(ops):
    g = gen(9)
    T, V, D = 900, 500, 264
    w = torch.randn(V, D, device="cuda", generator=g)
    rows = torch.randn(T, D, device="cuda", generator=g)
    ids = make_ids(T, V, "text", torch.int64, g)
    base = torch.randn(V, D, device="cuda", generator=g)
    fwd = ops.embedding_forward(w, ids, scale=2.0)
    bwd = ops.embedding_backward(rows, ids, base.clone(), accumulate=True)
    whole = ops.embedding_backward(rows, ids, num_embeddings=V)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = ops.embedding_forward(w, ids, scale=2.0, stream=s)
    c = ops.embedding_backward(rows, ids, num_embeddings=V, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, fwd) and torch.equal(c, whole)
    # captured once, replayed on new inputs
    out, total = torch.empty_like(fwd), base.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.embedding_forward(w, ids, scale=2.0, out=out)
        ops.embedding_backward(rows, ids, total, accumulate=True)
    total.copy_(base)
    graph.replay()
    assert torch.equal(out, fwd) and torch.equal(total, bwd)
    ids.copy_(make_ids(T, V, "runs", torch.int64, g))
    rows.normal_(generator=g)
    total.copy_(base)
    graph.replay()
    assert torch.equal(out, ops.embedding_forward(w, ids, scale=2.0))
    assert torch.equal(total, ops.embedding_backward(rows, ids, base.clone(), accumulate=True))


def test_refusals(ops):
    w = torch.randn(10, 16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    rows = torch.randn(4, 16, device="cuda")
    with pytest.raises(TypeError):
        ops.embedding_forward(w, ids.to(torch.int16))
    with pytest.raises(TypeError):
        ops.embedding_forward(w.double(), ids)
    with pytest.raises(ValueError):
        ops.embedding_forward(w.t(), ids)
    with pytest.raises(ValueError):
        ops.embedding_forward(w, ids.cpu())
    with pytest.raises(ValueError):
        ops.embedding_forward(w.cpu(), ids)
    with pytest.raises(ValueError):
        ops.embedding_forward(w, ids, out=torch.empty(4, 15, device="cuda"))
    with pytest.raises(ValueError):
        ops.embedding_forward(w, torch.zeros(8, dtype=torch.int64, device="cuda")[::2])
    with pytest.raises(ValueError):
        ops.embedding_backward(rows[:3], ids, w)
    with pytest.raises(ValueError):
        ops.embedding_backward(rows, ids)
    with pytest.raises(ValueError):
        ops.embedding_backward(rows, ids, torch.empty(10, 15, device="cuda"))
    with pytest.raises(ValueError):
        ops.embedding_backward(rows[:1].expand(4, 16), ids, w)      # a broadcast gradient: rows on top of one another
    from lm_head_vocab_gb300 import LMLossError
    many = torch.zeros(20001, dtype=torch.int64, device="cuda")
    with pytest.raises(LMLossError) as e:                            # more than the handle's workspace
        ops.embedding_backward(torch.empty(20001, 4200, device="cuda"), many, num_embeddings=3)
    assert e.value.status == 1


@pytest.mark.parametrize("T,V", [(131072, 50000), (131073, 50000), (150001, 7)])
def test_gradient_of_many_positions(T, V):
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=T, max_dim=16, max_rows=0)
    g = gen(T)
    rows = torch.randint(-4, 5, (T, 13), device="cuda", generator=g).to(BF)
    ids = make_ids(T, V, "text", torch.int64, g)
    for accumulate in (False, True):
        old = torch.full((V, 13), 3.0, device="cuda")
        total = h.embedding_backward(rows, ids, old.clone(), accumulate=accumulate)
        ref, _, _ = reference(rows, ids, V, 1.0, old if accumulate else None)
        assert torch.equal(total.double().cpu(), ref)
    h.close()


@pytest.mark.parametrize("T", [5, 2049])
@pytest.mark.parametrize("D", [1, 3, 7, 8, 9, 15, 17, 100, 1001, 2047])
def test_gradient_widths(ops, T, D):
    # rows that start at every offset from a vector boundary, exact in whole numbers
    g = gen(T + D)
    V = 130
    ids = make_ids(T, V, "text", torch.int64, g)
    for gt, ot in PAIRS:
        rows = torch.randint(-3, 4, (T, D), device="cuda", generator=g).to(gt)
        for accumulate in (False, True):
            old = torch.randint(-3, 4, (V, D), device="cuda", generator=g).to(ot)
            total = ops.embedding_backward(rows, ids, old.clone(), accumulate=accumulate)
            ref, _, _ = reference(rows, ids, V, 1.0, old if accumulate else None)
            assert torch.equal(total.double().cpu(), ref.to(ot).double())
        w = torch.randn(V, D, device="cuda", generator=g).to(gt)
        out = ops.embedding_forward(w, ids, out_dtype=ot)
        ref = torch.where((ids >= 0)[:, None], w[ids.clamp(min=0)].float(), 0.0).to(ot)
        assert torch.equal(out, ref)
