"""4-bit vocabulary tables on the GPU against fp64: made, looked up, multiplied with hidden rows.

A lookup is one product (q - z) s of an exact whole number and an fp32 value, and one with the
scale, each rounded once in fp32, then to the type.  Logits, from the arithmetic: a hidden value's upper part is
off by half a step of 2^-10 of the power of two at or below its group's largest, 2^-11 of that largest at most;
the lower part rounds this to 11 bits, so a pair leaves 2^-23 of a group's, thus of a row's largest; an fp16
alone 2^-24 of a row's largest and nothing else, as 16-bit values fit it.  Within a group products are
exact and their fp32 sums lose at most 2^-23 of the group's sum of magnitudes for each addition, group + 2
of them; the groups' scaled sums 2^-24 for each of G + 4 operations; the type's rounding.  Quantized values
are exact.
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
    h = VocabOps(0, max_tokens=0, max_dim=8192, max_rows=512)
    yield h
    h.close()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def table(ops, V, D, group, scales, zeros, seed=1):
    """A random table whose padding, which no call may use, holds values that would show."""
    t = ops.new_table4(V, D, group_size=group, zeros=zeros, scale_dtype=scales)
    g = gen(seed)
    t.values._base.copy_(torch.randint(0, 256, t.values._base.shape, device="cuda", generator=g, dtype=torch.uint8))
    t.scales._base.fill_(float("nan"))
    t.scales.copy_(torch.rand(t.scales.shape, device="cuda", generator=g) * 0.02 + 0.001)
    if zeros:
        t.zeros._base.fill_(255)
        t.zeros.copy_(torch.randint(0, 16, t.zeros.shape, device="cuda", generator=g, dtype=torch.uint8))
    return t


def parts(t):
    """(q - z) [V, D] and the scales [V, D], in fp64."""
    D, g = t.columns, t.group_size
    q = torch.stack([t.values & 15, t.values >> 4], -1).flatten(1)[:, :D].double()
    s = t.scales.double().t().repeat_interleave(g, 1)[:, :D]
    z = 8.0 if t.zeros is None else t.zeros.double().t().repeat_interleave(g, 1)[:, :D]
    return q - z, s


# ------------------------------------------------------------------- lookup
@pytest.mark.parametrize("out", [BF, H, F])
@pytest.mark.parametrize("V,D,group,scales,zeros", [(1, 1, 32, H, False), (7, 31, 32, F, True), (100, 33, 64, BF, True),
                                                    (333, 128, 128, H, False), (50, 1001, 32, F, True),
                                                    (1000, 4096, 128, H, True), (64, 130, 64, BF, False)])
def test_lookup(ops, out, V, D, group, scales, zeros):
    t = table(ops, V, D, group, scales, zeros)
    n, s = parts(t)
    for shape, ids_dtype in (((5,), torch.int64), ((3, 67), torch.int32)):
        ids = torch.randint(0, V, shape, device="cuda", generator=gen(3)).to(ids_dtype)
        ids.view(-1)[1] = -100
        for scale in (1.0, 7.3):
            got = ops.table4_lookup(t, ids, scale=scale, out_dtype=out)
            i = ids.view(-1).long()
            want = torch.where((i >= 0)[:, None], (n * s)[i.clamp(min=0)] * float(np.float32(scale)), 0.0).view(*shape, D)
            assert got.shape == want.shape and got.dtype == out
            tol = want.abs() * (half_step(out) * (1 + 2.0 ** -8) + 2 * EPS) + (2.0 ** -25 if out is H else 0)
            assert bool(((got.double() - want).abs() <= tol).all())
    assert ops.device_error() == 0


@pytest.mark.parametrize("D,extra,shift", [(1001, 0, 0), (1001, 3, 5), (96, 7, 1), (128, 8, 8)])
def test_lookup_into_strided_rows(ops, D, extra, shift):
    t = table(ops, 200, D, 32, H, True)
    ids = torch.randint(0, 200, (37,), device="cuda", generator=gen(5))
    for dtype in (BF, F):
        flat = torch.full((shift + 37 * (D + extra) + 64,), 5.0, device="cuda", dtype=dtype)
        out = flat[shift:shift + 37 * (D + extra)].view(37, D + extra)[:, :D]
        ops.table4_lookup(t, ids, out=out)
        assert torch.equal(out, ops.table4_lookup(t, ids, out_dtype=dtype))
        out.fill_(5.0)
        assert bool((flat == 5.0).all())


def test_lookup_of_bad_ids(ops):
    import lm_head_vocab_gb300._lib as L
    t = table(ops, 20, 70, 64, H, False)
    ids = torch.tensor([3, 20, -1, 2 ** 40, -100], device="cuda")
    r = ops.table4_lookup(t, ids, out_dtype=F)
    assert ops.device_error() == L.LMLOSS_ERR_BAD_TARGET and ops.device_error() == 0
    assert torch.isnan(r).all(1).tolist() == [False, True, True, True, False] and not r[4].any()
    assert ops.table4_lookup(t, ids[:0]).shape == (0, 70)


# ----------------------------------------------------------------- quantize
def quantized(w, group, zeros, scale_dtype):
    """q, s, z of the definition, quotients in fp64."""
    V, D = w.shape
    G = (D + group - 1) // group
    x = torch.nn.functional.pad(w.float(), (0, G * group - D)).view(V, G, group)
    if zeros:
        lo, hi = x.amin(2).clamp(max=0), x.amax(2).clamp(min=0)
        s = ((hi - lo).double() / 15).float().to(scale_dtype)   # (in 32 bits torch multiplies by 1 / 15)
        by = torch.where(s > 0, s, 1).double()[..., None]
        z = torch.where(s > 0, (-lo.double() / by[..., 0]).round().clamp(0, 15), 0.0)
        q = ((x.double() / by).round() + z[..., None]).clamp(0, 15)
        q = torch.where(s[..., None] > 0, q, z[..., None])
    else:
        s = (x.abs().amax(2).double() / 7).float().to(scale_dtype)
        by = torch.where(s > 0, s, 1).double()[..., None]
        q = (x.double() / by).round().clamp(-8, 7)
        q, z = torch.where(s[..., None] > 0, q, 0.0) + 8, None
    return q.view(V, -1)[:, :D], s.t(), None if z is None else z.t()


@pytest.mark.parametrize("dtype", [BF, H, F])
@pytest.mark.parametrize("scales", [BF, H, F])
@pytest.mark.parametrize("V,D,group,zeros", [(1, 1, 32, True), (5, 31, 32, False), (33, 200, 64, True), (130, 257, 128, True),
                                             (70, 1024, 128, False), (17, 96, 32, True)])
def test_quantize(ops, dtype, scales, V, D, group, zeros):
    w = (torch.randn(V, D, device="cuda", generator=gen(V + D)) * 0.02).to(dtype)
    w[0] = 0                                                 # a group of zeros
    if V > 4:
        w[1] = w[1].abs()                                    # one sign: the range reaches to 0
        w[2] = 1e-5                                          # all equal
        w[3, ::3] *= 1e-4
        w[4] = (torch.arange(D, device="cuda") % 15 - 7).to(dtype) / 2   # halves and whole numbers of steps
    t = ops.quantize_table(w, group_size=group, zeros=zeros, scale_dtype=scales)
    assert ops.device_error() == 0
    q, s, z = quantized(w, group, zeros, scales)
    assert torch.equal(t.scales, s)
    if zeros:
        assert torch.equal(t.zeros.double(), z)
    got = torch.stack([t.values & 15, t.values >> 4], -1).flatten(1)
    assert torch.equal(got[:, :D].double(), q)
    assert not got[:, D:].any()


def test_quantize_strided_weights_into_a_table(ops):
    V, D = 60, 301
    flat = torch.randn(V * 333 + 9, device="cuda", generator=gen(7))
    for dtype in (BF, F):
        w = flat.to(dtype)[5:5 + V * 333].view(V, 333)[:, :D]
        t = table(ops, V, D, 64, H, True, 9)
        before = t.values._base.clone(), t.scales._base.clone(), t.zeros._base.clone()
        assert ops.quantize_table(w, t) is t
        fresh = ops.quantize_table(w.contiguous(), group_size=64, zeros=True)
        assert torch.equal(t.values, fresh.values) and torch.equal(t.scales, fresh.scales) and torch.equal(t.zeros, fresh.zeros)
        # what lies beside the table is left alone
        assert torch.equal(t.values._base[:, (D + 1) // 2:], before[0][:, (D + 1) // 2:])
        assert torch.equal(t.scales._base[:, V:].isnan(), before[1][:, V:].isnan())
        assert torch.equal(t.zeros._base[:, V:], before[2][:, V:])


def test_quantize_what_is_not_finite(ops):
    import lm_head_vocab_gb300._lib as L
    w = torch.randn(6, 64, device="cuda", generator=gen(11))
    clean = ops.quantize_table(w, group_size=32)
    w[1, 40] = float("nan")
    w[2, 3] = INF
    w[3, 3] = -INF
    w[4, 0] = 1e6                                            # a scale past fp16
    t = ops.quantize_table(w, group_size=32)
    assert ops.device_error() == L.LMLOSS_ERR_RANGE and ops.device_error() == 0
    bad = torch.zeros(2, 6, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[0, 2] = bad[0, 3] = bad[0, 4] = True
    assert torch.equal(t.scales.isnan(), bad) and torch.equal(t.scales[~bad], clean.scales[~bad])
    rows = ops.table4_lookup(t, torch.arange(6, device="cuda"), out_dtype=F)
    assert torch.equal(rows.isnan(), bad.t().repeat_interleave(32, 1))
    fine = ops.quantize_table(w[4:], group_size=32, scale_dtype=BF)
    assert ops.device_error() == 0 and bool(fine.scales.isfinite().all())


# ------------------------------------------------------------------- logits
def check_logits(ops, t, x, out=F, scale=1.0, into=None):
    got = ops.table4_logits(t, x, scale=scale, out_dtype=out, out=into)
    assert ops.device_error() == 0
    n, s = parts(t)
    D, group = t.columns, t.group_size
    G = (D + group - 1) // group
    w, xd = n * s, x.reshape(-1, D).double()
    want = xd @ w.t() * float(np.float32(scale))
    mag = xd.abs() @ w.abs().t() * abs(float(np.float32(scale)))
    tops = xd.abs().amax(1, keepdim=True) * w.abs().sum(1)[None] * abs(float(np.float32(scale)))
    tol = mag * ((group + 2) * 2.0 ** -23 + 2.0 ** -23 + (G + 4) * EPS) + tops * 2.0 ** -23
    tol += want.abs() * half_step(out) + (2.0 ** -25 if out is H else 2.0 ** -126)
    got = got.reshape(want.shape).double()
    over = (got - want).abs() > tol
    assert not bool(over.any()), f"{int(over.sum())} beyond, {((got - want).abs() / tol).max().item()} of the tolerance"
    return got


def hidden(T, D, dtype, seed=21):
    return torch.randn(T, D, device="cuda", generator=gen(seed)).to(dtype)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 40, 64, 65, 130])
@pytest.mark.parametrize("x,out", [(BF, BF), (H, H), (F, F)])
def test_logits_rows(ops, T, x, out):
    check_logits(ops, table(ops, 700, 256, 128, H, False), hidden(T, 256, x), out)


@pytest.mark.parametrize("V", [1, 2, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("D", [1, 2, 31, 32, 33, 64, 96, 130, 257, 1001])
def test_logits_sizes(ops, V, D):
    for i, (group, scales, zeros) in enumerate([(32, F, True), (64, BF, False), (128, H, True)]):
        T = (3, 20, 70)[(V + D + i) % 3]
        check_logits(ops, table(ops, V, D, group, scales, zeros, V + D), hidden(T, D, (F, BF, H)[(V + i) % 3]), F)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scales", [BF, H, F])
@pytest.mark.parametrize("zeros", [False, True])
def test_logits_table_kinds(ops, group, scales, zeros):
    t = table(ops, 300, 1184, group, scales, zeros)
    if zeros:
        t.zeros[0] = 255                                     # any byte is a zero point
    for T, x, out in ((1, BF, BF), (33, F, F), (12, H, BF)):
        check_logits(ops, t, hidden(T, 1184, x), out, scale=0.37)


@pytest.mark.parametrize("V,D,T", [(40000, 2048, 1), (20011, 4096, 5), (9001, 8192, 70), (2500, 5120, 300)])
def test_logits_large(ops, V, D, T):
    check_logits(ops, table(ops, V, D, 128, H, False), hidden(T, D, BF), BF)
    check_logits(ops, table(ops, V, D, 32, BF, True), hidden(T, D, F), F)


@pytest.mark.parametrize("x,out", [(BF, BF), (F, F), (H, F)])
@pytest.mark.parametrize("shift,extra,oshift,oextra", [(0, 0, 1, 0), (1, 3, 3, 1), (8, 8, 0, 8)])
def test_logits_strides(ops, x, out, shift, extra, oshift, oextra):
    T, V, D = 11, 517, 333
    t = table(ops, V, D, 64, H, True)
    flat = torch.full((shift + T * (D + extra) + 64,), float("nan"), device="cuda", dtype=x)
    rows = flat[shift:shift + T * (D + extra)].view(T, D + extra)[:, :D]
    rows.copy_(hidden(T, D, x))
    oflat = torch.full((oshift + T * (V + oextra) + 64,), 5.0, device="cuda", dtype=out)
    into = oflat[oshift:oshift + T * (V + oextra)].view(T, V + oextra)[:, :V]
    check_logits(ops, t, rows, out, into=into)
    into.fill_(5.0)
    assert bool((oflat == 5.0).all())


def test_logits_shapes(ops):
    t = table(ops, 90, 64, 32, H, False)
    x = hidden(12, 64, BF)
    flat = ops.table4_logits(t, x)
    assert flat.dtype is BF
    assert torch.equal(ops.table4_logits(t, x.view(3, 4, 64)).view(12, 90), flat)
    assert torch.equal(ops.table4_logits(t, x[5]), flat[5])
    assert ops.table4_logits(t, x[:0]).shape == (0, 90)


@pytest.mark.parametrize("x", [BF, H, F])
def test_logits_of_unequal_rows(ops, x):
    # rows of very different sizes: each keeps its own precision
    t = table(ops, 200, 320, 64, H, True)
    rows = hidden(9, 320, x)
    big = {BF: 1e30, H: 1e3, F: 1e30}[x]
    rows[1] *= big
    rows[2] /= big
    rows[3] = 0
    rows[4, ::2] *= 2.0 ** -12
    rows[5] = 0
    rows[5, 7] = 1.0
    check_logits(ops, t, rows, F)


@pytest.mark.parametrize("x", [BF, H, F])
def test_logits_of_infinities_and_nan(ops, x):
    V, D = 150, 200
    t = table(ops, V, D, 32, H, True)
    rows = hidden(6, D, x)
    clean = ops.table4_logits(t, rows, out_dtype=F)
    rows[1, 3] = float("nan")
    rows[2, 100] = INF
    rows[3, 100] = -INF
    rows[4, 0], rows[4, 199] = INF, -INF
    got = ops.table4_logits(t, rows, out_dtype=F)
    n, s = parts(t)
    want = rows.double() @ (n * s).t()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got == INF, want == INF) and torch.equal(got == -INF, want == -INF)
    assert torch.equal(got[[0, 5]], clean[[0, 5]])


def test_logits_repeat_and_do_not_depend_on_neighbours(ops):
    t = table(ops, 1000, 512, 64, H, True)
    x = hidden(60, 512, BF)
    a = ops.table4_logits(t, x, out_dtype=F)
    assert torch.equal(a, ops.table4_logits(t, x, out_dtype=F))


@pytest.mark.parametrize("x", [BF, H, F])
@pytest.mark.parametrize("T", [1, 6, 12, 40, 100])
def test_fp32_logits_have_fp32_precision(ops, x, T):
    # Of normal inputs a pair's rounding is uniform within 2^-23 of a group's largest, some three standard
    # deviations: 3 * 2^-23 / sqrt(3) a column, 2^-22 of the logits' size; the 32 groups' additions add less than
    # sqrt(32) 2^-24 / sqrt(3) = 2^-22.3 of it.  Together less than 2^-21; products cut off at some 2^-24 of
    # what a subnormal's exponent could hold are past it.
    for group, D, zeros in ((32, 1024, True), (128, 4096, False)):
        t = table(ops, 600, D, group, F, zeros)
        rows = hidden(T, D, x)
        n, s = parts(t)
        want = rows.double() @ (n * s).t()
        got = ops.table4_logits(t, rows, out_dtype=F).double()
        assert (got - want).pow(2).mean().sqrt().item() < 2.0 ** -21 * want.pow(2).mean().sqrt().item()


@pytest.mark.parametrize("x", [BF, F])
def test_logits_of_more_rows_than_a_launch_takes(ops, x):
    check_logits(ops, table(ops, 131, 70, 32, H, True), hidden(2100, 70, x), x)


@pytest.mark.parametrize("x", [BF, F])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_few_rows_too_long_for_shared_memory(ops, x, T):
    check_logits(ops, table(ops, 200, 30001, 128, BF, True), hidden(T, 30001, x), F)


@pytest.mark.parametrize("T", [3, 8, 12, 30, 60, 90, 300])
@pytest.mark.parametrize("V", [1, 63, 64, 65, 127, 128, 129, 513])
def test_logits_at_tile_borders(ops, V, T):
    t = table(ops, V, 160, 32, BF, True)
    flat = torch.full((T * (V + 3) + 64,), 5.0, device="cuda")
    out = flat[1:1 + T * (V + 3)].view(T, V + 3)[:, :V]
    check_logits(ops, t, hidden(T, 160, F), F, into=out)
    out.fill_(5.0)
    assert bool((flat == 5.0).all())   # nothing beside the rows


@pytest.mark.parametrize("x", [BF, H, F])
@pytest.mark.parametrize("T", [4, 8, 14, 20, 50, 130])
def test_a_row_that_is_not_finite_among_others(ops, x, T):
    t = table(ops, 300, 200, 64, H, False)
    rows = hidden(T, 200, x)
    clean = ops.table4_logits(t, rows, out_dtype=F)
    bad = [0, T // 2, T - 1]
    for i, r in enumerate(bad):
        rows[r, 199 - i] = (INF, -INF, float("nan"))[i]
    got = ops.table4_logits(t, rows, out_dtype=F)
    n, s = parts(t)
    want = rows.double() @ (n * s).t()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got == INF, want == INF) and torch.equal(got == -INF, want == -INF)
    others = [r for r in range(T) if r not in bad]
    assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("T", [3, 8, 20, 100])
def test_a_row_does_not_depend_on_its_neighbours(ops, T):
    t = table(ops, 500, 384, 128, F, True)
    x = hidden(T, 384, F)
    a = ops.table4_logits(t, x)
    y = x * 1e20
    y[T // 2] = x[T // 2]
    assert torch.equal(ops.table4_logits(t, y)[T // 2], a[T // 2])


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [1, 7, 8, 9, 33, 241, 247, 248, 249, 256, 257, 500])
def test_lookup_at_every_alignment(ops, dtype, D):
    t = table(ops, 100, D, 32, H, True)
    ids = torch.randint(0, 100, (9,), device="cuda", generator=gen(61))
    n, s = parts(t)
    want = (n * s)[ids].to(dtype)          # fp64 to the type: the product is exact in fp32 (8 and 11 bits)
    for shift in range(16 // dtype.itemsize):
        for extra in (0, 1, 3):
            flat = torch.full((32 + shift + 9 * (D + extra),), 5.0, device="cuda", dtype=dtype)
            at = 16 + shift
            out = flat[at:at + 9 * (D + extra)].view(-1)[:9 * (D + extra)].view(9, D + extra)[:, :D]
            ops.table4_lookup(t, ids, out=out)
            assert torch.equal(out, want)
            out.fill_(5.0)
            assert bool((flat == 5.0).all())


@pytest.mark.parametrize("dtype,scales", [(F, F), (F, H), (BF, BF), (BF, H), (BF, F), (H, H), (H, F)])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_at_the_ends_of_the_types(ops, dtype, scales, zeros):
    # scales that are subnormal or round to zero, weights next to the largest, groups of equal and of zero weights
    lo, hi = (-24, 15) if H in (dtype, scales) else (-149 if dtype is F else -133, 127)
    sizes = [2.0 ** e for e in (lo, lo + 1, lo + 2, lo + 3, lo + 4, lo + 7, lo + 12, lo + 25, lo + 31, hi - 3)]
    w = torch.randn(len(sizes) * 4, 64, device="cuda", generator=gen(71)).clamp_(-3.9, 3.9).double()
    for i, size in enumerate(sizes):
        w[4 * i:4 * i + 4] *= size
        w[4 * i + 2] = size * 3
        w[4 * i + 3, ::2] = 0
    w = w.to(dtype)
    t = ops.quantize_table(w, group_size=32, zeros=zeros, scale_dtype=scales)
    q, s, z = quantized(w, 32, zeros, scales)
    got = torch.stack([t.values & 15, t.values >> 4], -1).flatten(1)[:, :64]
    assert torch.equal(t.scales, s) and torch.equal(got.double(), q)
    assert not zeros or torch.equal(t.zeros.double(), z)
    assert ops.device_error() == 0


# ------------------------------------------------- together, streams, graphs
def test_a_decoding_step(ops):
    # a tied 4-bit vocabulary: embeddings of the last tokens in, log-probabilities and beams out
    V, D = 2003, 256
    w = torch.randn(V, D, device="cuda", generator=gen(31)) * 0.05
    t = ops.quantize_table(w, group_size=64, zeros=True)
    last = torch.randint(0, V, (8,), device="cuda", generator=gen(33))

    def step():
        h = ops.table4_lookup(t, last, scale=16.0, out_dtype=BF)
        z = ops.table4_logits(t, h, out_dtype=F)
        return h, z, ops.token_logprobs(z, last, num_top=4), ops.beam_step(z, torch.zeros(2, 4, device="cuda"), num_candidates=4)
    h, z, r, b = step()
    n, s = parts(t)
    want = h.double() @ (n * s).t()
    lp = torch.log_softmax(want, 1)
    # logits of about |h| |w| sqrt(D) = 13 within 2^-16, and the log-probabilities' own 2^-17
    assert bool(((r.logp.double() - lp.gather(1, last[:, None])[:, 0]).abs() < 2.0 ** -12).all())
    assert torch.equal(r.top_tokens, z.sort(dim=1, descending=True, stable=True)[1][:, :4])
    assert bool((b.lse.view(-1) - r.lse).abs().max() < 2.0 ** -16)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    last.copy_(torch.randint(0, V, (8,), device="cuda", generator=gen(35)))
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert torch.equal(out[1], again[1]) and torch.equal(out[2].logp, again[2].logp) and torch.equal(out[3].tokens, again[3].tokens)
    assert ops.device_error() == 0


def test_on_a_stream_of_the_callers(ops):
    w = torch.randn(3000, 512, device="cuda", generator=gen(41))
    x, ids = hidden(20, 512, BF), torch.arange(0, 3000, 7, device="cuda")
    want = ops.quantize_table(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t = ops.quantize_table(w, stream=s)
    z = ops.table4_logits(t, x, stream=s)
    e = ops.table4_lookup(t, ids, stream=s)
    s.synchronize()
    assert torch.equal(t.values, want.values)
    assert torch.equal(z, ops.table4_logits(want, x)) and torch.equal(e, ops.table4_lookup(want, ids))


def test_more_rows_than_the_handle():
    import lm_head_vocab_gb300._lib as L
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_dim=64, max_rows=4, max_vocab=1000)
    t = h.quantize_table(torch.randn(100, 64, device="cuda"))
    assert h.table4_logits(t, torch.randn(4, 64, device="cuda")).shape == (4, 100)
    big = h.quantize_table(torch.randn(100, 8192, device="cuda"))
    try:
        h.table4_logits(big, torch.randn(600, 8192, device="cuda"))
    except L.LMLossError as e:
        assert "bytes of workspace needed" in str(e)
    h.close()


def test_handles_of_several_threads():
    import threading
    from lm_head_vocab_gb300 import VocabOps
    w = torch.randn(3000, 256, device="cuda", generator=gen(81))
    xs = [hidden(n, 256, BF, seed=90 + n) for n in (1, 20, 70)]
    h = VocabOps(0, max_tokens=0, max_dim=256, max_rows=128, max_vocab=3000)
    t = h.quantize_table(w)
    want = [(h.table4_logits(t, x), h.token_logprobs(h.table4_logits(t, x, out_dtype=F), num_top=5)) for x in xs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            mine = VocabOps(0, max_tokens=0, max_dim=256, max_rows=128, max_vocab=3000)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    z = mine.table4_logits(t, xs[i])
                    r = mine.token_logprobs(mine.table4_logits(t, xs[i], out_dtype=F), num_top=5)
                torch.cuda.current_stream().synchronize()
            assert torch.equal(z, want[i][0]) and torch.equal(r.top_tokens, want[i][1].top_tokens) and torch.equal(r.lse, want[i][1].lse)
            mine.close()
        except BaseException as e:
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i % 3,)) for i in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    h.close()
    assert not failed, failed


def test_offsets_past_32_bits(ops):
    # weights of 2.5e9 elements, rows of as many, logits of 2.4e9: the far ends are those of the same rows alone
    V, D, far = 600064, 4160, 4000
    w = torch.empty(V, D, device="cuda", dtype=BF)
    w.normal_(0.0, 0.02, generator=gen(101))
    t = ops.quantize_table(w, group_size=64, zeros=True)
    end = ops.quantize_table(w[-far:], group_size=64, zeros=True)
    assert torch.equal(t.values[-far:], end.values) and torch.equal(t.scales[:, -far:], end.scales)
    assert torch.equal(t.zeros[:, -far:], end.zeros)
    ids = torch.arange(V, device="cuda")
    rows = ops.table4_lookup(t, ids, out=w)
    assert torch.equal(rows[-far:], ops.table4_lookup(end, ids[:far], out_dtype=BF))
    del w, rows
    x = hidden(4000, D, BF)
    z = ops.table4_logits(t, x)
    assert torch.equal(z[:, -far:], ops.table4_logits(end, x))
    one = ops.table4_logits(t, x[:1])
    assert torch.equal(one[:, -far:], ops.table4_logits(end, x[:1]))
    assert ops.device_error() == 0


def test_two_graphs_of_one_handle_in_turn(ops):
    # they share the handle's workspace and counters, and run one after the other
    t = table(ops, 5003, 768, 64, H, True)
    xs = [hidden(T, 768, BF, seed=110 + T) for T in (20, 90)]
    runs = []
    for x in xs:
        def step(x=x):
            z = ops.table4_logits(t, x, out_dtype=F)
            return z, ops.token_logprobs(z[:3], num_top=20)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((graph, out, step))
    for i, x in enumerate(xs):
        x.copy_(hidden(len(x), 768, BF, seed=120 + i))
    for _ in range(3):
        for graph, _, _ in runs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out, step in runs:
        z, r = step()
        assert torch.equal(out[0], z) and torch.equal(out[1].top_tokens, r.top_tokens) and torch.equal(out[1].lse, r.lse)
        assert torch.equal(out[1].top_logp, r.top_logp) and torch.equal(out[1].entropy, r.entropy)
    assert ops.device_error() == 0
