"""Which layouts a reordering takes and refuses: on the host by the bytes that a state's sides
really touch, on a GPU by what comes out."""
import itertools
import random

import pytest
import torch

import lm_head_vocab_gb300._lib as L

OK, BAD = L.LMLOSS_OK, L.LMLOSS_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    L.build()
    return L.load()


def state(src, dst, inner, rows, outer, src_outer, dst_outer):
    s = L.lmloss_beam_state(src=src, dst=dst, inner=inner, src_row_stride=rows[0], dst_row_stride=rows[1])
    s.outer[:], s.src_outer_stride[:], s.dst_outer_stride[:] = outer, src_outer, dst_outer
    return s


def check(*states, B=2, K=2, K_out=2):
    return L.lmloss_beam_check_states((L.lmloss_beam_state * len(states))(*states), B, K, K_out)


def touched(base, row_stride, rows, outer, strides, inner):
    out = set()
    for r, *o in itertools.product(range(rows), *map(range, outer)):
        at = base + r * row_stride + sum(a * b for a, b in zip(o, strides))
        out.update(range(at, at + inner))
    return out


def test_overlapping_sides_are_always_refused():
    rng = random.Random(5)
    taken = 0
    for _ in range(30000):
        outer = [rng.choice([1, 1, 2, 3]) for _ in range(3)]
        inner = rng.randint(1, 6)
        strides = [[rng.choice([1, 4, 6, 8, 12, 16, 24, 48, rng.randint(1, 60)]) for _ in range(4)] for _ in range(2)]
        if rng.random() < 0.7:
            strides[1] = strides[0]
        src, dst = 1000 + rng.randint(0, 120), 1000 + rng.randint(0, 120)
        if src == dst:
            continue
        got = check(state(src, dst, inner, (strides[0][0], strides[1][0]), outer, strides[0][1:], strides[1][1:]))
        if got == OK:
            taken += 1
            a = touched(src, strides[0][0], 4, outer, strides[0][1:], inner)
            assert not a & touched(dst, strides[1][0], 4, outer, strides[1][1:], inner)
    assert taken > 1000


@pytest.mark.parametrize("swap", [False, True])
def test_interleaved_halves_are_taken(swap):
    # [rows, 2 halves, heads 3, positions 7 of 8, 16 bytes]
    row, half = 2 * 3 * 8 * 16, 3 * 8 * 16
    a, b = (0x10000 + half, 0x10000) if swap else (0x10000, 0x10000 + half)
    heads = dict(outer=[3, 1, 1], src_outer=[128, 0, 0], dst_outer=[128, 0, 0])
    assert check(state(a, b, 7 * 16, (row, row), **heads)) == OK
    # up to the next row's first byte, and one more
    assert check(state(a, b + 16, 7 * 16, (row, row), **heads)) == OK
    assert check(state(a, b + 17, 7 * 16, (row, row), **heads)) == BAD
    # [rows, heads, 2 halves, 16 bytes]
    assert check(state(a, a + 16, 16, (96, 96), [3, 1, 1], [32, 0, 0], [32, 0, 0])) == OK
    assert check(state(a, a + 15, 16, (96, 96), [3, 1, 1], [32, 0, 0], [32, 0, 0])) == BAD
    # two columns of a matrix
    assert check(state(a, a + 4, 4, (32, 32), [1, 1, 1], [0, 0, 0], [0, 0, 0])) == OK


def test_runs_written_on_top_of_one_another_are_refused():
    def st(dst_row, dst_outer, outer=(1, 1, 1), inner=16):
        return state(0x10000, 0x40000, inner, (64, dst_row), list(outer), [16, 16, 16], [dst_outer] * 3)
    assert check(st(64, 0)) == OK and check(st(16, 0)) == OK
    assert check(st(0, 0)) == BAD and check(st(15, 0)) == BAD
    assert check(st(0, 0), B=3, K=1, K_out=1) == BAD          # one beam a sequence: rows of three sequences
    assert check(st(0, 0), B=1, K=1, K_out=1) == OK
    assert check(st(0, 0, inner=0), B=3, K=1, K_out=1) == OK  # nothing is written
    for k in range(3):
        outer = [3 if i == k else 1 for i in range(3)]
        assert check(st(64, 16, outer)) == OK
        assert check(st(64, 0, outer)) == BAD and check(st(64, 15, outer)) == BAD


def test_states_that_write_to_one_another_are_refused():
    def st(src, dst, inner=64):
        return state(src, dst, inner, (64, 64), [1, 1, 1], [0, 0, 0], [0, 0, 0])
    a, b, c, d = 0x10000, 0x20000, 0x30000, 0x40000
    assert check(st(a, c), st(b, d)) == OK and check(st(a, a), st(b, b)) == OK
    assert check(st(a, c), st(a, d)) == OK                 # one source for two
    assert check(st(a, b), st(b, a)) == BAD                # a swap
    assert check(st(a, b), st(c, a)) == BAD and check(st(c, a), st(a, b)) == BAD
    assert check(st(a, c), st(b, c)) == BAD
    assert check(st(a, a), st(a, a)) == BAD                # twice in place
    assert check(st(a, a), st(a, b)) == BAD and check(st(a, b), st(b, b)) == BAD
    assert check(st(a, b), st(b, a, inner=0)) == OK        # nothing moves


@pytest.mark.parametrize("n", [2, 3, 100, 511, 512, 513, 1500])
def test_states_that_write_to_one_another_among_many(n):
    rng = random.Random(n)
    place = [0x100000 + 256 * i for i in rng.sample(range(10 * n), 2 * n)]

    def run(edit=lambda st: None):
        st = [state(place[2 * i], place[2 * i + (i % 3 != 0)], 16, (16, 16), [1, 1, 1], [0, 0, 0], [0, 0, 0]) for i in range(n)]
        edit(st)
        return check(*st)
    assert run() == OK
    for a, b in ((0, n - 1), (n - 1, 0), (n // 2, (n // 2 + 1) % n), (rng.randrange(1, n), 0)):
        assert run(lambda st: setattr(st[a], "src", st[b].dst)) == BAD
        assert run(lambda st: setattr(st[a], "dst", st[b].dst)) == BAD
        # every third is in place: what another reads there is written
        assert run(lambda st: setattr(st[a], "src", st[b].src)) == (BAD if b % 3 == 0 else OK)


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    h = VocabOps(0, max_tokens=0, max_rows=0)
    yield h
    h.close()


def moved(t, parents):
    K = t.shape[0] // parents.shape[0]
    return t[(parents.long() + torch.arange(parents.shape[0], device="cuda")[:, None] * K).flatten()]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [1, 2, 3])
def test_halves_at_any_place_of_a_cache(ops, dim):
    g = torch.Generator(device="cuda").manual_seed(dim)
    shape = [12, 3, 9, 10]
    shape.insert(dim, 2)
    kv = torch.randn(shape, device="cuda", generator=g)
    parents = torch.randint(0, 4, (3, 4), device="cuda", generator=g, dtype=torch.int32)
    src, dst = kv.select(dim, 0)[:, :, :7], kv.select(dim, 1)[:, :, :7]
    before = kv.clone()
    want = moved(src, parents)
    ops.beam_reorder([src], parents, out=[dst])
    assert torch.equal(dst, want) and ops.device_error() == 0
    dst.copy_(before.select(dim, 1)[:, :, :7])
    assert torch.equal(kv, before)                    # nothing else was written


@pytest.mark.gpu
def test_no_sequences(ops):
    # what a beam step over no sequences leaves can be reordered too
    parents = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    states = [torch.empty(0, 7, device="cuda"), torch.empty(0, 2, 3, device="cuda", dtype=torch.bfloat16)]
    got = ops.beam_reorder(states, parents)
    assert [t.shape for t in got] == [t.shape for t in states] and [t.dtype for t in got] == [t.dtype for t in states]
    assert ops.beam_reorder(states, parents, out="inplace") == states
    kv = torch.empty(2, 0, 5, device="cuda")
    assert ops.beam_reorder([kv], parents, dim=1)[0].shape == (2, 0, 5)
    with pytest.raises(ValueError):
        ops.beam_reorder([torch.empty(4, 7, device="cuda")], parents)
