"""The vocabulary operators' C entry points on the host: struct layouts, refusals,
workspace sizes.  No GPU needed (no compute calls)."""
import ctypes
import re

import pytest

import lm_head_vocab_gb300._lib as L

OK, BAD, UNS = L.LMLOSS_OK, L.LMLOSS_ERR_INVALID_ARG, L.LMLOSS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    L.build()
    return L.load()


@pytest.mark.parametrize("name", ["lmloss_embedding_args", "lmloss_beam_args", "lmloss_beam_state"])
def test_struct_layout_matches_header(name):
    txt = open(L.HEADER).read()
    i = txt.index("} %s;" % name)
    body = txt[txt.rindex("typedef struct {", 0, i):i]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"(\w+)(?:\[\d+\])?\s*;", body)
    assert fields == [f for f, _ in getattr(L, name)._fields_]


def test_constants_match_header(lib):
    txt = open(L.HEADER).read()
    assert re.search(r"LMLOSS_FP16 = %d\b" % L.LMLOSS_FP16, txt)
    assert re.search(r"#define LMLOSS_MAX_BEAMS %d\b" % L.LMLOSS_MAX_BEAMS, txt)
    assert re.search(r"LMLOSS_ERR_BAD_PARENT = %d\b" % L.LMLOSS_ERR_BAD_PARENT, txt)
    assert "parent" in L.lmloss_status_string(L.LMLOSS_ERR_BAD_PARENT)


def _emb(**kw):
    a = L.lmloss_embedding_args(ids=0x10000, T=4, V=10, D=16, table=0x20000, ld_table=16, rows=0x30000, ld_rows=16,
                                ids_dtype=L.LMLOSS_INT64, table_dtype=L.LMLOSS_BF16, rows_dtype=L.LMLOSS_FP32,
                                scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"T": 0, "ids": None, "rows": None}, OK), ({"T": -1}, BAD), ({"V": 0}, BAD), ({"D": 0}, BAD),
    ({"ld_table": 15}, BAD), ({"ld_rows": 15}, BAD), ({"ids": None}, BAD), ({"table": None}, BAD), ({"rows": None}, BAD),
    ({"ids": 0x10004}, BAD), ({"ids": 0x10004, "ids_dtype": L.LMLOSS_INT32}, OK), ({"ids_dtype": 2}, BAD),
    ({"table": 0x20001}, BAD), ({"rows": 0x30002}, BAD), ({"table_dtype": 3}, BAD), ({"rows_dtype": -1}, BAD),
    ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD), ({"scale": 0.0}, OK), ({"accumulate": 2}, BAD),
    ({"T": 1 << 30}, UNS), ({"V": (1 << 31) - 1}, UNS), ({"ld_table": 1 << 60}, BAD), ({"ld_rows": 1 << 60}, BAD),
    ({"table_dtype": L.LMLOSS_FP16, "rows_dtype": L.LMLOSS_BF16}, OK),
])
def test_embedding_validation(lib, kw, expect):
    assert L.lmloss_embedding_check_args(_emb(**kw)) == expect


def _beam(**kw):
    a = L.lmloss_beam_args(logits=0x10000, B=2, V=100, ld=100, K=4, M=8, dtype=L.LMLOSS_BF16, eos_token=-1,
                           scores=0x20000, scores_out=0x30000, parents_out=0x40000, tokens_out=0x50000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"B": 0, "logits": None, "scores": None}, OK), ({"B": -1}, BAD), ({"V": 0}, BAD), ({"ld": 99}, BAD),
    ({"K": 0}, BAD), ({"K": 65}, BAD), ({"M": 0}, BAD), ({"M": 65}, BAD), ({"dtype": 5}, BAD),
    ({"length_penalty": -1.0}, BAD), ({"length_penalty": float("inf")}, BAD), ({"length_penalty": float("nan")}, BAD),
    ({"length_penalty": 0.6}, BAD), ({"length_penalty": 0.6, "lengths": 0x60000}, OK),
    ({"lengths_out": 0x60000}, BAD), ({"eos_token": 100}, BAD), ({"eos_token": -2}, BAD), ({"eos_token": 99}, OK),
    ({"finished": 0x60000}, BAD), ({"finished": 0x60000, "eos_token": 0}, OK),
    ({"token_mask": 0x60000}, OK), ({"token_mask": 0x60000, "mask_stride": 3}, BAD),
    ({"token_mask": 0x60000, "mask_stride": 4}, OK), ({"mask_stride": -1}, BAD),
    ({"logits": None}, BAD), ({"logits": 0x10001}, BAD), ({"dtype": L.LMLOSS_FP32, "logits": 0x10002}, BAD),
    ({"scores": None}, BAD), ({"scores_out": None}, BAD), ({"parents_out": None}, BAD), ({"tokens_out": None}, BAD),
    ({"V": (1 << 31) - 1, "ld": 1 << 31}, UNS), ({"ld": 1 << 60}, BAD),
])
def test_beam_validation(lib, kw, expect):
    assert L.lmloss_beam_check_args(_beam(**kw)) == expect


def _state(**kw):
    """One [8 rows, 3, 64 bytes] state out of place."""
    s = L.lmloss_beam_state(src=0x10000, dst=0x20000, inner=64, src_row_stride=192, dst_row_stride=192)
    s.outer[:] = [3, 1, 1]
    s.src_outer_stride[:] = [64, 0, 0]
    s.dst_outer_stride[:] = [64, 0, 0]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(s, k)[:] = v
        else:
            setattr(s, k, v)
    return (L.lmloss_beam_state * 1)(s)


@pytest.mark.parametrize("kw,K,Ko,expect", [
    ({}, 4, 4, OK), ({}, 4, 5, OK), ({}, 0, 4, BAD), ({}, 65, 4, BAD), ({}, 4, 0, BAD), ({}, 4, 65, BAD),
    ({"src": None}, 4, 4, BAD), ({"dst": None}, 4, 4, BAD), ({"inner": -1}, 4, 4, BAD),
    ({"inner": 0, "src": None, "dst": None}, 4, 4, OK), ({"outer": [0, 1, 1], "src": None}, 4, 4, OK),
    ({"outer": [-1, 1, 1]}, 4, 4, BAD), ({"src_row_stride": -192}, 4, 4, BAD), ({"dst_row_stride": 0}, 4, 4, BAD),
    ({"dst": 0x10000}, 4, 4, OK), ({"dst": 0x10000}, 4, 5, BAD),                 # in place
    ({"dst": 0x10000, "dst_row_stride": 256}, 4, 4, BAD),
    ({"dst": 0x10000, "dst_outer_stride": [128, 0, 0]}, 4, 4, BAD),
    ({"dst": 0x10000 + 8 * 192 - 1}, 4, 4, BAD), ({"dst": 0x10000 + 8 * 192}, 4, 4, OK),   # overlap
    ({"src": 0x20000 + 8 * 192 - 64}, 4, 4, BAD), ({"src": 0x20000 + 8 * 192}, 4, 4, OK),
    ({"src_row_stride": 1 << 62}, 4, 4, BAD),
])
def test_reorder_validation(lib, kw, K, Ko, expect):
    assert L.lmloss_beam_check_states(_state(**kw), 2, K, Ko) == expect


def test_null_handles_and_arguments(lib):
    z = ctypes.c_size_t()
    assert lib.lmloss_vocab_create(None, 0, 0) == BAD
    assert lib.lmloss_vocab_destroy(None) == BAD
    assert lib.lmloss_vocab_get_device_error(None) == BAD
    assert lib.lmloss_embedding_check_args(None) == BAD
    assert lib.lmloss_embedding_workspace(None, ctypes.byref(z)) == BAD
    assert lib.lmloss_embedding_workspace(ctypes.byref(_emb()), None) == BAD
    assert lib.lmloss_embedding_forward(None, ctypes.byref(_emb()), None) == BAD
    assert lib.lmloss_embedding_backward(None, ctypes.byref(_emb()), None) == BAD
    assert lib.lmloss_beam_check_args(None) == BAD
    assert lib.lmloss_beam_workspace(None, ctypes.byref(z)) == BAD
    assert lib.lmloss_beam_workspace(ctypes.byref(_beam()), None) == BAD
    assert lib.lmloss_beam_step(None, ctypes.byref(_beam()), None) == BAD
    assert lib.lmloss_beam_check_states(None, 1, 1, 1, 1) == BAD
    assert lib.lmloss_beam_check_states(None, 0, 1, 1, 1) == OK
    assert lib.lmloss_beam_reorder(None, None, 0, None, 1, 1, 1, None) == BAD


def test_workspace_grows_with_its_arguments(lib):
    # a handle sized for the largest call serves the smaller ones
    sizes = [L.lmloss_embedding_workspace(_emb(T=t, D=d, ld_table=d, ld_rows=d, ids=None, table=None, rows=None))
             for t, d in ((0, 1), (1, 1), (33, 16), (1000, 1000), (65536, 1000), (65536, 8192))]
    assert sizes == sorted(sizes)
    sizes = [L.lmloss_beam_workspace(_beam(B=b, K=k, M=m, V=v, ld=v))
             for b, k, m, v in ((0, 1, 1, 1), (1, 1, 1, 1), (1, 4, 8, 32003), (16, 8, 16, 128256), (64, 8, 16, 262144))]
    assert sizes == sorted(sizes)
    # rows of one sequence or of many: the same workspace serves both
    one = L.lmloss_beam_workspace(_beam(B=64, K=1, M=64, V=262144, ld=262144, dtype=L.LMLOSS_FP32))
    assert one >= L.lmloss_beam_workspace(_beam(B=4, K=16, M=64, V=200000, ld=200000, dtype=L.LMLOSS_BF16))


def test_rows_too_long_for_a_step_are_refused(lib):
    longest = (1 << 31) - (1 << 16)
    assert L.lmloss_beam_workspace(_beam(K=64, V=longest, ld=longest)) > 0
    with pytest.raises(L.LMLossError) as e:
        L.lmloss_beam_workspace(_beam(K=64, V=longest + 1, ld=longest + 1))
    assert e.value.status == UNS
