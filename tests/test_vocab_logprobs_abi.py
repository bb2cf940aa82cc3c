"""The C entry points of token log-probabilities and of 4-bit tables on the host: struct layouts,
refusals, workspace sizes; and what VocabOps refuses before it calls them.  No GPU needed."""
import ctypes
import re

import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import Table4, VocabOps

OK, BAD, UNS = L.LMLOSS_OK, L.LMLOSS_ERR_INVALID_ARG, L.LMLOSS_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    L.build()
    return L.load()


@pytest.mark.parametrize("name", ["lmloss_logprobs_args", "lmloss_logprobs_grad_args", "lmloss_table4",
                                  "lmloss_table4_quantize_args", "lmloss_table4_lookup_args", "lmloss_table4_logits_args"])
def test_struct_layout_matches_header(name):
    txt = open(L.HEADER).read()
    i = txt.index("} %s;" % name)
    body = re.sub(r"/\*.*?\*/", "", txt[txt.rindex("typedef struct {", 0, i):i], flags=re.S)
    c = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float, "lmloss_table4": L.lmloss_table4}
    fields = [(m[1], ctypes.c_void_p if "*" in m[0] else c[m[0].split()[-1]])
              for m in re.findall(r"([\w ]+?\s*\*?)\s*\b(\w+)\s*;", body[body.index("{") + 1:])]
    assert fields == [tuple(f) for f in getattr(L, name)._fields_]


def test_constants_match_header(lib):
    txt = open(L.HEADER).read()
    for n in ("LMLOSS_MAX_ALTERNATIVES", "LMLOSS_MAX_GIVEN"):
        assert re.search(r"#define %s %d\b" % (n, getattr(L, n)), txt)


def _fill(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _logprobs(**kw):
    return _fill(L.lmloss_logprobs_args(logits=0x10000, T=3, V=100, ld=100, dtype=L.LMLOSS_BF16, tokens=0x20000, n=2,
                                        temperature=1.0, M=4, logp_out=0x30000, top_logp_out=0x40000,
                                        top_tokens_out=0x50000), kw)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"T": 0, "logits": None, "tokens": None}, OK), ({"T": -1}, BAD), ({"V": 0}, BAD), ({"ld": 99}, BAD),
    ({"n": -1}, BAD), ({"n": 0, "tokens": None, "logp_out": None}, OK), ({"tokens": None}, BAD), ({"logp_out": None}, BAD),
    ({"tokens": 0x20004}, BAD), ({"tokens": 0x20004, "ids_dtype": L.LMLOSS_INT32}, OK), ({"ids_dtype": 2}, BAD),
    ({"M": -1}, BAD), ({"M": 65}, BAD), ({"M": 64}, OK), ({"M": 0, "top_logp_out": None, "top_tokens_out": None}, OK),
    ({"top_logp_out": None}, BAD), ({"top_tokens_out": None}, BAD), ({"dtype": 3}, BAD), ({"logits": None}, BAD),
    ({"logits": 0x10001}, BAD), ({"temperature": 0.0}, BAD), ({"temperature": -1.0}, BAD), ({"temperature": NAN}, BAD),
    ({"temperature": INF}, BAD), ({"temperature": 2.0 ** 20}, OK), ({"temperature": 2.0 ** 21}, BAD),
    ({"temperature": 2.0 ** -20}, OK), ({"temperature": 2.0 ** -21}, BAD), ({"mask_stride": -1}, BAD),
    ({"token_mask": 0x60000}, OK), ({"token_mask": 0x60000, "mask_stride": 3}, BAD),
    ({"token_mask": 0x60000, "mask_stride": 4}, OK), ({"V": (1 << 31) - 1, "ld": 1 << 31}, UNS), ({"T": 1 << 30}, UNS),
    ({"n": (1 << 20) + 1}, UNS), ({"ld": 1 << 60}, BAD),
])
def test_logprobs_validation(lib, kw, expect):
    assert L.lmloss_logprobs_check_args(_logprobs(**kw)) == expect


def _grad(**kw):
    return _fill(L.lmloss_logprobs_grad_args(logits=0x10000, T=3, V=100, ld=104, dtype=L.LMLOSS_BF16, tokens=0x20000,
                                             n=2, temperature=1.0, lse=0x30000, grad_logp=0x40000, grad_out=0x50000,
                                             ld_grad=100), kw)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"T": 0, "logits": None, "grad_out": None, "lse": None}, OK), ({"T": -1}, BAD), ({"ld": 99}, BAD),
    ({"ld_grad": 99}, BAD), ({"lse": None}, BAD), ({"grad_out": None}, BAD), ({"logits": None}, BAD),
    ({"grad_out": 0x50001}, BAD), ({"n": 0, "tokens": None, "grad_logp": None}, OK), ({"grad_logp": None}, BAD),
    ({"tokens": None}, BAD), ({"n": 1024}, OK), ({"n": 1025}, UNS), ({"grad_entropy": 0x60000}, BAD),
    ({"grad_entropy": 0x60000, "entropy": 0x70000}, OK), ({"temperature": 0.0}, BAD), ({"dtype": -1}, BAD),
    ({"grad_out": 0x10000}, BAD), ({"grad_out": 0x10000, "ld_grad": 104}, OK),          # in place: the same stride
    ({"grad_out": 0x10000, "T": 1}, OK),
    ({"grad_out": 0x10000 + 2 * (2 * 104 + 100)}, OK), ({"grad_out": 0x10000 + 2 * (2 * 104 + 99)}, BAD),
    ({"grad_out": 0x10000 - 2 * (2 * 100 + 100)}, OK), ({"grad_out": 0x10000 - 2 * (2 * 100 + 99)}, BAD),
    ({"token_mask": 0x60000, "mask_stride": 3}, BAD), ({"V": (1 << 31) - 1, "ld": 1 << 31, "ld_grad": 1 << 31}, UNS),
])
def test_gradient_validation(lib, kw, expect):
    assert L.lmloss_logprobs_check_grad_args(_grad(**kw)) == expect


def _table(**kw):
    return _fill(L.lmloss_table4(values=0x10000, ld_values=32, scales=0x20000, ld_scales=104, zeros=0x30000, ld_zeros=112,
                                 V=100, D=50, group=32, scale_dtype=L.LMLOSS_FP16), kw)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"values": None}, BAD), ({"scales": None}, BAD), ({"zeros": None, "ld_zeros": 0}, OK), ({"V": 0}, BAD),
    ({"D": 0}, BAD), ({"D": 64}, OK), ({"D": 65}, BAD), ({"ld_values": 40}, BAD), ({"ld_values": 16}, BAD),
    ({"values": 0x10008}, BAD), ({"scales": 0x20008}, BAD), ({"zeros": 0x30008}, BAD), ({"group": 16}, BAD),
    ({"group": 256}, BAD), ({"group": 0}, BAD), ({"scale_dtype": 3}, BAD), ({"ld_scales": 100}, BAD),
    ({"ld_scales": 100, "scale_dtype": L.LMLOSS_FP32}, OK), ({"ld_scales": 96}, BAD), ({"ld_zeros": 104}, BAD),
    ({"ld_zeros": 96}, BAD), ({"V": 1 << 31}, UNS), ({"D": (1 << 20) + 1}, UNS), ({"ld_values": 1 << 60}, BAD),
    ({"ld_scales": 1 << 60}, BAD),
])
def test_table_validation(lib, kw, expect):
    assert L.lmloss_table4_check(_table(**kw)) == expect
    t = _table(**kw)
    q = L.lmloss_table4_quantize_args(t, 0x40000, 1 << 21, L.LMLOSS_BF16)
    assert L.lmloss_table4_check_quantize_args(q) == expect
    a = L.lmloss_table4_lookup_args(t, 0x40000, 5, 0x50000, 1 << 21, L.LMLOSS_INT64, L.LMLOSS_BF16, 1.0)
    assert L.lmloss_table4_check_lookup_args(a) == expect
    a = L.lmloss_table4_logits_args(t, 0x40000, 5, 1 << 21, 0x50000, 1 << 32, L.LMLOSS_BF16, L.LMLOSS_BF16, 1.0)
    assert L.lmloss_table4_check_logits_args(a) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"weight": None}, BAD), ({"weight": 0x40001}, BAD), ({"ld_weight": 49}, BAD), ({"weight_dtype": 3}, BAD),
    ({"ld_weight": 1 << 60}, BAD),
])
def test_quantize_validation(lib, kw, expect):
    a = L.lmloss_table4_quantize_args(_table(), 0x40000, 50, L.LMLOSS_BF16)
    assert L.lmloss_table4_check_quantize_args(_fill(a, kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"T": 0, "ids": None, "rows": None}, OK), ({"T": -1}, BAD), ({"ids": None}, BAD), ({"rows": None}, BAD),
    ({"ids": 0x40004}, BAD), ({"ids": 0x40004, "ids_dtype": L.LMLOSS_INT32}, OK), ({"ids_dtype": 2}, BAD),
    ({"rows": 0x50001}, BAD), ({"ld_rows": 49}, BAD), ({"rows_dtype": 3}, BAD), ({"scale": NAN}, BAD), ({"scale": INF}, BAD),
    ({"T": 1 << 30}, UNS), ({"ld_rows": 1 << 60}, BAD),
])
def test_lookup_validation(lib, kw, expect):
    a = L.lmloss_table4_lookup_args(_table(), 0x40000, 5, 0x50000, 50, L.LMLOSS_INT64, L.LMLOSS_BF16, 1.0)
    assert L.lmloss_table4_check_lookup_args(_fill(a, kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"T": 0, "hidden": None, "logits": None}, OK), ({"T": -1}, BAD), ({"hidden": None}, BAD),
    ({"logits": None}, BAD), ({"hidden": 0x40001}, BAD), ({"logits": 0x50001}, BAD), ({"ld_hidden": 49}, BAD),
    ({"ld_logits": 99}, BAD), ({"hidden_dtype": 3}, BAD), ({"logits_dtype": 3}, BAD), ({"scale": NAN}, BAD),
    ({"T": 1 << 24}, UNS), ({"ld_hidden": 1 << 60}, BAD), ({"ld_logits": 1 << 60}, BAD),
])
def test_logits_validation(lib, kw, expect):
    a = L.lmloss_table4_logits_args(_table(), 0x40000, 5, 50, 0x50000, 100, L.LMLOSS_BF16, L.LMLOSS_BF16, 1.0)
    assert L.lmloss_table4_check_logits_args(_fill(a, kw)) == expect


def test_null_handles_and_arguments(lib):
    z, table = ctypes.c_size_t(), _table()
    logits = L.lmloss_table4_logits_args(table, 0x40000, 5, 50, 0x50000, 100, 0, 0, 1.0)
    calls = [(lib.lmloss_logprobs_forward, _logprobs()), (lib.lmloss_logprobs_backward, _grad()),
             (lib.lmloss_table4_quantize, L.lmloss_table4_quantize_args(table, 0x40000, 50, 0)),
             (lib.lmloss_table4_lookup, L.lmloss_table4_lookup_args(table, 0x40000, 5, 0x50000, 50, 0, 0, 1.0)),
             (lib.lmloss_table4_logits, logits)]
    for call, a in calls:
        assert call(None, ctypes.byref(a), None) == BAD
    for check in (lib.lmloss_logprobs_check_args, lib.lmloss_logprobs_check_grad_args, lib.lmloss_table4_check,
                  lib.lmloss_table4_check_quantize_args, lib.lmloss_table4_check_lookup_args,
                  lib.lmloss_table4_check_logits_args):
        assert check(None) == BAD
    for ws, a in ((lib.lmloss_logprobs_workspace, _logprobs()), (lib.lmloss_table4_logits_workspace, logits)):
        assert ws(None, ctypes.byref(z)) == BAD
        assert ws(ctypes.byref(a), None) == BAD


def test_workspace_grows_with_its_arguments(lib):
    sizes = [L.lmloss_logprobs_workspace(_logprobs(T=t, M=m, V=v, ld=v))
             for t, m, v in ((0, 0, 1), (1, 0, 1), (1, 5, 1000), (70, 20, 128256), (100000, 64, 262144))]
    assert sizes == sorted(sizes) and sizes[-1] < 2.5e6
    sizes = []
    for t, d in ((0, 1), (1, 1), (1, 4096), (40, 4096), (512, 4096), (512, 8192), (5000, 8192)):
        a = L.lmloss_table4_logits_args(T=t)
        a.table.V, a.table.D, a.table.group = 1000, d, 32
        sizes.append(L.lmloss_table4_logits_workspace(a))
    assert sizes == sorted(sizes)


@pytest.fixture(scope="module")
def ops(lib):
    h = VocabOps.__new__(VocabOps)      # no handle: tensors on the host, the checks before a call only
    h.device, h._index, h.handle, h.workspace_bytes = torch.device("cpu"), -1, None, 0
    return h


def test_wrapper_refuses(ops, monkeypatch):
    monkeypatch.setattr("lm_head_vocab_gb300.vocab._raw_stream", lambda index: 0)
    z, lse = torch.zeros(3, 40), torch.zeros(3)
    t = torch.zeros(3, 2, dtype=torch.int64)
    for error, kw in [(TypeError, dict(tokens=t.float())), (ValueError, dict(tokens=t[:2])),
                      (ValueError, dict(tokens=t.t().contiguous().t())), (ValueError, dict(num_top=65)),
                      (ValueError, dict(num_top=-1)), (TypeError, dict(token_mask=torch.zeros(3, 2))),
                      (ValueError, dict(token_mask=torch.zeros(2, 2, dtype=torch.int32))),
                      (ValueError, dict(token_mask=torch.zeros(3, 1, dtype=torch.int32)))]:
        with pytest.raises(error):
            ops.token_logprobs(z, **kw)
    with pytest.raises(TypeError):
        ops.token_logprobs(z.double())
    g = torch.zeros(3, 2)
    for error, kw in [(ValueError, dict(tokens=t)), (ValueError, dict(grad_logp=g)), (ValueError, dict(tokens=t, grad_logp=g[:, :1])),
                      (TypeError, dict(tokens=t, grad_logp=g.half())), (ValueError, dict(grad_entropy=lse)),
                      (ValueError, dict(grad_entropy=lse[:2], entropy=lse)), (ValueError, dict(grad="out")),
                      (ValueError, dict(grad=torch.zeros(3, 41))), (ValueError, dict(grad=torch.zeros(3, 40).half())),
                      (ValueError, dict(tokens=torch.zeros(3, 1025, dtype=torch.int64), grad_logp=torch.zeros(3, 1025)))]:
        with pytest.raises(error):
            ops.token_logprobs_backward(z, lse, **kw)
    table = ops.new_table4(20, 50, group_size=32, zeros=True)
    assert ops._table4(table).ld_values == 32 and ops._table4(table).ld_scales == 32
    one = ops.new_table4(1, 50)
    assert L.lmloss_table4_check(ops._table4(one)) == OK
    v, s, q = table.values, table.scales, table.zeros
    for error, bad in [(ValueError, Table4(v, s, q, 51, 32)), (ValueError, Table4(v, s, q, 50, 64)),
                       (ValueError, Table4(v, s, q, 50, 16)), (TypeError, Table4(v, s.double(), q, 50, 32)),
                       (TypeError, Table4(v.int(), s, q, 50, 32)), (TypeError, Table4(v, s, q.int(), 50, 32)),
                       (ValueError, Table4(v.contiguous(), s, q, 50, 32)), (ValueError, Table4(v, s[:, :19], q, 50, 32)),
                       (ValueError, Table4(v, s.contiguous(), q, 50, 32)), (ValueError, Table4(v, s, q[:1], 50, 32))]:
        with pytest.raises(error):
            ops.table4_lookup(bad, t)
        with pytest.raises(error):
            ops.table4_logits(bad, torch.zeros(2, 50))
    with pytest.raises(ValueError):
        ops.table4_logits(table, torch.zeros(2, 49))
    with pytest.raises(ValueError):
        ops.table4_logits(table, torch.zeros(2, 50), out=torch.zeros(2, 21))
    with pytest.raises(ValueError):
        ops.quantize_table(torch.zeros(20, 51), table)
    with pytest.raises(ValueError):
        ops.new_table4(0, 50)
    with pytest.raises(TypeError):
        ops.new_table4(3, 50, scale_dtype=torch.int8)
