"""PyTorch-facing wrapper of the vocabulary operators of the lmloss C ABI:
embedding lookup and gradient, beam search's step, reordering of beam states,
log-probabilities of given tokens with their gradient, and vocabulary tables in 4 bits.

Tensors only supply device pointers, strides and the current CUDA stream; every
step runs in the library's kernels, and there is no CPU path.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import List, Optional, Sequence, Union

import torch

from . import _lib
from ._lib import LMLossError

_FLOATS = {torch.bfloat16: _lib.LMLOSS_BF16, torch.float32: _lib.LMLOSS_FP32, torch.float16: _lib.LMLOSS_FP16}
_ONES = (1, 1, 1)
_IDS = {torch.int64: _lib.LMLOSS_INT64, torch.int32: _lib.LMLOSS_INT32}


# a call's time on the host is a good part of a small call's: devices are compared by
# number, and the current stream is asked for as a number
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(t: torch.Tensor, name: str, dtype, rows: int, cols: int, index: int):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.size(0) != rows or t.size(1) != cols:
        raise ValueError(f"{name}: expected shape {(rows, cols)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the handle on cuda:{index}")


def _matrix(t: torch.Tensor, name: str, index: int):
    """(type, rows, columns, row stride) of a 2-d float tensor with unit column stride and
    rows that do not overlap."""
    dtype = _FLOATS.get(t.dtype)
    if dtype is None:
        raise TypeError(f"{name}: must be bfloat16, float16 or float32, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the handle on cuda:{index}")
    if t.dim() != 2:
        raise ValueError(f"{name}: must have two dimensions")
    rows, cols = t.size(0), t.size(1)
    ld, unit = t.stride()
    # (a lazily negated view is every second number of a conjugated one: never of unit stride)
    if unit != 1 and t.is_neg():
        raise ValueError(f"{name}: a lazily conjugated or negated view; resolve it first")
    if rows <= 1:
        ld = cols
    if cols < 1 or (cols > 1 and unit != 1) or ld < cols:
        raise ValueError(f"{name}: must have at least one column, unit column stride and a row stride of at least "
                         f"its columns")
    return dtype, rows, cols, ld


def _flat(t: torch.Tensor, name: str, T: int, D: int):
    """[..., D] as the [T, D] that a call takes."""
    if t.dim() == 2:
        return t
    try:
        return t.view(T, D)
    except RuntimeError:
        raise ValueError(f"{name}: the positions of a tensor of more dimensions must lie one row stride apart") from None


@dataclass
class BeamStep:
    scores: torch.Tensor                        # [B, M] float32
    parents: torch.Tensor                       # [B, M] int32
    tokens: torch.Tensor                        # [B, M] int64
    lse: torch.Tensor                           # [B, K] float32
    finished: torch.Tensor                      # [B, M] uint8
    lengths: Optional[torch.Tensor] = None      # [B, M] int32


@dataclass
class TokenLogprobs:
    logp: Optional[torch.Tensor]                # [T, n] float32 (the given tokens' shape)
    lse: torch.Tensor                           # [T] float32
    entropy: Optional[torch.Tensor]             # [T] float32
    top_logp: Optional[torch.Tensor] = None     # [T, M] float32
    top_tokens: Optional[torch.Tensor] = None   # [T, M] int64
    row_max: Optional[torch.Tensor] = None      # [T] float32: the largest allowed logit
    log_sum: Optional[torch.Tensor] = None      # [T] float32: lse - row_max / temperature


@dataclass
class Table4:
    """A [V, columns] table in 4 bits: scales[g, v] * (q - zeros[g, v]) with g = column // group_size,
    zeros 8 where there are none.  Every row and every group begins on a 16-byte boundary
    (`VocabOps.new_table4` makes such tensors, as views of wider ones)."""
    values: torch.Tensor                        # [V, ceil(columns / 2)] uint8: the lower column in the low half
    scales: torch.Tensor                        # [G, V] float16, bfloat16 or float32
    zeros: Optional[torch.Tensor]               # [G, V] uint8
    columns: int
    group_size: int = 128


class VocabOps:
    """One handle of the vocabulary operators, with workspace for embedding
    gradients of up to max_tokens positions and max_dim columns, for beam steps of
    up to max_rows rows of logits at vocabularies of up to max_vocab and, allocated
    by the first call that needs it, for log-probabilities of the same and for logits from
    4-bit tables of up to max_rows rows and max_dim columns.

    Calls run on `stream`, or on the current stream, and do not synchronise; calls
    on one handle must not overlap.  A `stream` other than the current one has to
    be ordered after the inputs' producers by the caller.
    """

    def __init__(self, device: Union[int, torch.device, None] = None, max_tokens: int = 1 << 16,
                 max_dim: int = 8192, max_rows: int = 1024, max_vocab: int = 1 << 18):
        if not torch.cuda.is_available():
            raise RuntimeError("VocabOps needs a CUDA device")
        if device is None:
            device = torch.cuda.current_device()
        elif not isinstance(device, int):
            device = torch.device(device).index or 0
        self.device = torch.device("cuda", device)
        self._index = device
        lib = _lib.load()
        self._forward, self._backward = lib.lmloss_embedding_forward, lib.lmloss_embedding_backward
        self._step, self._reorder = lib.lmloss_beam_step, lib.lmloss_beam_reorder
        self._logprobs, self._logprobs_grad = lib.lmloss_logprobs_forward, lib.lmloss_logprobs_backward
        self._quantize, self._lookup4, self._logits4 = (lib.lmloss_table4_quantize, lib.lmloss_table4_lookup,
                                                        lib.lmloss_table4_logits)
        need = 0
        if max_tokens > 0:
            a = _lib.lmloss_embedding_args(T=max_tokens, V=max_vocab, D=max_dim, ld_table=max_dim, ld_rows=max_dim,
                                           scale=1.0)
            need = _lib.lmloss_embedding_workspace(a)
        if max_rows > 0:
            b = _lib.lmloss_beam_args(B=max_rows, K=1, M=_lib.LMLOSS_MAX_BEAMS, V=max_vocab, ld=max_vocab,
                                      dtype=_lib.LMLOSS_FP32, eos_token=-1)
            need = max(need, _lib.lmloss_beam_workspace(b))
        self.workspace_bytes = need
        self.handle = _lib.lmloss_vocab_create(device, need)
        # Log-probabilities and 4-bit tables have a handle of their own, so that what the other operators
        # accept goes by their maxima alone; and a workspace from the first call on that needs one, so that
        # who never makes such a call pays nothing for it.  Of maxima past what those calls take, what they take.
        self.logprobs_workspace_bytes = self.scores_workspace_bytes = 0
        if max_rows > 0:
            V, D = min(max_vocab, (1 << 31) - (1 << 16)), min(max(max_dim, 1), 1 << 20)
            c = _lib.lmloss_logprobs_args(T=min(max_rows, (1 << 30) - 1), V=V, ld=V, M=_lib.LMLOSS_MAX_ALTERNATIVES,
                                          temperature=1.0)
            self.logprobs_workspace_bytes = _lib.lmloss_logprobs_workspace(c)
            d = _lib.lmloss_table4_logits_args(T=min(max_rows, (1 << 24) - 1))
            d.table.V, d.table.D, d.table.group = V, D, 32
            self.scores_workspace_bytes = max(self.logprobs_workspace_bytes, _lib.lmloss_table4_logits_workspace(d))
        self.scores_handle = _lib.lmloss_vocab_create(device, 0)
        self._reserved = 0

    def close(self):
        for name in ("handle", "scores_handle"):
            if getattr(self, name, None) is not None:
                _lib.lmloss_vocab_destroy(getattr(self, name))
                setattr(self, name, None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def device_error(self) -> int:
        """Read and clear an error of the calls so far, 0 if there is none (synchronises the device).  The embedding's and
        the beams' calls keep one, log-probabilities and 4-bit tables another: with both there, the second is read by
        the next call."""
        return _lib.lmloss_vocab_get_device_error(self.handle) or _lib.lmloss_vocab_get_device_error(self.scores_handle)

    def _refused(self, status, where, args, check, workspace, there=None):
        """The error for a refused call: where the arguments are in order, what the workspace lacks."""
        there = self.workspace_bytes if there is None else there
        if status == _lib.LMLOSS_ERR_INVALID_ARG and check(args) == _lib.LMLOSS_OK:
            need = workspace(args)
            if need > there:
                where += (f" ({need} bytes of workspace needed, {there} there: the handle's max_tokens, "
                          f"max_dim, max_rows or max_vocab is too small)")
        return LMLossError(status, where)

    def _with_workspace(self, status, call, args, raw, where, check, workspace, bytes_):
        """A log-probability's or a 4-bit table's call that was refused, again with the operator's workspace of
        `bytes_` if it is the first that needs it; else its error."""
        if self._reserved < bytes_ and status == _lib.LMLOSS_ERR_INVALID_ARG and check(args) == _lib.LMLOSS_OK:
            status = _lib.lmloss_vocab_reserve(self.scores_handle, bytes_)
            if status != _lib.LMLOSS_OK:
                raise LMLossError(status, f"{where} ({bytes_} bytes of workspace)")
            self._reserved = bytes_
            status = call(self.scores_handle, args, raw)
        if status != _lib.LMLOSS_OK:
            raise self._refused(status, where, args, check, workspace, self._reserved)

    # ------------------------------------------------------------- streams
    def _enter(self, stream, *tensors):
        """(stream, context for allocations) for a call on a stream of the caller's: where that is not
        the current one the outputs belong to it, and the caching allocator learns that it uses the
        inputs."""
        if stream == torch.cuda.current_stream(self.device):
            return stream.cuda_stream, contextlib.nullcontext()
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream, torch.cuda.stream(stream)

    # ----------------------------------------------------------- embedding
    def _ids(self, ids: torch.Tensor) -> int:
        dtype = _IDS.get(ids.dtype)
        if dtype is None:
            raise TypeError(f"ids: must be int64 or int32, got {ids.dtype}")
        if not ids.is_contiguous():
            raise ValueError("ids: must be contiguous")
        if ids.get_device() != self._index:
            raise ValueError(f"ids: on {ids.device}, the handle on {self.device}")
        return dtype

    def embedding_forward(self, weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                          out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """scale * weight[ids], [*ids.shape, D]: weight [V, D] and the result each
        bfloat16, float16 or float32 (the weight's type if not said).  An id of -100
        gives zeros; another outside [0, V) NaN and the error word.  ids are contiguous;
        out's rows may be strided, one stride between them all."""
        id_type = self._ids(ids)
        w_type, V, D, ld = _matrix(weight, "weight", self._index)
        if stream is None:
            raw, ctx = _raw_stream(self._index), None
        else:
            raw, ctx = self._enter(stream, weight, ids, out)
        T = ids.numel()
        shape = (T, D) if ids.dim() == 1 else (*ids.shape, D)
        if out is None:
            if out_dtype is None:
                out_dtype = weight.dtype
            r_type, ld_rows = _FLOATS.get(out_dtype), D
            if r_type is None:
                raise TypeError(f"out_dtype: must be bfloat16, float16 or float32, got {out_dtype}")
            if ctx is None:
                out = torch.empty(shape, dtype=out_dtype, device=self.device)
            else:
                with ctx:
                    out = torch.empty(shape, dtype=out_dtype, device=self.device)
        else:
            if out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
                raise ValueError(f"out: expected {shape}{'' if out_dtype is None else f' of {out_dtype}'}")
            r_type, _, _, ld_rows = _matrix(_flat(out, "out", T, D), "out", self._index)
        a = _lib.lmloss_embedding_args(ids.data_ptr(), T, V, D, weight.data_ptr(), ld, out.data_ptr(), ld_rows,
                                       id_type, w_type, r_type, scale, 0)
        st = self._forward(self.handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_embedding_forward")
        return out

    def embedding_backward(self, grad: torch.Tensor, ids: torch.Tensor, grad_weight: Optional[torch.Tensor] = None, *,
                           num_embeddings: Optional[int] = None, scale: float = 1.0, accumulate: bool = False,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The table's gradient [V, D] from the embeddings' gradient [*ids.shape, D].

        grad_weight is written as a whole, or with accumulate added to (a table tied
        to the LM head: the head's own gradient is there already); without it one of
        num_embeddings rows in grad's type is made.  Sums run in fp32 in an order
        that the ids alone fix.  ids are contiguous; grad's rows may be strided, one
        stride between them all."""
        id_type = self._ids(ids)
        if grad.shape[:-1] != ids.shape:
            raise ValueError(f"grad: expected [*{tuple(ids.shape)}, D], got {tuple(grad.shape)}")
        T = ids.numel()
        rows = _flat(grad, "grad", T, grad.shape[-1])
        r_type, _, D, ld_rows = _matrix(rows, "grad", self._index)
        if stream is None:
            raw, ctx = _raw_stream(self._index), contextlib.nullcontext()
        else:
            raw, ctx = self._enter(stream, grad, ids, grad_weight)
        if grad_weight is None:
            if num_embeddings is None or accumulate:
                raise ValueError("without grad_weight: num_embeddings and no accumulate")
            with ctx:
                grad_weight = torch.empty((num_embeddings, D), dtype=grad.dtype, device=self.device)
        t_type, V, cols, ld = _matrix(grad_weight, "grad_weight", self._index)
        if cols != D or num_embeddings not in (None, V):
            raise ValueError("grad_weight: must be [num_embeddings, D]")
        a = _lib.lmloss_embedding_args(ids.data_ptr(), T, V, D, grad_weight.data_ptr(), ld, rows.data_ptr(), ld_rows,
                                       id_type, t_type, r_type, scale, 1 if accumulate else 0)
        st = self._backward(self.handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise self._refused(st, "lmloss_embedding_backward", a, _lib.lmloss_embedding_check_args,
                                _lib.lmloss_embedding_workspace)
        return grad_weight

    # ---------------------------------------------------------------- beams
    def beam_step(self, logits: torch.Tensor, scores: torch.Tensor, *, num_candidates: Optional[int] = None,
                  finished: Optional[torch.Tensor] = None, eos_token: int = -1,
                  lengths: Optional[torch.Tensor] = None, length_penalty: float = 0.0,
                  token_mask: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> BeamStep:
        """The num_candidates (K if not said) best continuations of each sequence's beams.

        logits [B * K, V] (bfloat16, float16 or float32, unit column stride), scores
        [B, K] float32 the beams' summed log-probabilities (-inf: no beam).  finished
        [B, K] uint8: a finished beam goes on as its one candidate with eos_token.
        lengths [B, K] int32 with length_penalty: candidates are ranked by score /
        length^length_penalty.  token_mask [B * K or 1, ceil(V / 32)] int32: bit v % 32
        of word v / 32 allows token v.  Equal candidates: the lower beam, then the lower
        token."""
        if scores.dim() != 2:
            raise ValueError("scores: must be [B, K]")
        dev, index = self.device, self._index
        B, K = scores.size(0), scores.size(1)
        _check(scores, "scores", torch.float32, B, K, index)
        dtype, rows, V, ld = _matrix(logits, "logits", index)
        if rows != B * K:
            raise ValueError(f"logits: must be [B * K, V] with B * K = {B * K}")
        M = K if num_candidates is None else num_candidates
        if not 1 <= M <= _lib.LMLOSS_MAX_BEAMS or not 1 <= K <= _lib.LMLOSS_MAX_BEAMS:
            raise ValueError(f"beams and candidates: 1 to {_lib.LMLOSS_MAX_BEAMS}, got {K} and {M}")
        fin = length = mask = None
        stride = 0
        if finished is not None:
            _check(finished, "finished", torch.uint8, B, K, index)
            fin = finished.data_ptr()
        if lengths is not None:
            _check(lengths, "lengths", torch.int32, B, K, index)
            length = lengths.data_ptr()
        if token_mask is not None:
            words = (V + 31) // 32
            if token_mask.dim() != 2 or token_mask.size(0) not in (1, B * K):
                raise ValueError(f"token_mask: must be [{B * K} or 1, {words}]")
            _check(token_mask, "token_mask", torch.int32, token_mask.size(0), words, index)
            mask = token_mask.data_ptr()
            stride = 0 if token_mask.size(0) == 1 else words
        if stream is None:
            raw, r = _raw_stream(index), self._beam_out(B, K, M, dev, lengths is not None)
        else:
            raw, ctx = self._enter(stream, logits, scores, finished, lengths, token_mask)
            with ctx:
                r = self._beam_out(B, K, M, dev, lengths is not None)
        a = _lib.lmloss_beam_args(logits.data_ptr(), B, V, ld, K, M, dtype, length_penalty, eos_token,
                                  scores.data_ptr(), fin, length, mask, stride,
                                  r.scores.data_ptr(), r.parents.data_ptr(), r.tokens.data_ptr(), r.lse.data_ptr(),
                                  r.finished.data_ptr(), None if length is None else r.lengths.data_ptr())
        st = self._step(self.handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise self._refused(st, "lmloss_beam_step", a, _lib.lmloss_beam_check_args, _lib.lmloss_beam_workspace)
        return r

    @staticmethod
    def _beam_out(B, K, M, dev, lengths):
        empty, f32, i32, shape = torch.empty, torch.float32, torch.int32, (B, M)
        return BeamStep(empty(shape, dtype=f32, device=dev), empty(shape, dtype=i32, device=dev),
                        empty(shape, dtype=torch.int64, device=dev), empty((B, K), dtype=f32, device=dev),
                        empty(shape, dtype=torch.uint8, device=dev),
                        empty(shape, dtype=i32, device=dev) if lengths else None)

    def beam_reorder(self, states: Sequence[torch.Tensor], parents: torch.Tensor, *,
                     out: Union[None, str, Sequence[torch.Tensor]] = None, dim: int = 0,
                     stream: Optional[torch.cuda.Stream] = None) -> List[torch.Tensor]:
        """Row b * K_out + m of every state (along `dim`) becomes its row b * K + parents[b, m];
        parents is [B, K_out] int32, and the states have B * K rows.

        States may be of any type and strided (a view of the positions written so
        far).  out: tensors of the same type and shape but for their rows; "inplace",
        or the states themselves, to reorder in place (K_out = K); None for new ones.
        Otherwise out must not overlap the states."""
        if parents.dim() != 2:
            raise ValueError("parents: must be [B, K_out]")
        B, Ko = parents.size(0), parents.size(1)
        _check(parents, "parents", torch.int32, B, Ko, self._index)
        if not states:
            return []
        rows = states[0].size(dim)
        if rows % B if B else rows:
            raise ValueError(f"states: {rows} rows along dim {dim} for {B} sequences")
        K = rows // B if B else Ko
        if not 1 <= Ko <= _lib.LMLOSS_MAX_BEAMS or not 1 <= K <= _lib.LMLOSS_MAX_BEAMS:
            raise ValueError(f"beams: 1 to {_lib.LMLOSS_MAX_BEAMS} a sequence, got {K} and {Ko}")
        if stream is None:
            raw, ctx = _raw_stream(self._index), contextlib.nullcontext()
        else:
            named = out if isinstance(out, (list, tuple)) else ()
            raw, ctx = self._enter(stream, parents, *states, *named)
        if out is None:
            with ctx:
                out = [torch.empty([B * Ko if i == dim % t.dim() else n for i, n in enumerate(t.shape)], dtype=t.dtype,
                                   device=self.device) for t in states]
        elif isinstance(out, str):
            if out != "inplace":
                raise ValueError("out: tensors, 'inplace' or None")
            out = list(states)
        elif len(out) != len(states):
            raise ValueError("out: as many tensors as states")
        n = len(states)
        arr = (_lib.lmloss_beam_state * n)(*[self._describe(t, o, dim, rows, B * Ko) for t, o in zip(states, out)])
        st = self._reorder(self.handle, arr, n, parents.data_ptr(), B, K, Ko, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_beam_reorder")
        return list(out)

    def _describe(self, t: torch.Tensor, o: torch.Tensor, dim: int, rows: int, rows_out: int):
        """One state's lmloss_beam_state: the dimensions that both sides keep contiguous become the
        run, the rest outer counts."""
        if t.get_device() != self._index or o.get_device() != self._index:
            raise ValueError(f"states: on {t.device} and {o.device}, the handle on {self.device}")
        if t.dtype != o.dtype:
            raise TypeError(f"out: {o.dtype} for a state of {t.dtype}")
        shape, oshape, ts, os_ = t.shape, o.shape, t.stride(), o.stride()
        # (real views that are lazily negated are every second number of a conjugated one)
        if (t.is_complex() or ts[-1] != 1 or os_[-1] != 1) and \
                (t.is_conj() != o.is_conj() or t.is_neg() != o.is_neg()):
            raise ValueError("states: a lazily conjugated or negated view on one side; resolve it first")
        d = dim if dim >= 0 else dim + len(shape)
        if shape[d] != rows:
            raise ValueError(f"states: {shape[d]} and {rows} rows along dim {dim}")
        if len(oshape) != len(shape) or oshape[d] != rows_out:
            raise ValueError(f"out: {tuple(oshape)} for a state of {tuple(shape)} and {rows_out} rows")
        es = t.element_size()
        if len(shape) == 2 and d == 0 and ts[1] == 1 and os_[1] == 1 and oshape[1] == shape[1]:
            # a matrix: a row is a run
            return _lib.lmloss_beam_state(t.data_ptr(), o.data_ptr(), shape[1] * es, ts[0] * es, os_[0] * es, _ONES)
        dims = []
        for i, n in enumerate(shape):
            if i == d:
                continue
            if oshape[i] != n:
                raise ValueError(f"out: {tuple(oshape)} for a state of {tuple(shape)} and {rows_out} rows")
            if n != 1:
                if os_[i] == 0:
                    raise ValueError("out: must not overlap itself")
                dims.append((os_[i], ts[i], n))
        dims.sort()
        run, outer = 1, []
        for so, si, n in dims:
            if n == 0:
                run = 0
            elif so == run and si == run and not outer:
                run *= n
            elif outer and so == outer[-1][0] * outer[-1][2] and si == outer[-1][1] * outer[-1][2]:
                outer[-1] = (outer[-1][0], outer[-1][1], outer[-1][2] * n)
            else:
                outer.append((so, si, n))
        if len(outer) > 3:
            raise ValueError("states: more than three strided dimensions beside the rows")
        while len(outer) < 3:
            outer.append((0, 0, 1))
        (s0, r0, n0), (s1, r1, n1), (s2, r2, n2) = outer
        return _lib.lmloss_beam_state(t.data_ptr(), o.data_ptr(), run * es, ts[d] * es, os_[d] * es, (n0, n1, n2),
                                      (r0 * es, r1 * es, r2 * es), (s0 * es, s1 * es, s2 * es))

    # ----------------------------------------------------- log-probabilities
    def _given(self, tokens: torch.Tensor, T: int):
        """(type, tokens a row) of given tokens [T, n] or [T]."""
        dtype = _IDS.get(tokens.dtype)
        if dtype is None:
            raise TypeError(f"tokens: must be int64 or int32, got {tokens.dtype}")
        if tokens.dim() not in (1, 2) or tokens.size(0) != T:
            raise ValueError(f"tokens: must be [{T}] or [{T}, n], got {tuple(tokens.shape)}")
        if not tokens.is_contiguous():
            raise ValueError("tokens: must be contiguous")
        if tokens.get_device() != self._index:
            raise ValueError(f"tokens: on {tokens.device}, the handle on {self.device}")
        return dtype, 1 if tokens.dim() == 1 else tokens.size(1)

    def _mask(self, token_mask: torch.Tensor, rows: int, V: int):
        """(pointer, words between rows) of a token mask [rows or 1, ceil(V / 32)]."""
        words = (V + 31) // 32
        if token_mask.dim() != 2 or token_mask.size(0) not in (1, rows):
            raise ValueError(f"token_mask: must be [{rows} or 1, {words}]")
        _check(token_mask, "token_mask", torch.int32, token_mask.size(0), words, self._index)
        return token_mask.data_ptr(), 0 if token_mask.size(0) == 1 else words

    def token_logprobs(self, logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, num_top: int = 0,
                       temperature: float = 1.0, token_mask: Optional[torch.Tensor] = None, entropy: bool = True,
                       for_gradient: bool = False, stream: Optional[torch.cuda.Stream] = None) -> TokenLogprobs:
        """Log-probabilities of the given tokens [T, n] or [T] (int64 or int32, contiguous) under
        softmax(logits / temperature), logits [T, V] (bfloat16, float16 or float32, unit column
        stride), with the rows' logsumexp and entropy, for_gradient its two parts that the gradient takes (row_max and
        log_sum), and the num_top (0 to 64) largest
        log-probabilities with their tokens, equal ones by token.

        token_mask [T or 1, ceil(V / 32)] int32: bit v % 32 of word v / 32 allows token v; the softmax is
        over the allowed ones.  A token of -100 gives 0, another outside [0, V) NaN and the error word, one
        that is not allowed -inf.  Fewer than num_top candidates: -inf and -100."""
        index = self._index
        dtype, T, V, ld = _matrix(logits, "logits", index)
        if not 0 <= num_top <= _lib.LMLOSS_MAX_ALTERNATIVES:
            raise ValueError(f"num_top: 0 to {_lib.LMLOSS_MAX_ALTERNATIVES}, got {num_top}")
        ids, n = (_lib.LMLOSS_INT64, 0) if tokens is None else self._given(tokens, T)
        mask, mask_stride = (None, 0) if token_mask is None else self._mask(token_mask, T, V)
        if stream is None:
            raw, r = _raw_stream(index), self._logprobs_out(tokens, T, num_top, entropy, for_gradient)
        else:
            raw, ctx = self._enter(stream, logits, tokens, token_mask)
            with ctx:
                r = self._logprobs_out(tokens, T, num_top, entropy, for_gradient)
        a = _lib.lmloss_logprobs_args(logits.data_ptr(), T, V, ld, dtype, ids, tokens.data_ptr() if n else None, n,
                                      temperature, num_top, mask, mask_stride, r.logp.data_ptr() if n else None,
                                      r.lse.data_ptr(), r.entropy.data_ptr() if entropy else None,
                                      r.top_logp.data_ptr() if num_top else None,
                                      r.top_tokens.data_ptr() if num_top else None)
        if for_gradient:
            a.row_max_out, a.log_sum_out = r.row_max.data_ptr(), r.log_sum.data_ptr()
        st = self._logprobs(self.scores_handle, a, raw)
        if st != _lib.LMLOSS_OK:
            self._with_workspace(st, self._logprobs, a, raw, "lmloss_logprobs_forward", _lib.lmloss_logprobs_check_args,
                                 _lib.lmloss_logprobs_workspace, self.logprobs_workspace_bytes)
        return r

    def _logprobs_out(self, tokens, T, M, entropy, for_gradient):
        # (a tensor like another costs the host half of what one of a shape does)
        empty, like, dev, f32 = torch.empty, torch.empty_like, self.device, torch.float32
        lse = empty((T,), dtype=f32, device=dev)
        top = empty((T, M), dtype=f32, device=dev) if M else None
        r = TokenLogprobs(None if tokens is None else like(tokens, dtype=f32), lse, like(lse) if entropy else None,
                          top, like(top, dtype=torch.int64) if M else None)
        if for_gradient:
            r.row_max, r.log_sum = like(lse), like(lse)
        return r

    def token_logprobs_backward(self, logits: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                tokens: Optional[torch.Tensor] = None, grad_logp: Optional[torch.Tensor] = None, *,
                                row_max: Optional[torch.Tensor] = None, log_sum: Optional[torch.Tensor] = None,
                                entropy: Optional[torch.Tensor] = None,
                                grad_entropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                                token_mask: Optional[torch.Tensor] = None,
                                grad: Union[None, str, torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The logits' gradient [T, V], in their type, from grad_logp (of the tokens' shape, float32, at most
        1024 tokens a row) and grad_entropy [T]: with the forward call's logits, row_max and log_sum (or lse), entropy,
        temperature and mask.  lse is not looked at beside row_max and log_sum; alone it leaves the probabilities off by
        a factor of e to 2^-24 of itself (1e-3 at an lse of 15000, as low temperatures have).  Gradients of alternatives: give their tokens.  grad: a tensor to write, "inplace" (over the logits), or
        None for a new one.  Columns that are not allowed, and rows in which nothing is, get 0."""
        index = self._index
        dtype, T, V, ld = _matrix(logits, "logits", index)
        if (tokens is None) != (grad_logp is None):
            raise ValueError("tokens and grad_logp: both or neither")
        ids, n = (_lib.LMLOSS_INT64, 0) if tokens is None else self._given(tokens, T)
        if n > _lib.LMLOSS_MAX_GIVEN:
            raise ValueError(f"tokens: at most {_lib.LMLOSS_MAX_GIVEN} a row, got {n}")
        if (row_max is None) != (log_sum is None):
            raise ValueError("row_max and log_sum: both or neither")
        if lse is None and log_sum is None:
            raise ValueError("the forward call's row_max and log_sum, or its lse, are needed")
        vectors = [("lse", lse, (T,))] if log_sum is None else [("row_max", row_max, (T,)), ("log_sum", log_sum, (T,))]
        if tokens is not None:
            vectors.append(("grad_logp", grad_logp, tuple(tokens.shape)))
        if grad_entropy is not None:
            if entropy is None:
                raise ValueError("grad_entropy: needs the forward call's entropy")
            vectors += [("entropy", entropy, (T,)), ("grad_entropy", grad_entropy, (T,))]
        for name, t, shape in vectors:
            if t.dtype != torch.float32:
                raise TypeError(f"{name}: expected {torch.float32}, got {t.dtype}")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous {shape}, got {tuple(t.shape)}")
            if t.get_device() != index:
                raise ValueError(f"{name}: on {t.device}, the handle on {self.device}")
        mask, mask_stride = (None, 0) if token_mask is None else self._mask(token_mask, T, V)
        if stream is None:
            raw, ctx = _raw_stream(index), contextlib.nullcontext()
        else:
            raw, ctx = self._enter(stream, logits, lse, row_max, log_sum, tokens, grad_logp, entropy, grad_entropy, token_mask,
                                   grad if isinstance(grad, torch.Tensor) else None)
        if grad is None:
            with ctx:
                grad = torch.empty((T, V), dtype=logits.dtype, device=self.device)
        elif isinstance(grad, str):
            if grad != "inplace":
                raise ValueError("grad: a tensor, 'inplace' or None")
            grad = logits
        g_type, rows, cols, ld_grad = _matrix(grad, "grad", index)
        if g_type != dtype or rows != T or cols != V:
            raise ValueError(f"grad: expected [{T}, {V}] of {logits.dtype}")
        a = _lib.lmloss_logprobs_grad_args(logits.data_ptr(), T, V, ld, dtype, ids, tokens.data_ptr() if n else None, n,
                                           temperature, mask, mask_stride, None if lse is None else lse.data_ptr(),
                                           grad_logp.data_ptr() if n else None,
                                           None if grad_entropy is None else entropy.data_ptr(),
                                           None if grad_entropy is None else grad_entropy.data_ptr(),
                                           grad.data_ptr(), ld_grad, None if log_sum is None else row_max.data_ptr(),
                                           None if log_sum is None else log_sum.data_ptr())
        st = self._logprobs_grad(self.scores_handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_logprobs_backward")
        return grad

    # ------------------------------------------------------- tables in 4 bits
    def new_table4(self, num_embeddings: int, columns: int, *, group_size: int = 128, zeros: bool = False,
                   scale_dtype: torch.dtype = torch.float16) -> Table4:
        """An unwritten 4-bit table of the layout that the calls below take."""
        if num_embeddings < 1 or columns < 1 or group_size not in (32, 64, 128):
            raise ValueError("a 4-bit table has at least one row and column, and groups of 32, 64 or 128")
        if scale_dtype not in _FLOATS:
            raise TypeError(f"scale_dtype: must be bfloat16, float16 or float32, got {scale_dtype}")
        G, wide, half = (columns + group_size - 1) // group_size, (num_embeddings + 15) // 16 * 16, (columns + 1) // 2
        ld, dev = (half + 15) // 16 * 16, self.device
        values = torch.empty((num_embeddings, ld), dtype=torch.uint8, device=dev).as_strided((num_embeddings, half), (ld, 1))
        scales = torch.empty((G, wide), dtype=scale_dtype, device=dev).as_strided((G, num_embeddings), (wide, 1))
        z = torch.empty((G, wide), dtype=torch.uint8, device=dev).as_strided((G, num_embeddings), (wide, 1)) if zeros else None
        return Table4(values, scales, z, columns, group_size)

    def _table4(self, t: Table4):
        """A table's lmloss_table4."""
        values, scales, zeros, D, g, index = t.values, t.scales, t.zeros, t.columns, t.group_size, self._index
        shape, s_shape, v_stride, s_stride, s_type = values.shape, scales.shape, values.stride(), scales.stride(), scales.dtype
        # what is in order, at once
        if len(shape) == 2 and g in (32, 64, 128) and D > 0 and values.dtype is torch.uint8 and s_type in _FLOATS:
            V, G = shape[0], (D + g - 1) // g
            bytes_, ld, v_at, s_at = v_stride[0], s_stride[0], values.data_ptr(), scales.data_ptr()
            if V > 1 and G > 1 and shape[1] == (D + 1) // 2 and s_shape == (G, V) and v_stride[1] == s_stride[1] == 1 and \
                    bytes_ >= shape[1] and ld >= V and (bytes_ | ld * s_type.itemsize | v_at | s_at) % 16 == 0 and \
                    values.get_device() == scales.get_device() == index:
                if zeros is None:
                    return _lib.lmloss_table4(v_at, bytes_, s_at, ld, None, 0, V, D, g, _FLOATS[s_type])
                z_stride, z_at = zeros.stride(), zeros.data_ptr()
                if zeros.dtype is torch.uint8 and zeros.shape == s_shape and z_stride[1] == 1 and z_stride[0] >= V and \
                        (z_stride[0] | z_at) % 16 == 0 and zeros.get_device() == index:
                    return _lib.lmloss_table4(v_at, bytes_, s_at, ld, z_at, z_stride[0], V, D, g, _FLOATS[s_type])
        return self._table4_looked_at(t)

    def _table4_looked_at(self, t: Table4):
        """The same for a table of one row or group, or the error of one that is not in order."""
        values, scales, zeros, index = t.values, t.scales, t.zeros, self._index
        V, D, g = values.size(0), t.columns, t.group_size
        if g not in (32, 64, 128):
            raise ValueError(f"table: groups of 32, 64 or 128 columns, got {g}")
        dtype = _FLOATS.get(scales.dtype)
        if values.dtype != torch.uint8 or dtype is None or (zeros is not None and zeros.dtype != torch.uint8):
            raise TypeError("table: values and zeros are uint8, scales bfloat16, float16 or float32")
        G = (D + g - 1) // g
        if values.dim() != 2 or V < 1 or D < 1 or values.size(1) != (D + 1) // 2:
            raise ValueError(f"table: values must be [V, {(D + 1) // 2}] for {D} columns, got {tuple(values.shape)}")
        lds = []
        for name, x, rows, es in (("values", values, V, 1), ("scales", scales, G, scales.element_size()),
                                  ("zeros", zeros, G, 1)):
            if x is None:
                lds.append(0)
                continue
            if x.get_device() != index:
                raise ValueError(f"table: {name} on {x.device}, the handle on {self.device}")
            if x.dim() != 2 or x.size(0) != rows or (name != "values" and x.size(1) != V):
                raise ValueError(f"table: {name} must be {[rows, 'columns / 2' if name == 'values' else V]}, "
                                 f"got {tuple(x.shape)}")
            ld, unit = x.stride()
            cols = x.size(1)
            if rows == 1:
                ld = (cols * es + 15) // 16 * 16 // es
            if (cols > 1 and unit != 1) or ld < cols or ld * es % 16 or x.data_ptr() % 16:
                raise ValueError(f"table: {name} must have unit column stride and rows on 16-byte boundaries")
            lds.append(ld)
        return _lib.lmloss_table4(values.data_ptr(), lds[0], scales.data_ptr(), lds[1],
                                  None if zeros is None else zeros.data_ptr(), lds[2], V, D, g, dtype)

    def quantize_table(self, weight: torch.Tensor, out: Optional[Table4] = None, *, group_size: int = 128,
                       zeros: bool = False, scale_dtype: torch.dtype = torch.float16,
                       stream: Optional[torch.cuda.Stream] = None) -> Table4:
        """The 4-bit table nearest to weight [V, D] (bfloat16, float16 or float32), group by group:
        without zeros s = max |w| / 7 and q = w / s + 8; with zeros s = (max - min) / 15 over the weights and 0,
        z = -min / s and q = w / s + z.  out: a table to write (its own groups, zeros and scales).  A
        group whose weights or scale are not finite gets a scale of NaN and the error word."""
        w_type, V, D, ld = _matrix(weight, "weight", self._index)
        if stream is None:
            raw, ctx = _raw_stream(self._index), contextlib.nullcontext()
        else:
            raw, ctx = self._enter(stream, weight, *(() if out is None else (out.values, out.scales, out.zeros)))
        if out is None:
            with ctx:
                out = self.new_table4(V, D, group_size=group_size, zeros=zeros, scale_dtype=scale_dtype)
        t = self._table4(out)
        if t.V != V or t.D != D:
            raise ValueError(f"out: a table of [{t.V}, {t.D}] for weights of [{V}, {D}]")
        a = _lib.lmloss_table4_quantize_args(t, weight.data_ptr(), ld, w_type)
        st = self._quantize(self.scores_handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_table4_quantize")
        return out

    def table4_lookup(self, table: Table4, ids: torch.Tensor, *, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """scale * table[ids], [*ids.shape, columns] in out_dtype (the scales' type if not said): ids and
        out as for `embedding_forward`."""
        id_type = self._ids(ids)
        t = self._table4(table)
        if stream is None:
            raw, ctx = _raw_stream(self._index), contextlib.nullcontext()
        else:
            raw, ctx = self._enter(stream, table.values, table.scales, table.zeros, ids, out)
        T, D = ids.numel(), table.columns
        out, r_type, ld_rows = self._result(out, out_dtype or table.scales.dtype, out_dtype, (*ids.shape, D), T, D, ctx)
        a = _lib.lmloss_table4_lookup_args(t, ids.data_ptr(), T, out.data_ptr(), ld_rows, id_type, r_type, scale)
        st = self._lookup4(self.scores_handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_table4_lookup")
        return out

    def _result(self, out, dtype, asked, shape, T, D, ctx):
        """(out, its type, its row stride): one of `shape` and `dtype` made, or the caller's looked at."""
        if out is None:
            r_type = _FLOATS.get(dtype)
            if r_type is None:
                raise TypeError(f"out_dtype: must be bfloat16, float16 or float32, got {dtype}")
            with ctx:
                return torch.empty(shape, dtype=dtype, device=self.device), r_type, D
        if out.shape != shape or (asked is not None and out.dtype != asked):
            raise ValueError(f"out: expected {shape}{'' if asked is None else f' of {asked}'}")
        r_type, _, _, ld = _matrix(_flat(out, "out", T, D), "out", self._index)
        return out, r_type, ld

    def table4_logits(self, table: Table4, hidden: torch.Tensor, *, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """scale * hidden @ table^T: logits [..., V] of hidden rows [..., columns] (bfloat16, float16 or float32),
        in out_dtype (hidden's if not said).  Rows of hidden and out may be strided, one stride between them all."""
        t = self._table4(table)
        D, V = table.columns, t.V
        if hidden.dim() < 1 or hidden.size(-1) != D:
            raise ValueError(f"hidden: must be [..., {D}], got {tuple(hidden.shape)}")
        T = hidden.numel() // D
        rows = _flat(hidden, "hidden", T, D)
        x_type, _, _, ld = _matrix(rows, "hidden", self._index)
        if stream is None:
            raw, ctx = _raw_stream(self._index), contextlib.nullcontext()
        else:
            raw, ctx = self._enter(stream, table.values, table.scales, table.zeros, hidden, out)
        out, o_type, ld_out = self._result(out, out_dtype or hidden.dtype, out_dtype, (*hidden.shape[:-1], V), T, V, ctx)
        a = _lib.lmloss_table4_logits_args(t, rows.data_ptr(), T, ld, out.data_ptr(), ld_out, x_type, o_type, scale)
        st = self._logits4(self.scores_handle, a, raw)
        if st != _lib.LMLOSS_OK:
            self._with_workspace(st, self._logits4, a, raw, "lmloss_table4_logits", _lib.lmloss_table4_check_logits_args,
                                 _lib.lmloss_table4_logits_workspace, self.scores_workspace_bytes)
        return out
