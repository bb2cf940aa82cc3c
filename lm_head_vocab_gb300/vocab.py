"""PyTorch-facing wrapper of the vocabulary operators of the lmloss C ABI:
embedding lookup and gradient, beam search's step, reordering of beam states.

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


class VocabOps:
    """One handle of the vocabulary operators, with workspace for embedding
    gradients of up to max_tokens positions and max_dim columns and for beam
    steps of up to max_rows rows of logits, at vocabularies of up to max_vocab.

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

    def close(self):
        if getattr(self, "handle", None) is not None:
            _lib.lmloss_vocab_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def device_error(self) -> int:
        """Read and clear the handle's error word (synchronises the device)."""
        return _lib.lmloss_vocab_get_device_error(self.handle)

    def _refused(self, status, where, args, check, workspace):
        """The error for a refused call: where the arguments are in order, what the workspace lacks."""
        if status == _lib.LMLOSS_ERR_INVALID_ARG and check(args) == _lib.LMLOSS_OK:
            need = workspace(args)
            if need > self.workspace_bytes:
                where += (f" ({need} bytes of workspace needed, {self.workspace_bytes} there: the handle's max_tokens, "
                          f"max_dim, max_rows or max_vocab is too small)")
        return LMLossError(status, where)

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
