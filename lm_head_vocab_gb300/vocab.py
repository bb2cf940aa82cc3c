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
_IDS = {torch.int64: _lib.LMLOSS_INT64, torch.int32: _lib.LMLOSS_INT32}


def _check(t: torch.Tensor, name: str, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the handle on {device}")


def _matrix(t: torch.Tensor, name: str, device):
    """(row stride) of a 2-d float tensor with unit column stride and rows that do not overlap."""
    if t.dtype not in _FLOATS:
        raise TypeError(f"{name}: must be bfloat16, float16 or float32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the handle on {device}")
    rows, cols = t.shape
    if cols < 1 or (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name}: must have at least one column, unit column stride and a row stride of at least "
                         f"its columns")
    return t.stride(0) if rows > 1 else cols


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

    # ------------------------------------------------------------- streams
    def _stream(self, stream, *tensors):
        """(stream, context for allocations): on a stream that is not the current one the outputs
        belong to it, and the caching allocator learns that it uses the inputs."""
        cur = torch.cuda.current_stream(self.device)
        if stream is None or stream == cur:
            return cur.cuda_stream, contextlib.nullcontext()
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream, torch.cuda.stream(stream)

    # ----------------------------------------------------------- embedding
    def _ids(self, ids: torch.Tensor):
        if ids.dtype not in _IDS:
            raise TypeError(f"ids: must be int64 or int32, got {ids.dtype}")
        if not ids.is_contiguous():
            raise ValueError("ids: must be contiguous")
        if ids.device != self.device:
            raise ValueError(f"ids: on {ids.device}, the handle on {self.device}")

    def embedding_forward(self, weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                          out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """scale * weight[ids], [*ids.shape, D]: weight [V, D] and the result each
        bfloat16, float16 or float32 (the weight's type if not said).  An id of -100
        gives zeros; another outside [0, V) NaN and the error word."""
        self._ids(ids)
        if weight.dim() != 2:
            raise ValueError("weight: must be [V, D]")
        ld = _matrix(weight, "weight", self.device)
        V, D = weight.shape
        raw, ctx = self._stream(stream, weight, ids, out)
        if out is None:
            with ctx:
                out = torch.empty(*ids.shape, D, dtype=out_dtype or weight.dtype, device=self.device)
        elif out.shape != (*ids.shape, D) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out: expected {(*ids.shape, D)}{'' if out_dtype is None else f' of {out_dtype}'}")
        T = ids.numel()
        rows = out if out.dim() == 2 else out.view(T, D)
        a = _lib.lmloss_embedding_args(ids.data_ptr(), T, V, D, weight.data_ptr(), ld, rows.data_ptr(),
                                       _matrix(rows, "out", self.device), _IDS[ids.dtype], _FLOATS[weight.dtype],
                                       _FLOATS[rows.dtype], scale, 0)
        st = _lib.lmloss_embedding_forward(self.handle, a, raw)
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
        that the ids alone fix."""
        self._ids(ids)
        if grad.shape[:-1] != ids.shape or grad.dim() != ids.dim() + 1:
            raise ValueError(f"grad: expected [*{tuple(ids.shape)}, D], got {tuple(grad.shape)}")
        T, D = ids.numel(), grad.shape[-1]
        rows = grad if grad.dim() == 2 else grad.view(T, D)
        ld = _matrix(rows, "grad", self.device)
        raw, ctx = self._stream(stream, grad, ids, grad_weight)
        if grad_weight is None:
            if num_embeddings is None or accumulate:
                raise ValueError("without grad_weight: num_embeddings and no accumulate")
            with ctx:
                grad_weight = torch.empty(num_embeddings, D, dtype=grad.dtype, device=self.device)
        elif grad_weight.dim() != 2 or grad_weight.shape[1] != D or num_embeddings not in (None, grad_weight.shape[0]):
            raise ValueError("grad_weight: must be [num_embeddings, D]")
        a = _lib.lmloss_embedding_args(ids.data_ptr(), T, grad_weight.shape[0], D, grad_weight.data_ptr(),
                                       _matrix(grad_weight, "grad_weight", self.device), rows.data_ptr(), ld,
                                       _IDS[ids.dtype], _FLOATS[grad_weight.dtype], _FLOATS[rows.dtype], scale,
                                       1 if accumulate else 0)
        st = _lib.lmloss_embedding_backward(self.handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_embedding_backward")
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
        dev = self.device
        B, K = scores.shape
        _check(scores, "scores", torch.float32, (B, K), dev)
        if logits.dim() != 2 or logits.shape[0] != B * K:
            raise ValueError(f"logits: must be [B * K, V] with B * K = {B * K}")
        ld = _matrix(logits, "logits", dev)
        V = logits.shape[1]
        M = K if num_candidates is None else num_candidates
        if not 1 <= M <= _lib.LMLOSS_MAX_BEAMS or not 1 <= K <= _lib.LMLOSS_MAX_BEAMS:
            raise ValueError(f"beams and candidates: 1 to {_lib.LMLOSS_MAX_BEAMS}, got {K} and {M}")
        if finished is not None:
            _check(finished, "finished", torch.uint8, (B, K), dev)
        if lengths is not None:
            _check(lengths, "lengths", torch.int32, (B, K), dev)
        stride = 0
        if token_mask is not None:
            words = (V + 31) // 32
            if token_mask.dim() != 2 or token_mask.shape[0] not in (1, B * K):
                raise ValueError(f"token_mask: must be [{B * K} or 1, {words}]")
            _check(token_mask, "token_mask", torch.int32, (token_mask.shape[0], words), dev)
            stride = 0 if token_mask.shape[0] == 1 else words
        raw, ctx = self._stream(stream, logits, scores, finished, lengths, token_mask)
        with ctx:
            r = BeamStep(torch.empty((B, M), dtype=torch.float32, device=dev),
                         torch.empty((B, M), dtype=torch.int32, device=dev),
                         torch.empty((B, M), dtype=torch.int64, device=dev),
                         torch.empty((B, K), dtype=torch.float32, device=dev),
                         torch.empty((B, M), dtype=torch.uint8, device=dev),
                         None if lengths is None else torch.empty((B, M), dtype=torch.int32, device=dev))
        a = _lib.lmloss_beam_args(logits.data_ptr(), B, V, ld, K, M, _FLOATS[logits.dtype], length_penalty, eos_token,
                                  scores.data_ptr(), None if finished is None else finished.data_ptr(),
                                  None if lengths is None else lengths.data_ptr(),
                                  None if token_mask is None else token_mask.data_ptr(), stride,
                                  r.scores.data_ptr(), r.parents.data_ptr(), r.tokens.data_ptr(), r.lse.data_ptr(),
                                  r.finished.data_ptr(), None if lengths is None else r.lengths.data_ptr())
        st = _lib.lmloss_beam_step(self.handle, a, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_beam_step")
        return r

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
        B, Ko = parents.shape
        _check(parents, "parents", torch.int32, (B, Ko), self.device)
        if not states:
            return []
        rows = states[0].shape[dim]
        if B == 0 or rows % B:
            raise ValueError(f"states: {rows} rows along dim {dim} for {B} sequences")
        K = rows // B
        if not 1 <= Ko <= _lib.LMLOSS_MAX_BEAMS or not 1 <= K <= _lib.LMLOSS_MAX_BEAMS:
            raise ValueError(f"beams: 1 to {_lib.LMLOSS_MAX_BEAMS} a sequence, got {K} and {Ko}")
        named = out if isinstance(out, (list, tuple)) else ()
        raw, ctx = self._stream(stream, parents, *states, *named)
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
        arr = (_lib.lmloss_beam_state * len(states))()
        for s, t, o in zip(arr, states, out):
            self._describe(s, t, o, dim, rows, B * Ko)
        st = _lib.lmloss_beam_reorder(self.handle, arr, parents.data_ptr(), B, K, Ko, raw)
        if st != _lib.LMLOSS_OK:
            raise LMLossError(st, "lmloss_beam_reorder")
        return list(out)

    def _describe(self, s, t: torch.Tensor, o: torch.Tensor, dim: int, rows: int, rows_out: int):
        """Fill one lmloss_beam_state: the dimensions that both sides keep contiguous become the run,
        the rest outer counts."""
        if t.device != self.device or o.device != self.device:
            raise ValueError(f"states: on {t.device} and {o.device}, the handle on {self.device}")
        if t.dtype != o.dtype:
            raise TypeError(f"out: {o.dtype} for a state of {t.dtype}")
        d = dim % t.dim()
        want = list(t.shape)
        if want[d] != rows:
            raise ValueError(f"states: {want[d]} and {rows} rows along dim {dim}")
        want[d] = rows_out
        if list(o.shape) != want:
            raise ValueError(f"out: expected shape {want}, got {list(o.shape)}")
        es = t.element_size()
        ts, os_ = t.stride(), o.stride()
        dims = []
        for i, n in enumerate(t.shape):
            if i == d:
                continue
            if n > 1 and os_[i] == 0:
                raise ValueError("out: must not overlap itself")
            if n != 1:
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
        s.src = t.data_ptr()
        s.dst = o.data_ptr()
        s.inner = run * es
        s.src_row_stride = ts[d] * es
        s.dst_row_stride = os_[d] * es
        for k in range(3):
            so, si, n = outer[k] if k < len(outer) else (0, 0, 1)
            s.outer[k] = n
            s.src_outer_stride[k] = si * es
            s.dst_outer_stride[k] = so * es
