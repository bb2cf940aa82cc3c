"""ctypes binding of the lmloss C ABI (include/lmloss.h): same names, argument
marshalling only.  The CUDA library must have been built (``build()``); nothing
here computes any part of the loss, and there is no CPU fallback."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_CSRC = os.path.join(_PKG, "csrc")
_BUILD = os.path.join(_PKG, "_build")
LIB_PATH = os.path.join(_BUILD, "liblmloss.so")
HEADER = os.path.join(_ROOT, "include", "lmloss.h")
# (source, extra flags, object): the host code with the small kernels, and the
# staged-row kernel's eight (dtype, teacher, temperature, entropy) instantiation
# sets, one object each so that they compile in parallel
UNITS = [("lmloss.cu", [], "lmloss.o")] + [
    ("fused_inst.cu", [f"-DLMLOSS_FUSED_VARIANT={k}"], f"fused_{k}.o") for k in range(8)] + [
    # the vocabulary operators
    (f"{name}.cu", [], f"{name}.o") for name in ("vocab_handle", "embedding", "beam_step", "beam_reorder", "logprobs", "table4",
                                               "table4_logits", "table4_rows")]
DEPENDS = ["lmloss.cu", "fused_inst.cu", "fused_entry.cuh", "kernels.cuh", "aux_kernels.cuh", "ptx.cuh",
           "vocab_common.cuh", "vocab_handle.cu", "embedding.cu", "beam_math.cuh", "beam_plan.cuh", "row_stream.cuh", "beam_step.cu", "beam_reorder.cu",
           "logprobs.cu", "table4.cuh", "tcgen05.cuh", "table4.cu", "table4_logits.cuh", "table4_logits.cu", "table4_rows.cu"]

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC"]

LMLOSS_OK = 0
LMLOSS_ERR_INVALID_ARG = 1
LMLOSS_ERR_UNSUPPORTED = 2
LMLOSS_ERR_CUDA = 3
LMLOSS_ERR_BAD_TARGET = 4
LMLOSS_ERR_BAD_SEGMENT = 5
LMLOSS_ERR_RANGE = 6
LMLOSS_ERR_TIMEOUT = 7
LMLOSS_ERR_BAD_PARENT = 8
LMLOSS_BF16 = 0
LMLOSS_FP32 = 1
LMLOSS_FP16 = 2
LMLOSS_INT64 = 0
LMLOSS_INT32 = 1
LMLOSS_MAX_BEAMS = 64
LMLOSS_MAX_ALTERNATIVES = 64
LMLOSS_MAX_GIVEN = 1024
LMLOSS_REDUCE_SUM = 0
LMLOSS_REDUCE_TOKEN_MEAN = 1
LMLOSS_IGNORE_INDEX = -100


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build(force: bool = False) -> str:
    """Compile the CUDA library for sm_103a into the package's _build folder:
    every translation unit at once, then one link."""
    os.makedirs(_BUILD, exist_ok=True)
    newest = max(os.path.getmtime(os.path.join(_CSRC, f)) for f in DEPENDS)
    newest = max(newest, os.path.getmtime(HEADER))
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest:
        return LIB_PATH
    work = os.path.join(_BUILD, f"tmp{os.getpid()}")
    os.makedirs(work, exist_ok=True)
    objs, procs = [], []
    try:
        for src, extra, obj in UNITS:
            o = os.path.join(work, obj)
            objs.append(o)
            cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-c", "-o", o, os.path.join(_CSRC, src)]
            procs.append((cmd, subprocess.Popen(cmd)))
        failed = [cmd for cmd, pr in procs if pr.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        tmp = os.path.join(work, "liblmloss.so")
        subprocess.run([_nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs],
                       check=True)
        os.replace(tmp, LIB_PATH)
    finally:
        for _, pr in procs:
            if pr.poll() is None:
                pr.kill()
                pr.wait()
        shutil.rmtree(work, ignore_errors=True)
    return LIB_PATH


class lmloss_args(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reduction", ctypes.c_int32),
        ("targets", ctypes.c_void_p),
        ("loss_mask", ctypes.c_void_p),
        ("ce_weight", ctypes.c_float),
        ("z_alpha", ctypes.c_float),
        ("teacher_logits", ctypes.c_void_p),
        ("kl_weight", ctypes.c_float),
        ("temperature", ctypes.c_float),
        ("segment_ids", ctypes.c_void_p),
        ("num_segments", ctypes.c_int32),
        ("advantages", ctypes.c_void_p),
        ("old_logprobs", ctypes.c_void_p),
        ("clip_eps_low", ctypes.c_float),
        ("clip_eps_high", ctypes.c_float),
        ("denominator", ctypes.c_double),
        ("grad_out", ctypes.c_void_p),
        ("loss_out", ctypes.c_void_p),
        ("logp_out", ctypes.c_void_p),
        ("lse_out", ctypes.c_void_p),
        ("kl_out", ctypes.c_void_p),
        ("count_out", ctypes.c_void_p),
        ("seg_count_out", ctypes.c_void_p),
        ("seg_ratio_out", ctypes.c_void_p),
        ("seg_flag_out", ctypes.c_void_p),
        ("seg_loss_out", ctypes.c_void_p),
        ("token_advantages", ctypes.c_void_p),
        ("entropy_out", ctypes.c_void_p),
    ]


class lmloss_call_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("launches", "path", "cluster", "threads", "nbuf", "grid", "smem_bytes", "reserved")]


class lmloss_embedding_args(ctypes.Structure):
    _fields_ = [
        ("ids", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("D", ctypes.c_int64),
        ("table", ctypes.c_void_p),
        ("ld_table", ctypes.c_int64),
        ("rows", ctypes.c_void_p),
        ("ld_rows", ctypes.c_int64),
        ("ids_dtype", ctypes.c_int32),
        ("table_dtype", ctypes.c_int32),
        ("rows_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("accumulate", ctypes.c_int32),
    ]


class lmloss_beam_args(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("B", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("K", ctypes.c_int32),
        ("M", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("length_penalty", ctypes.c_double),
        ("eos_token", ctypes.c_int64),
        ("scores", ctypes.c_void_p),
        ("finished", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p),
        ("token_mask", ctypes.c_void_p),
        ("mask_stride", ctypes.c_int64),
        ("scores_out", ctypes.c_void_p),
        ("parents_out", ctypes.c_void_p),
        ("tokens_out", ctypes.c_void_p),
        ("lse_out", ctypes.c_void_p),
        ("finished_out", ctypes.c_void_p),
        ("lengths_out", ctypes.c_void_p),
    ]


class lmloss_beam_state(ctypes.Structure):
    _fields_ = [
        ("src", ctypes.c_void_p),
        ("dst", ctypes.c_void_p),
        ("inner", ctypes.c_int64),
        ("src_row_stride", ctypes.c_int64),
        ("dst_row_stride", ctypes.c_int64),
        ("outer", ctypes.c_int64 * 3),
        ("src_outer_stride", ctypes.c_int64 * 3),
        ("dst_outer_stride", ctypes.c_int64 * 3),
    ]


class lmloss_logprobs_args(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("ids_dtype", ctypes.c_int32),
        ("tokens", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("temperature", ctypes.c_float),
        ("M", ctypes.c_int32),
        ("token_mask", ctypes.c_void_p),
        ("mask_stride", ctypes.c_int64),
        ("logp_out", ctypes.c_void_p),
        ("lse_out", ctypes.c_void_p),
        ("entropy_out", ctypes.c_void_p),
        ("top_logp_out", ctypes.c_void_p),
        ("top_tokens_out", ctypes.c_void_p),
        ("row_max_out", ctypes.c_void_p),
        ("log_sum_out", ctypes.c_void_p),
    ]


class lmloss_logprobs_grad_args(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("ids_dtype", ctypes.c_int32),
        ("tokens", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("temperature", ctypes.c_float),
        ("token_mask", ctypes.c_void_p),
        ("mask_stride", ctypes.c_int64),
        ("lse", ctypes.c_void_p),
        ("grad_logp", ctypes.c_void_p),
        ("entropy", ctypes.c_void_p),
        ("grad_entropy", ctypes.c_void_p),
        ("grad_out", ctypes.c_void_p),
        ("ld_grad", ctypes.c_int64),
        ("row_max", ctypes.c_void_p),
        ("log_sum", ctypes.c_void_p),
    ]


class lmloss_table4(ctypes.Structure):
    _fields_ = [
        ("values", ctypes.c_void_p),
        ("ld_values", ctypes.c_int64),
        ("scales", ctypes.c_void_p),
        ("ld_scales", ctypes.c_int64),
        ("zeros", ctypes.c_void_p),
        ("ld_zeros", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("D", ctypes.c_int64),
        ("group", ctypes.c_int32),
        ("scale_dtype", ctypes.c_int32),
    ]


class lmloss_table4_quantize_args(ctypes.Structure):
    _fields_ = [
        ("table", lmloss_table4),
        ("weight", ctypes.c_void_p),
        ("ld_weight", ctypes.c_int64),
        ("weight_dtype", ctypes.c_int32),
    ]


class lmloss_table4_lookup_args(ctypes.Structure):
    _fields_ = [
        ("table", lmloss_table4),
        ("ids", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("rows", ctypes.c_void_p),
        ("ld_rows", ctypes.c_int64),
        ("ids_dtype", ctypes.c_int32),
        ("rows_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class lmloss_table4_logits_args(ctypes.Structure):
    _fields_ = [
        ("table", lmloss_table4),
        ("hidden", ctypes.c_void_p),
        ("T", ctypes.c_int64),
        ("ld_hidden", ctypes.c_int64),
        ("logits", ctypes.c_void_p),
        ("ld_logits", ctypes.c_int64),
        ("hidden_dtype", ctypes.c_int32),
        ("logits_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load the built library.  Raises if it was never built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"lmloss CUDA library not built ({LIB_PATH} missing); run build() first")
    lib = ctypes.CDLL(LIB_PATH)
    h = ctypes.c_void_p
    st = ctypes.c_int
    sig = {
        "lmloss_create": ([ctypes.POINTER(h), ctypes.c_int, ctypes.c_int64, ctypes.c_int32], st),
        "lmloss_destroy": ([h], st),
        "lmloss_check_args": ([ctypes.POINTER(lmloss_args)], st),
        "lmloss_forward_backward": ([h, ctypes.POINTER(lmloss_args), ctypes.c_void_p], st),
        "lmloss_get_device_error": ([h], st),
        "lmloss_status_string": ([st], ctypes.c_char_p),
        "lmloss_set_launch_config": ([h, ctypes.c_int, ctypes.c_int, ctypes.c_int], st),
        "lmloss_forward_backward_host": ([h, ctypes.POINTER(lmloss_args), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_void_p], st),
        "lmloss_set_timing": ([h, ctypes.c_int], st),
        "lmloss_get_timing": ([h, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32)], st),
        "lmloss_get_call_info": ([h, ctypes.POINTER(lmloss_call_info)], st),
        "lmloss_selftest_bounded_wait": ([h, ctypes.c_longlong], st),
        "lmloss_shard_stats": ([h, ctypes.POINTER(lmloss_args), ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                ctypes.c_void_p], st),
        "lmloss_shard_merge": ([h, ctypes.POINTER(lmloss_args), ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32,
                                ctypes.c_void_p], st),
        "lmloss_shard_grad": ([h, ctypes.POINTER(lmloss_args), ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p], st),
        "lmloss_vocab_create": ([ctypes.POINTER(h), ctypes.c_int, ctypes.c_size_t], st),
        "lmloss_vocab_reserve": ([h, ctypes.c_size_t], st),
        "lmloss_vocab_destroy": ([h], st),
        "lmloss_vocab_get_device_error": ([h], st),
        "lmloss_embedding_check_args": ([ctypes.POINTER(lmloss_embedding_args)], st),
        "lmloss_embedding_workspace": ([ctypes.POINTER(lmloss_embedding_args), ctypes.POINTER(ctypes.c_size_t)], st),
        "lmloss_embedding_forward": ([h, ctypes.POINTER(lmloss_embedding_args), ctypes.c_void_p], st),
        "lmloss_embedding_backward": ([h, ctypes.POINTER(lmloss_embedding_args), ctypes.c_void_p], st),
        "lmloss_beam_check_args": ([ctypes.POINTER(lmloss_beam_args)], st),
        "lmloss_beam_workspace": ([ctypes.POINTER(lmloss_beam_args), ctypes.POINTER(ctypes.c_size_t)], st),
        "lmloss_beam_step": ([h, ctypes.POINTER(lmloss_beam_args), ctypes.c_void_p], st),
        "lmloss_beam_check_states": ([ctypes.POINTER(lmloss_beam_state), ctypes.c_int32, ctypes.c_int64,
                                      ctypes.c_int32, ctypes.c_int32], st),
        "lmloss_beam_reorder": ([h, ctypes.POINTER(lmloss_beam_state), ctypes.c_int32, ctypes.c_void_p,
                                 ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p], st),
        "lmloss_logprobs_check_args": ([ctypes.POINTER(lmloss_logprobs_args)], st),
        "lmloss_logprobs_workspace": ([ctypes.POINTER(lmloss_logprobs_args), ctypes.POINTER(ctypes.c_size_t)], st),
        "lmloss_logprobs_forward": ([h, ctypes.POINTER(lmloss_logprobs_args), ctypes.c_void_p], st),
        "lmloss_logprobs_check_grad_args": ([ctypes.POINTER(lmloss_logprobs_grad_args)], st),
        "lmloss_logprobs_backward": ([h, ctypes.POINTER(lmloss_logprobs_grad_args), ctypes.c_void_p], st),
        "lmloss_table4_check": ([ctypes.POINTER(lmloss_table4)], st),
        "lmloss_table4_check_quantize_args": ([ctypes.POINTER(lmloss_table4_quantize_args)], st),
        "lmloss_table4_check_lookup_args": ([ctypes.POINTER(lmloss_table4_lookup_args)], st),
        "lmloss_table4_check_logits_args": ([ctypes.POINTER(lmloss_table4_logits_args)], st),
        "lmloss_table4_quantize": ([h, ctypes.POINTER(lmloss_table4_quantize_args), ctypes.c_void_p], st),
        "lmloss_table4_lookup": ([h, ctypes.POINTER(lmloss_table4_lookup_args), ctypes.c_void_p], st),
        "lmloss_table4_logits_workspace": ([ctypes.POINTER(lmloss_table4_logits_args),
                                            ctypes.POINTER(ctypes.c_size_t)], st),
        "lmloss_table4_logits": ([h, ctypes.POINTER(lmloss_table4_logits_args), ctypes.c_void_p], st),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def exported_names():
    """Function names declared in include/lmloss.h."""
    import re
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:lmloss_status|const char\*)\s+(lmloss_\w+)\s*\(", txt, re.M)))


class LMLossError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        msg = lmloss_status_string(status)
        super().__init__(f"{where}: {msg} (status {status})" if where else f"{msg} (status {status})")


# ---- same-name wrappers over the C entry points -----------------------------
def lmloss_status_string(status: int) -> str:
    return load().lmloss_status_string(int(status)).decode()


def lmloss_create(device: int, max_T: int, max_segments: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    st = load().lmloss_create(ctypes.byref(h), int(device), int(max_T), int(max_segments))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_create")
    return h


def lmloss_destroy(handle) -> int:
    return load().lmloss_destroy(handle)


def lmloss_check_args(args: lmloss_args) -> int:
    return load().lmloss_check_args(ctypes.byref(args))


def lmloss_forward_backward(handle, args: lmloss_args, stream: int) -> int:
    return load().lmloss_forward_backward(handle, ctypes.byref(args), ctypes.c_void_p(stream))


def lmloss_get_device_error(handle) -> int:
    return load().lmloss_get_device_error(handle)


def lmloss_forward_backward_host(handle, args, host_logits, host_teacher, chunk_rows: int, stream) -> int:
    return load().lmloss_forward_backward_host(handle, ctypes.byref(args), host_logits, host_teacher, chunk_rows,
                                               ctypes.c_void_p(stream))


def lmloss_set_launch_config(handle, cluster: int = 0, threads: int = 0, nbuf: int = 0) -> int:
    return load().lmloss_set_launch_config(handle, cluster, threads, nbuf)


def lmloss_set_timing(handle, enable: bool) -> int:
    return load().lmloss_set_timing(handle, 1 if enable else 0)


def lmloss_get_timing(handle):
    """(summed main-kernel milliseconds, calls recorded) since timing was enabled."""
    ms = ctypes.c_float()
    n = ctypes.c_int32()
    st = load().lmloss_get_timing(handle, ctypes.byref(ms), ctypes.byref(n))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_get_timing")
    return float(ms.value), int(n.value)


def lmloss_selftest_bounded_wait(handle, limit_cycles: int) -> int:
    return load().lmloss_selftest_bounded_wait(handle, int(limit_cycles))


def lmloss_get_call_info(handle) -> dict:
    info = lmloss_call_info()
    st = load().lmloss_get_call_info(handle, ctypes.byref(info))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_get_call_info")
    return {n: getattr(info, n) for n, _ in lmloss_call_info._fields_}


def lmloss_forward_backward_noalloc(args: lmloss_args, stream: int) -> int:
    """Allocation-free variant of lmloss_forward_backward on the current device.

    For callers that may not allocate device memory once running (an
    inference-engine plugin whose enqueue step must not allocate, or a service
    that plans all device memory at start-up).  The workspace is a fixed array
    inside the library; a call with more than LMLOSS_NOALLOC_MAX_T rows or
    LMLOSS_NOALLOC_MAX_SEGMENTS segments returns LMLOSS_ERR_INVALID_ARG.  The
    first call on a device does a one-time look-up (make it before any stream
    capture); calls that overlap on the GPU share the array and race.
    """
    fn = load().lmloss_forward_backward_noalloc
    fn.argtypes = [ctypes.POINTER(lmloss_args), ctypes.c_void_p]
    fn.restype = ctypes.c_int
    return fn(ctypes.byref(args), ctypes.c_void_p(stream))


# ---- vocabulary operators
def lmloss_vocab_create(device: int, workspace_bytes: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    st = load().lmloss_vocab_create(ctypes.byref(h), int(device), int(workspace_bytes))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_vocab_create")
    return h


def lmloss_vocab_reserve(handle, workspace_bytes: int) -> int:
    return load().lmloss_vocab_reserve(handle, workspace_bytes)


def lmloss_vocab_destroy(handle) -> int:
    return load().lmloss_vocab_destroy(handle)


def lmloss_vocab_get_device_error(handle) -> int:
    return load().lmloss_vocab_get_device_error(handle)


def lmloss_embedding_check_args(args: lmloss_embedding_args) -> int:
    return load().lmloss_embedding_check_args(ctypes.byref(args))


def lmloss_embedding_workspace(args: lmloss_embedding_args) -> int:
    n = ctypes.c_size_t()
    st = load().lmloss_embedding_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_embedding_workspace")
    return n.value


def lmloss_embedding_forward(handle, args: lmloss_embedding_args, stream: int) -> int:
    return load().lmloss_embedding_forward(handle, ctypes.byref(args), stream)


def lmloss_embedding_backward(handle, args: lmloss_embedding_args, stream: int) -> int:
    return load().lmloss_embedding_backward(handle, ctypes.byref(args), stream)


def lmloss_beam_check_args(args: lmloss_beam_args) -> int:
    return load().lmloss_beam_check_args(ctypes.byref(args))


def lmloss_beam_workspace(args: lmloss_beam_args) -> int:
    n = ctypes.c_size_t()
    st = load().lmloss_beam_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_beam_workspace")
    return n.value


def lmloss_beam_step(handle, args: lmloss_beam_args, stream: int) -> int:
    return load().lmloss_beam_step(handle, ctypes.byref(args), stream)


def lmloss_beam_check_states(states, B: int, K: int, K_out: int) -> int:
    """states: a ctypes array of lmloss_beam_state."""
    return load().lmloss_beam_check_states(states, len(states), B, K, K_out)


def lmloss_beam_reorder(handle, states, parents: int, B: int, K: int, K_out: int, stream: int) -> int:
    return load().lmloss_beam_reorder(handle, states, len(states), parents, B, K, K_out, stream)

def lmloss_logprobs_check_args(args: lmloss_logprobs_args) -> int:
    return load().lmloss_logprobs_check_args(ctypes.byref(args))


def lmloss_logprobs_workspace(args: lmloss_logprobs_args) -> int:
    n = ctypes.c_size_t()
    st = load().lmloss_logprobs_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_logprobs_workspace")
    return n.value


def lmloss_logprobs_forward(handle, args: lmloss_logprobs_args, stream: int) -> int:
    return load().lmloss_logprobs_forward(handle, ctypes.byref(args), stream)


def lmloss_logprobs_check_grad_args(args: lmloss_logprobs_grad_args) -> int:
    return load().lmloss_logprobs_check_grad_args(ctypes.byref(args))


def lmloss_logprobs_backward(handle, args: lmloss_logprobs_grad_args, stream: int) -> int:
    return load().lmloss_logprobs_backward(handle, ctypes.byref(args), stream)


def lmloss_table4_check(args: lmloss_table4) -> int:
    return load().lmloss_table4_check(ctypes.byref(args))


def lmloss_table4_check_quantize_args(args: lmloss_table4_quantize_args) -> int:
    return load().lmloss_table4_check_quantize_args(ctypes.byref(args))


def lmloss_table4_check_lookup_args(args: lmloss_table4_lookup_args) -> int:
    return load().lmloss_table4_check_lookup_args(ctypes.byref(args))


def lmloss_table4_check_logits_args(args: lmloss_table4_logits_args) -> int:
    return load().lmloss_table4_check_logits_args(ctypes.byref(args))


def lmloss_table4_logits_workspace(args: lmloss_table4_logits_args) -> int:
    n = ctypes.c_size_t()
    st = load().lmloss_table4_logits_workspace(ctypes.byref(args), ctypes.byref(n))
    if st != LMLOSS_OK:
        raise LMLossError(st, "lmloss_table4_logits_workspace")
    return n.value


def lmloss_table4_quantize(handle, args: lmloss_table4_quantize_args, stream: int) -> int:
    return load().lmloss_table4_quantize(handle, ctypes.byref(args), stream)


def lmloss_table4_lookup(handle, args: lmloss_table4_lookup_args, stream: int) -> int:
    return load().lmloss_table4_lookup(handle, ctypes.byref(args), stream)


def lmloss_table4_logits(handle, args: lmloss_table4_logits_args, stream: int) -> int:
    return load().lmloss_table4_logits(handle, ctypes.byref(args), stream)
