"""Python binding of libmuse_lmhead.so: the Muse Glimmer decode output stage
(final RMSNorm -> Q5_K LM-head matvec -> scale -> soft cap -> argmax) on one
GB300.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  The functions named
``muse_lmhead_*`` mirror the C-ABI in include/muse_lmhead.h one to one (plain
integers for pointers and streams); :class:`LMHead` wraps them for torch
tensors.  If the compiled library is missing, importing works but every call
raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple

__all__ = [
    "LMHead", "TokenScores", "MuseError", "library_path", "load_library",
    "muse_lmhead_init", "muse_lmhead_forward", "muse_lmhead_forward_host",
    "muse_lmhead_launches_per_forward", "muse_lmhead_path_name", "muse_lmhead_device_status",
    "muse_lmhead_destroy", "muse_lmhead_status_string", "muse_lmhead_forward_b1_noalloc",
    "muse_lmhead_noalloc_device_status",
    "muse_lmhead_forward_group", "muse_lmhead_forward_group_host", "MuseGemvSegment", "MUSE_MAX_SEGMENTS",
    "muse_lmhead_forward_logprobs",
    "muse_lmhead_init_format", "MUSE_FORMAT_Q5_K", "MUSE_FORMAT_Q4_K", "BLOCK_BYTES",
    "muse_lmhead_clear_device_status", "muse_lmhead_selftest_wait_timeout",
    "muse_lmhead_set_argmax_key", "MUSE_ARGMAX_CAPPED", "MUSE_ARGMAX_PRECAP",
    "muse_lmhead_score", "muse_lmhead_forward_score", "muse_lmhead_distill", "muse_lmhead_backward", "MUSE_MAX_TOP",
    "muse_lmhead_embed", "muse_lmhead_embed_backward", "muse_lmhead_embed_backward_workspace",
    "muse_lmhead_sample", "muse_lmhead_forward_sample", "MuseSampling",
    "EXPORTED_SYMBOLS",
    "LOGIT_SCALE", "SOFTCAP", "RMS_EPS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuse_lmhead.so")

# Constants of the Muse Glimmer checkpoint ("Chapter 20 — Final norm, LM head,
# and the soft cap", §20.1 and §20.5): read from GGUF metadata there, passed as
# call arguments here.
LOGIT_SCALE = 0.196116
SOFTCAP = 20.0
RMS_EPS = 1e-5

EXPORTED_SYMBOLS = (
    "muse_lmhead_init", "muse_lmhead_forward", "muse_lmhead_forward_host",
    "muse_lmhead_launches_per_forward", "muse_lmhead_path_name", "muse_lmhead_device_status",
    "muse_lmhead_destroy", "muse_lmhead_status_string", "muse_lmhead_forward_b1_noalloc",
    "muse_lmhead_noalloc_device_status",
    "muse_lmhead_forward_group", "muse_lmhead_forward_group_host", "muse_lmhead_forward_logprobs",
    "muse_lmhead_init_format",
    "muse_lmhead_clear_device_status", "muse_lmhead_selftest_wait_timeout", "muse_lmhead_set_argmax_key",
    "muse_lmhead_score", "muse_lmhead_forward_score", "muse_lmhead_distill", "muse_lmhead_backward",
    "muse_lmhead_embed", "muse_lmhead_embed_backward", "muse_lmhead_embed_backward_workspace",
    "muse_lmhead_sample", "muse_lmhead_forward_sample",
)

MUSE_OK = 0
MUSE_MAX_BATCH = 32
MUSE_MAX_SEGMENTS = 4
MUSE_FORMAT_Q5_K = 0
MUSE_FORMAT_Q4_K = 1
FORMATS = {"q5_k": MUSE_FORMAT_Q5_K, "q4_k": MUSE_FORMAT_Q4_K}
BLOCK_BYTES = {"q5_k": 176, "q4_k": 144}
STATUS_WAIT_TIMEOUT = 1
MUSE_ARGMAX_CAPPED = 0      # argmax key: the returned (capped) logit
MUSE_ARGMAX_PRECAP = 1      # argmax key: scale * raw, before the cap
MUSE_MAX_TOP = 64           # alternatives of a row that are returned (score) or given (distill), at most
MUSE_DTYPE_F32, MUSE_DTYPE_F16, MUSE_DTYPE_BF16 = 0, 1, 2
MUSE_DTYPE_BLOCKS = 3       # a token table of blocks in the handle's format
ARGMAX_KEYS = {"capped": MUSE_ARGMAX_CAPPED, "precap": MUSE_ARGMAX_PRECAP}

_lib = None


class MuseGemvSegment(ctypes.Structure):
    """struct muse_gemv_segment of the C header: one matrix of a grouped forward."""
    _fields_ = [("weights", ctypes.c_void_p), ("n_rows", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("cap", ctypes.c_float)]


class MuseSampling(ctypes.Structure):
    """struct muse_sampling of the C header: a value of each setting, or a device array of one a row."""
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


class MuseError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {muse_lmhead_status_string(status)} (status {status})")


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load the compiled library; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"libmuse_lmhead.so is not built ({LIB_PATH}); run `python -c \"import __graft_entry__ as g; "
            "g.build()\"` or `python q5_lm_head_gb300/_build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.muse_lmhead_init.restype = i32
    lib.muse_lmhead_init.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i32]
    lib.muse_lmhead_init_format.restype = i32
    lib.muse_lmhead_init_format.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i32, i32]
    lib.muse_lmhead_forward.restype = i32
    lib.muse_lmhead_forward.argtypes = [vp, vp, i32, vp, f32, vp, f32, f32, vp, vp, vp]
    lib.muse_lmhead_forward_host.restype = i32
    lib.muse_lmhead_forward_host.argtypes = [vp, vp, i32, vp, f32, vp, f32, f32, vp, vp, vp]
    lib.muse_lmhead_launches_per_forward.restype = i32
    lib.muse_lmhead_launches_per_forward.argtypes = [vp, i32, i32]
    lib.muse_lmhead_path_name.restype = ctypes.c_char_p
    lib.muse_lmhead_path_name.argtypes = [vp, i32]
    lib.muse_lmhead_device_status.restype = i32
    lib.muse_lmhead_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.muse_lmhead_destroy.restype = None
    lib.muse_lmhead_destroy.argtypes = [vp]
    lib.muse_lmhead_status_string.restype = ctypes.c_char_p
    lib.muse_lmhead_status_string.argtypes = [i32]
    lib.muse_lmhead_forward_b1_noalloc.restype = i32
    lib.muse_lmhead_forward_b1_noalloc.argtypes = [i32, vp, vp, f32, vp, i64, i64, f32, f32, vp, vp, vp]
    lib.muse_lmhead_noalloc_device_status.restype = i32
    lib.muse_lmhead_noalloc_device_status.argtypes = [i32, vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.muse_lmhead_clear_device_status.restype = i32
    lib.muse_lmhead_clear_device_status.argtypes = [vp, vp]
    lib.muse_lmhead_selftest_wait_timeout.restype = i32
    lib.muse_lmhead_selftest_wait_timeout.argtypes = [vp, vp]
    lib.muse_lmhead_set_argmax_key.restype = i32
    lib.muse_lmhead_set_argmax_key.argtypes = [vp, i32]
    lib.muse_lmhead_forward_logprobs.restype = i32
    lib.muse_lmhead_forward_logprobs.argtypes = [vp, vp, i32, vp, f32, vp, f32, f32, vp, vp, vp, vp]
    lib.muse_lmhead_forward_group.restype = i32
    lib.muse_lmhead_forward_group.argtypes = [vp, vp, vp, f32, ctypes.POINTER(MuseGemvSegment), i32, vp]
    lib.muse_lmhead_forward_group_host.restype = i32
    lib.muse_lmhead_forward_group_host.argtypes = [vp, vp, vp, f32, ctypes.POINTER(MuseGemvSegment), i32, vp]
    lib.muse_lmhead_score.restype = i32
    lib.muse_lmhead_score.argtypes = [vp, vp, i32, i64, i64, vp, f32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.muse_lmhead_forward_score.restype = i32
    lib.muse_lmhead_forward_score.argtypes = [vp, vp, i32, vp, f32, vp, f32, f32, vp, vp, f32, i32, vp, vp, vp, vp,
                                              vp, vp, vp]
    lib.muse_lmhead_distill.restype = i32
    lib.muse_lmhead_distill.argtypes = [vp, vp, i32, i64, i64, vp, vp, i32, i32, vp, f32, vp, vp, i64, vp]
    lib.muse_lmhead_backward.restype = i32
    lib.muse_lmhead_backward.argtypes = [vp, vp, vp, vp, i32, vp, f32, vp, f32, f32, vp, vp, vp]
    how = ctypes.POINTER(MuseSampling)
    lib.muse_lmhead_sample.restype = i32
    lib.muse_lmhead_sample.argtypes = [vp, vp, i32, i64, i64, how, vp, vp, vp, vp]
    lib.muse_lmhead_forward_sample.restype = i32
    lib.muse_lmhead_forward_sample.argtypes = [vp, vp, i32, vp, f32, vp, f32, f32, vp, how, vp, vp, vp, vp]
    lib.muse_lmhead_embed.restype = i32
    lib.muse_lmhead_embed.argtypes = [vp, vp, i32, i64, vp, i64, f32, vp, i32, i64, vp]
    lib.muse_lmhead_embed_backward.restype = i32
    lib.muse_lmhead_embed_backward.argtypes = [vp, vp, i32, i64, vp, i64, f32, vp, i32, i64, i32, vp, i64, vp]
    lib.muse_lmhead_embed_backward_workspace.restype = i32
    lib.muse_lmhead_embed_backward_workspace.argtypes = [vp, i64, ctypes.POINTER(i64)]
    _lib = lib
    return lib


# ------------------------------------------------------------ same-named C-ABI calls
def muse_lmhead_init(device: int, n_rows: int, k: int, max_batch: int) -> int:
    """Returns the handle (an integer) or raises MuseError."""
    h = ctypes.c_void_p()
    st = load_library().muse_lmhead_init(ctypes.byref(h), device, n_rows, k, max_batch)
    if st != MUSE_OK:
        raise MuseError(st, "muse_lmhead_init")
    return h.value


def muse_lmhead_init_format(device: int, n_rows: int, k: int, max_batch: int, fmt: int) -> int:
    """Returns the handle (an integer) or raises MuseError."""
    h = ctypes.c_void_p()
    st = load_library().muse_lmhead_init_format(ctypes.byref(h), device, n_rows, k, max_batch, fmt)
    if st != MUSE_OK:
        raise MuseError(st, "muse_lmhead_init_format")
    return h.value


def muse_lmhead_forward(h: int, hidden: int, batch: int, gamma: int | None, eps: float, weights: int,
                        scale: float, cap: float, logits: int, argmax: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_forward(h, hidden, batch, gamma, eps, weights, scale, cap, logits,
                                              argmax, stream)


def muse_lmhead_forward_host(h: int, hidden_host: int, batch: int, gamma: int | None, eps: float,
                             weights: int, scale: float, cap: float, logits_host: int | None,
                             argmax_host: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_forward_host(h, hidden_host, batch, gamma, eps, weights, scale, cap,
                                                   logits_host, argmax_host, stream)


def muse_lmhead_launches_per_forward(h: int, batch: int, with_norm: bool) -> int:
    return load_library().muse_lmhead_launches_per_forward(h, batch, int(bool(with_norm)))


def muse_lmhead_path_name(h: int, batch: int) -> str | None:
    r = load_library().muse_lmhead_path_name(h, batch)
    return None if r is None else r.decode()


def muse_lmhead_device_status(h: int) -> int:
    v = ctypes.c_uint32()
    st = load_library().muse_lmhead_device_status(h, ctypes.byref(v))
    if st != MUSE_OK:
        raise MuseError(st, "muse_lmhead_device_status")
    return v.value


def muse_lmhead_destroy(h: int | None) -> None:
    if h:
        load_library().muse_lmhead_destroy(h)


def muse_lmhead_forward_b1_noalloc(device: int, hidden: int, gamma: int | None, eps: float, weights: int,
                                   n_rows: int, k: int, scale: float, cap: float, logits: int,
                                   argmax: int | None, stream: int | None) -> int:
    """Batch-1 forward without a handle that allocates no device memory (see the C header)."""
    return load_library().muse_lmhead_forward_b1_noalloc(device, hidden, gamma, eps, weights, n_rows, k, scale,
                                                         cap, logits, argmax, stream)


def muse_lmhead_noalloc_device_status(device: int, stream: int | None) -> int:
    """Status word of the no-alloc forward on `device`, read after the work
    queued on `stream` and cleared (see the C header); raises on a failed read."""
    v = ctypes.c_uint32()
    st = load_library().muse_lmhead_noalloc_device_status(device, stream, ctypes.byref(v))
    if st != MUSE_OK:
        raise MuseError(st, "muse_lmhead_noalloc_device_status")
    return v.value


def muse_lmhead_status_string(status: int) -> str:
    return load_library().muse_lmhead_status_string(status).decode()


# ------------------------------------------------------------ torch-facing wrapper
def muse_lmhead_clear_device_status(h: int, stream: int | None = None) -> int:
    return load_library().muse_lmhead_clear_device_status(h, stream)


def muse_lmhead_set_argmax_key(h: int | None, key: int) -> int:
    return load_library().muse_lmhead_set_argmax_key(h, key)


def muse_lmhead_selftest_wait_timeout(h: int, stream: int | None = None) -> int:
    return load_library().muse_lmhead_selftest_wait_timeout(h, stream)


def muse_lmhead_forward_logprobs(h: int, hidden: int, batch: int, gamma: int | None, eps: float, weights: int,
                                 scale: float, cap: float, logprobs: int, lse: int | None, argmax: int | None,
                                 stream: int | None) -> int:
    return load_library().muse_lmhead_forward_logprobs(h, hidden, batch, gamma, eps, weights, scale, cap,
                                                       logprobs, lse, argmax, stream)


def muse_lmhead_forward_group(h: int | None, hidden: int, gamma: int | None, eps: float, segments,
                              stream: int | None) -> int:
    """segments: sequence of (weights_ptr, n_rows, out_ptr, scale, cap)."""
    arr = (MuseGemvSegment * max(1, len(segments)))()
    for i, (w, n, o, sc, cp) in enumerate(segments):
        arr[i] = MuseGemvSegment(w, n, o, sc, cp)
    return load_library().muse_lmhead_forward_group(h, hidden, gamma, eps, arr, len(segments), stream)


def muse_lmhead_forward_group_host(h: int | None, hidden_host: int, gamma: int | None, eps: float, segments,
                                   stream: int | None) -> int:
    """segments: sequence of (weights_ptr (device), n_rows, out_ptr (host), scale, cap)."""
    arr = (MuseGemvSegment * max(1, len(segments)))()
    for i, (w, n, o, sc, cp) in enumerate(segments):
        arr[i] = MuseGemvSegment(w, n, o, sc, cp)
    return load_library().muse_lmhead_forward_group_host(h, hidden_host, gamma, eps, arr, len(segments), stream)


def muse_lmhead_score(h: int | None, logits: int, dtype: int, n: int, ld: int, tokens: int | None,
                      temperature: float, n_top: int, logprob: int | None, rank: int | None, lse: int | None,
                      entropy: int | None, top_ids: int | None, top_logprobs: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_score(h, logits, dtype, n, ld, tokens, temperature, n_top, logprob, rank, lse,
                                            entropy, top_ids, top_logprobs, stream)


def muse_lmhead_forward_score(h: int | None, hidden: int, batch: int, gamma: int | None, eps: float, weights: int,
                              scale: float, cap: float, logits: int, tokens: int | None, temperature: float,
                              n_top: int, logprob: int | None, rank: int | None, lse: int | None,
                              entropy: int | None, top_ids: int | None, top_logprobs: int | None,
                              stream: int | None) -> int:
    return load_library().muse_lmhead_forward_score(h, hidden, batch, gamma, eps, weights, scale, cap, logits, tokens,
                                                    temperature, n_top, logprob, rank, lse, entropy, top_ids,
                                                    top_logprobs, stream)


def muse_lmhead_distill(h: int | None, logits: int, dtype: int, n: int, ld: int, teacher_ids: int,
                        teacher_logprobs: int, n_top: int, tail: int, row_weight: int | None, temperature: float,
                        loss: int | None, grad: int | None, grad_ld: int, stream: int | None) -> int:
    return load_library().muse_lmhead_distill(h, logits, dtype, n, ld, teacher_ids, teacher_logprobs, n_top, tail,
                                              row_weight, temperature, loss, grad, grad_ld, stream)


def muse_lmhead_backward(h: int | None, grad_logits: int, logits: int | None, hidden: int | None, batch: int,
                         gamma: int | None, eps: float, weights: int, scale: float, cap: float, grad_hidden: int,
                         grad_gamma: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_backward(h, grad_logits, logits, hidden, batch, gamma, eps, weights, scale, cap,
                                               grad_hidden, grad_gamma, stream)


def muse_lmhead_sample(h: int | None, logits: int, dtype: int, n: int, ld: int, how: MuseSampling | None,
                       uniforms: int, tokens: int, logprobs: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_sample(h, logits, dtype, n, ld, how, uniforms, tokens, logprobs, stream)


def muse_lmhead_forward_sample(h: int | None, hidden: int, batch: int, gamma: int | None, eps: float, weights: int,
                               scale: float, cap: float, logits: int, how: MuseSampling | None, uniforms: int,
                               tokens: int, logprobs: int | None, stream: int | None) -> int:
    return load_library().muse_lmhead_forward_sample(h, hidden, batch, gamma, eps, weights, scale, cap, logits, how,
                                                     uniforms, tokens, logprobs, stream)


def muse_lmhead_embed(h: int | None, table: int, table_type: int, table_ld: int, tokens: int, n: int, scale: float,
                      out: int, out_dtype: int, out_ld: int, stream: int | None) -> int:
    return load_library().muse_lmhead_embed(h, table, table_type, table_ld, tokens, n, scale, out, out_dtype, out_ld,
                                            stream)


def muse_lmhead_embed_backward(h: int | None, grad: int, dtype: int, grad_ld: int, tokens: int, n: int, scale: float,
                               grad_table: int, table_dtype: int, table_ld: int, accumulate: int, workspace: int,
                               workspace_bytes: int, stream: int | None) -> int:
    return load_library().muse_lmhead_embed_backward(h, grad, dtype, grad_ld, tokens, n, scale, grad_table, table_dtype,
                                                     table_ld, accumulate, workspace, workspace_bytes, stream)


def muse_lmhead_embed_backward_workspace(h: int | None, n: int) -> int:
    """Bytes of workspace for n positions, or raises MuseError."""
    v = ctypes.c_int64()
    st = load_library().muse_lmhead_embed_backward_workspace(h, n, ctypes.byref(v))
    if st != MUSE_OK:
        raise MuseError(st, "muse_lmhead_embed_backward_workspace")
    return v.value


_stream_of = None


def _current_stream():
    """Function of a device index: its current stream's handle (without a Stream object, where torch has that call)."""
    global _stream_of
    if _stream_of is None:
        import torch
        _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _stream_of


_dtypes = None


def _row_dtypes():
    """MUSE_DTYPE of a torch dtype."""
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {torch.float32: MUSE_DTYPE_F32, torch.float16: MUSE_DTYPE_F16, torch.bfloat16: MUSE_DTYPE_BF16}
    return _dtypes


class TokenScores(NamedTuple):
    """What LMHead.score returns, one entry a row (None for what was not asked for)."""
    logprob: Any        # [n] f32, the given token's (0 in a padded row)
    rank: Any           # [n] int32, how many tokens come before it (-1 in a padded row)
    lse: Any            # [n] f32, the normaliser at the given temperature
    entropy: Any        # [n] f32, natural log
    top_ids: Any        # [n, n_top] int32
    top_logprobs: Any   # [n, n_top] f32


class LMHead:
    """A handle for one [n_rows x k] Q5_K (or, fmt="q4_k", Q4_K) matrix and batches up to max_batch.

    Calls run on torch's current stream, or on the one given as `stream`.  A call
    on another stream than the current one does not wait for it, nor does the
    current one wait: that is the caller's, as with torch's own operations.  Its
    tensors' memory is safe either way: results are allocated for `stream`, and
    neither inputs nor results, once let go, are used again before both streams
    are done with them."""

    def __init__(self, n_rows: int, k: int, max_batch: int = MUSE_MAX_BATCH, device: int | None = None,
                 fmt: str = "q5_k"):
        import torch
        if fmt not in FORMATS:
            raise ValueError(f"fmt must be one of {sorted(FORMATS)}")
        self.device = torch.cuda.current_device() if device is None else int(device)
        self.n_rows, self.k, self.max_batch = int(n_rows), int(k), int(max_batch)
        self.fmt, self.block_bytes = fmt, BLOCK_BYTES[fmt]
        self.handle = muse_lmhead_init_format(self.device, self.n_rows, self.k, self.max_batch, FORMATS[fmt])

    def close(self):
        if getattr(self, "handle", None):
            muse_lmhead_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _allocator(self, stream, *used):
        """torch.empty for a call's results; with a stream of its own, for that stream's use, and
        the call's other tensors are marked as used there."""
        import torch
        if stream is None or stream.cuda_stream == _current_stream()(self.device):
            return torch.empty
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=self.device)
        for t in used:
            if t is not None and t.is_cuda:
                t.record_stream(stream)

        def empty(shape, dtype, device):
            # A block of the current stream's may still be in use by what is queued there.
            current, device_before = torch.cuda.current_stream(self.device), torch.cuda.current_device()
            torch.cuda.set_stream(stream)      # a context manager a tensor would cost the call 20 us
            try:
                t = torch.empty(shape, dtype=dtype, device=device)
            finally:
                torch.cuda.set_stream(current)
                if device_before != self.device:
                    torch.cuda.set_device(device_before)
            t.record_stream(current)
            return t

        return empty

    def _check(self, t, name, dtype, shape=None):
        if t.dtype != dtype or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{name}: need a contiguous {dtype} tensor on cuda:{self.device}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
        return t.data_ptr()

    def forward(self, hidden, weights, gamma=None, eps: float = RMS_EPS, scale: float = LOGIT_SCALE,
                cap: float = SOFTCAP, want_argmax: bool = True, logits=None, argmax=None, stream=None):
        """logits [B, n_rows] f32 (and argmax [B] int32) for hidden [B, k] f32 on the GPU."""
        import torch
        if hidden.dim() == 1:
            hidden = hidden.unsqueeze(0)
        b = hidden.shape[0]
        hp = self._check(hidden, "hidden", torch.float32, (b, self.k))
        wp = self._check(weights, "weights", torch.uint8)
        if weights.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
            raise ValueError("weights: wrong number of bytes for this handle")
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        empty = self._allocator(stream, hidden, weights, gamma, logits, argmax)
        if logits is None:
            logits = empty((b, self.n_rows), dtype=torch.float32, device=hidden.device)
        lp = self._check(logits, "logits", torch.float32, (b, self.n_rows))
        ap = None
        if want_argmax:
            if argmax is None:
                argmax = empty((b,), dtype=torch.int32, device=hidden.device)
            ap = self._check(argmax, "argmax", torch.int32, (b,))
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        st = muse_lmhead_forward(self.handle, hp, b, gp, float(eps), wp, float(scale), float(cap), lp, ap,
                                 s.cuda_stream)
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward")
        return (logits, argmax) if want_argmax else logits

    def forward_host(self, hidden_host, weights, gamma=None, eps: float = RMS_EPS, scale: float = LOGIT_SCALE,
                     cap: float = SOFTCAP, logits_host=None, argmax_host=None, stream=None):
        """Host-memory forward: hidden_host [B, k] f32 CPU tensor (pinned for speed); returns CPU tensors.
        Pinned output tensors (the default) are written by the kernels directly through the
        device's mapping of host memory; pageable ones are filled by a copy after the kernels."""
        import torch
        if hidden_host.dim() == 1:
            hidden_host = hidden_host.unsqueeze(0)
        if hidden_host.device.type != "cpu" or hidden_host.dtype != torch.float32 or not hidden_host.is_contiguous():
            raise ValueError("hidden_host: need a contiguous f32 CPU tensor")
        b = hidden_host.shape[0]
        if logits_host is None:
            logits_host = torch.empty((b, self.n_rows), dtype=torch.float32, pin_memory=True)
        if argmax_host is None:
            argmax_host = torch.empty((b,), dtype=torch.int32, pin_memory=True)
        wp = self._check(weights, "weights", torch.uint8)
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        st = muse_lmhead_forward_host(self.handle, hidden_host.data_ptr(), b, gp, float(eps), wp, float(scale),
                                      float(cap), logits_host.data_ptr(), argmax_host.data_ptr(), s.cuda_stream)
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_host")
        return logits_host, argmax_host

    def forward_logprobs(self, hidden, weights, gamma=None, eps: float = RMS_EPS, scale: float = LOGIT_SCALE,
                         cap: float = SOFTCAP, want_argmax: bool = True, logprobs=None, lse=None, argmax=None,
                         stream=None):
        """(logprobs [B, n_rows], lse [B][, argmax [B]]): log-softmax of the capped logits."""
        import torch
        if hidden.dim() == 1:
            hidden = hidden.unsqueeze(0)
        b = hidden.shape[0]
        hp = self._check(hidden, "hidden", torch.float32, (b, self.k))
        wp = self._check(weights, "weights", torch.uint8)
        if weights.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
            raise ValueError("weights: wrong number of bytes for this handle")
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        empty = self._allocator(stream, hidden, weights, gamma, logprobs, lse, argmax)
        if logprobs is None:
            logprobs = empty((b, self.n_rows), dtype=torch.float32, device=hidden.device)
        lp = self._check(logprobs, "logprobs", torch.float32, (b, self.n_rows))
        if lse is None:
            lse = empty((b,), dtype=torch.float32, device=hidden.device)
        sp = self._check(lse, "lse", torch.float32, (b,))
        ap = None
        if want_argmax:
            if argmax is None:
                argmax = empty((b,), dtype=torch.int32, device=hidden.device)
            ap = self._check(argmax, "argmax", torch.int32, (b,))
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        st = muse_lmhead_forward_logprobs(self.handle, hp, b, gp, float(eps), wp, float(scale), float(cap), lp, sp,
                                          ap, s.cuda_stream)
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_logprobs")
        return (logprobs, lse, argmax) if want_argmax else (logprobs, lse)

    def forward_group(self, hidden, segments, gamma=None, eps: float = RMS_EPS, stream=None):
        """Up to four matrices against one input row in one launch.

        hidden [k] (or [1, k]) f32 on the GPU; segments: sequence of
        (weights uint8 tensor, n_rows, scale, cap, out or None).  Returns the
        list of outputs ([n_rows] f32 each)."""
        import torch
        h = hidden.reshape(-1)
        hp = self._check(h, "hidden", torch.float32, (self.k,))
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        outs, descs = [], []
        segments = list(segments)
        empty = self._allocator(stream, hidden, gamma, *(seg[0] for seg in segments), *(seg[4] for seg in segments))
        for (w, n, scale, cap, out) in segments:
            wp = self._check(w, "weights", torch.uint8)
            if w.numel() != n * (self.k // 256) * self.block_bytes:
                raise ValueError("weights: wrong number of bytes for n_rows")
            if out is None:
                out = empty((n,), dtype=torch.float32, device=hidden.device)
            op = self._check(out, "out", torch.float32, (n,))
            outs.append(out)
            descs.append((wp, n, op, float(scale), float(cap)))
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        st = muse_lmhead_forward_group(self.handle, hp, gp, float(eps), descs, s.cuda_stream)
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_group")
        return outs

    def forward_group_host(self, hidden_host, segments, gamma=None, eps: float = RMS_EPS, stream=None):
        """The grouped forward from host memory: hidden_host [k] (or [1, k]) f32
        CPU tensor; segments: sequence of (weights uint8 tensor on the GPU,
        n_rows, scale, cap, out CPU tensor or None).  Outputs default to pinned
        CPU tensors, which the kernel writes directly; returns them."""
        import torch
        h = hidden_host.reshape(-1)
        if h.device.type != "cpu" or h.dtype != torch.float32 or not h.is_contiguous() or h.numel() != self.k:
            raise ValueError("hidden_host: need a contiguous f32 CPU tensor of k values")
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        outs, descs = [], []
        for (w, n, scale, cap, out) in segments:
            wp = self._check(w, "weights", torch.uint8)
            if w.numel() != n * (self.k // 256) * self.block_bytes:
                raise ValueError("weights: wrong number of bytes for n_rows")
            if out is None:
                out = torch.empty((n,), dtype=torch.float32, pin_memory=True)
            if out.device.type != "cpu" or out.dtype != torch.float32 or not out.is_contiguous() or out.numel() != n:
                raise ValueError("out: need a contiguous f32 CPU tensor of n_rows values")
            outs.append(out)
            descs.append((wp, n, out.data_ptr(), float(scale), float(cap)))
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        st = muse_lmhead_forward_group_host(self.handle, h.data_ptr(), gp, float(eps), descs, s.cuda_stream)
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_group_host")
        return outs

    def _rows(self, t, name, width=None):
        """(pointer, MUSE_DTYPE, rows, distance) of a matrix of logits (or of `width` columns) whose rows are contiguous."""
        dtype = _row_dtypes().get(t.dtype)
        if dtype is None or t.get_device() != self.device:
            raise ValueError(f"{name}: need a float32, float16 or bfloat16 tensor on cuda:{self.device}")
        shape, v = t.shape, self.n_rows if width is None else width
        if len(shape) != 2 or shape[1] != v:
            raise ValueError(f"{name}: shape {tuple(shape)}, need [n, {v}]")
        n = shape[0]
        ld, step = t.stride()
        if (v > 1 and step != 1) or (n > 1 and ld < v):
            raise ValueError(f"{name}: strides {t.stride()}, need contiguous rows that do not overlap")
        return t.data_ptr(), dtype, n, ld if n > 1 else v

    def _stream(self, stream):
        return _current_stream()(self.device) if stream is None else stream.cuda_stream

    def _score_outputs(self, n, tokens, n_top, device, empty):
        """(TokenScores, pointers of tokens and outputs in the C order)"""
        import torch
        if not 0 <= n_top <= MUSE_MAX_TOP:
            raise ValueError(f"n_top: 0..{MUSE_MAX_TOP}")
        f, i, rows = torch.float32, torch.int32, (n,)
        tp = lp = rp = ip = pp = logprob = rank = ids = top = None
        if tokens is not None:
            tp = self._check(tokens, "tokens", i, rows)
            logprob, rank = empty(rows, dtype=f, device=device), empty(rows, dtype=i, device=device)
            lp, rp = logprob.data_ptr(), rank.data_ptr()
        lse, entropy = empty(rows, dtype=f, device=device), empty(rows, dtype=f, device=device)
        if n_top > 0:
            ids = empty((n, n_top), dtype=i, device=device)
            top = empty((n, n_top), dtype=f, device=device)
            ip, pp = ids.data_ptr(), top.data_ptr()
        return (TokenScores(logprob, rank, lse, entropy, ids, top),
                tp, lp, rp, lse.data_ptr(), entropy.data_ptr(), ip, pp)

    def score(self, logits, tokens=None, n_top: int = 0, temperature: float = 1.0, stream=None) -> TokenScores:
        """Log probability and rank of tokens [n] int32, normaliser, entropy and top alternatives of each row.

        logits [n, n_rows], f32, f16 or bf16, contiguous rows any distance
        apart, any n: what a forward returned (softmax and logprobs are taken
        over the capped logits).  Masked logits are -infinity; a token outside
        0..n_rows-1 marks a padded row.  See muse_lmhead_score in the C header."""
        if logits.dim() == 1:
            logits = logits.unsqueeze(0)
        ptr, dtype, n, ld = self._rows(logits, "logits")
        out, tp, *at = self._score_outputs(n, tokens, n_top, logits.device, self._allocator(stream, logits, tokens))
        st = load_library().muse_lmhead_score(self.handle, ptr, dtype, n, ld, tp, temperature, n_top, *at,
                                              self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_score")
        return out

    def forward_score(self, hidden, weights, gamma=None, eps: float = RMS_EPS, scale: float = LOGIT_SCALE,
                      cap: float = SOFTCAP, tokens=None, n_top: int = 0, temperature: float = 1.0, logits=None,
                      stream=None):
        """(logits [B, n_rows], TokenScores): the forward, and the scores of its logits."""
        import torch
        if hidden.dim() == 1:
            hidden = hidden.unsqueeze(0)
        b = hidden.shape[0]
        hp = self._check(hidden, "hidden", torch.float32, (b, self.k))
        wp = self._check(weights, "weights", torch.uint8)
        if weights.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
            raise ValueError("weights: wrong number of bytes for this handle")
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        empty = self._allocator(stream, hidden, weights, gamma, logits, tokens)
        if logits is None:
            logits = empty((b, self.n_rows), dtype=torch.float32, device=hidden.device)
        lp = self._check(logits, "logits", torch.float32, (b, self.n_rows))
        out, tp, *at = self._score_outputs(b, tokens, n_top, hidden.device, empty)
        st = muse_lmhead_forward_score(self.handle, hp, b, gp, float(eps), wp, float(scale), float(cap), lp, tp,
                                       float(temperature), n_top, *at, self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_score")
        return logits, out

    def distill(self, logits, teacher_ids, teacher_logprobs, row_weight=None, temperature: float = 1.0,
                tail: bool = False, want_grad: bool = True, grad=None, stream=None):
        """(loss [n] f32, grad [n, n_rows] or None): distillation from a teacher's top alternatives.

        logits [n, n_rows] as for score; teacher_ids [n, n_top] int32 and
        teacher_logprobs [n, n_top] f32, such as score returns.  tail: the
        tokens outside teacher_ids are one more class (else the teacher is
        renormalised over its entries).  row_weight [n] f32 scales loss and
        gradient.  grad (the logits' dtype; may be the logits themselves) is
        made when not given, unless want_grad is false.  See
        muse_lmhead_distill in the C header."""
        import torch
        ptr, dtype, n, ld = self._rows(logits, "logits")
        top = teacher_ids.shape[1] if teacher_ids.dim() == 2 else 0
        if not 1 <= top <= MUSE_MAX_TOP:
            raise ValueError(f"teacher_ids: need [n, 1..{MUSE_MAX_TOP}]")
        ip = self._check(teacher_ids, "teacher_ids", torch.int32, (n, top))
        pp = self._check(teacher_logprobs, "teacher_logprobs", torch.float32, (n, top))
        wp = None if row_weight is None else self._check(row_weight, "row_weight", torch.float32, (n,))
        empty = self._allocator(stream, logits, teacher_ids, teacher_logprobs, row_weight, grad)
        loss = empty((n,), dtype=torch.float32, device=logits.device)
        gp, gld = None, 0
        if grad is None and want_grad:
            grad = empty((n, self.n_rows), dtype=logits.dtype, device=logits.device)
        if grad is not None:
            gp, gtype, gn, gld = self._rows(grad, "grad")
            if gtype != dtype or gn != n:
                raise ValueError("grad: need the logits' shape and dtype")
        st = load_library().muse_lmhead_distill(self.handle, ptr, dtype, n, ld, ip, pp, top, 1 if tail else 0, wp,
                                                temperature, loss.data_ptr(), gp, gld, self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_distill")
        return loss, grad

    def backward(self, grad_logits, weights, logits=None, hidden=None, gamma=None, eps: float = RMS_EPS,
                 scale: float = LOGIT_SCALE, cap: float = SOFTCAP, grad_hidden=None, stream=None):
        """(grad_hidden [B, k], grad_gamma [k] or None) from grad_logits [B, n_rows] f32.

        weights, gamma, eps, scale and cap as in the forward; logits (what it
        returned, masked or not: nothing goes back through one outside
        -cap..cap) is needed with a cap, hidden with gamma.  The first call
        allocates the handle's workspace: make it before a graph's capture.
        See muse_lmhead_backward in the C header."""
        import torch
        if grad_logits.dim() == 1:
            grad_logits = grad_logits.unsqueeze(0)
        b = grad_logits.shape[0]
        tp = self._check(grad_logits, "grad_logits", torch.float32, (b, self.n_rows))
        wp = self._check(weights, "weights", torch.uint8)
        if weights.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
            raise ValueError("weights: wrong number of bytes for this handle")
        lp = hp = gp = ap = grad_gamma = None
        empty = self._allocator(stream, grad_logits, weights, logits, hidden, gamma, grad_hidden)
        if logits is not None:
            if logits.dim() == 1:
                logits = logits.unsqueeze(0)
            lp = self._check(logits, "logits", torch.float32, (b, self.n_rows))
        if gamma is not None:
            if hidden is None:
                raise ValueError("hidden: needed with gamma")
            if hidden.dim() == 1:
                hidden = hidden.unsqueeze(0)
            hp = self._check(hidden, "hidden", torch.float32, (b, self.k))
            gp = self._check(gamma, "gamma", torch.float32, (self.k,))
            grad_gamma = empty((self.k,), dtype=torch.float32, device=grad_logits.device)
            ap = grad_gamma.data_ptr()
        if grad_hidden is None:
            grad_hidden = empty((b, self.k), dtype=torch.float32, device=grad_logits.device)
        op = self._check(grad_hidden, "grad_hidden", torch.float32, (b, self.k))
        st = load_library().muse_lmhead_backward(self.handle, tp, lp, hp, b, gp, eps, wp, scale, cap, op, ap,
                                                 self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_backward")
        return grad_hidden, grad_gamma

    def _sampling(self, n, temperature, top_k, top_p, min_p):
        """MuseSampling of settings that are numbers or tensors [n]."""
        import torch
        how = MuseSampling(1.0, 0, 1.0, 0.0)
        if isinstance(temperature, torch.Tensor):
            how.temperatures = self._check(temperature, "temperature", torch.float32, (n,))
        else:
            how.temperature = temperature
            if how.temperature == 0.0 and temperature != 0:
                raise ValueError(f"temperature: {temperature}, need 2^-20 .. 2^20, or 0")
        if isinstance(top_k, torch.Tensor):
            how.top_ks = self._check(top_k, "top_k", torch.int32, (n,))
        else:
            how.top_k = max(0, min(int(top_k), self.n_rows))
        if isinstance(top_p, torch.Tensor):
            how.top_ps = self._check(top_p, "top_p", torch.float32, (n,))
        else:
            how.top_p = top_p
        if isinstance(min_p, torch.Tensor):
            how.min_ps = self._check(min_p, "min_p", torch.float32, (n,))
        else:
            how.min_p = min_p
        return how

    def sample(self, logits, uniforms, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
        """(tokens [n] int32, logprobs [n] f32): the next token of each row, drawn from uniforms [n] f32 in 0..1.

        logits [n, n_rows] as for score.  temperature (0: the first of the
        largest logits), top_k (0: off), top_p (1: off) and min_p (0: off) are
        numbers, or tensors [n] on the device (f32, top_k int32) with a setting
        for each row.  The filters apply in this order; logprobs are those that
        the tokens were drawn with, over what the filters left.  A row of
        nothing but masked logits has token -1.  See muse_lmhead_sample in the C header."""
        import torch
        if logits.dim() == 1:
            logits = logits.unsqueeze(0)
        ptr, dtype, n, ld = self._rows(logits, "logits")
        up = self._check(uniforms, "uniforms", torch.float32, (n,))
        how = self._sampling(n, temperature, top_k, top_p, min_p)
        empty = torch.empty if stream is None else self._allocator(
            stream, logits, uniforms, *(s for s in (temperature, top_k, top_p, min_p) if isinstance(s, torch.Tensor)))
        tokens = empty((n,), dtype=torch.int32, device=logits.device)
        logprobs = empty((n,), dtype=torch.float32, device=logits.device)
        st = load_library().muse_lmhead_sample(self.handle, ptr, dtype, n, ld, how, up, tokens.data_ptr(),
                                               logprobs.data_ptr(), self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_sample")
        return tokens, logprobs

    def forward_sample(self, hidden, weights, uniforms, gamma=None, eps: float = RMS_EPS, scale: float = LOGIT_SCALE,
                       cap: float = SOFTCAP, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, logits=None, stream=None):
        """(logits [B, n_rows], tokens [B], logprobs [B]): the forward, and the next tokens drawn from its logits."""
        import torch
        if hidden.dim() == 1:
            hidden = hidden.unsqueeze(0)
        b = hidden.shape[0]
        hp = self._check(hidden, "hidden", torch.float32, (b, self.k))
        wp = self._check(weights, "weights", torch.uint8)
        if weights.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
            raise ValueError("weights: wrong number of bytes for this handle")
        gp = None if gamma is None else self._check(gamma, "gamma", torch.float32, (self.k,))
        up = self._check(uniforms, "uniforms", torch.float32, (b,))
        how = self._sampling(b, temperature, top_k, top_p, min_p)
        empty = self._allocator(stream, hidden, weights, gamma, logits, uniforms,
                                *(s for s in (temperature, top_k, top_p, min_p) if isinstance(s, torch.Tensor)))
        if logits is None:
            logits = empty((b, self.n_rows), dtype=torch.float32, device=hidden.device)
        lp = self._check(logits, "logits", torch.float32, (b, self.n_rows))
        tokens = empty((b,), dtype=torch.int32, device=hidden.device)
        logprobs = empty((b,), dtype=torch.float32, device=hidden.device)
        st = load_library().muse_lmhead_forward_sample(self.handle, hp, b, gp, float(eps), wp, float(scale), float(cap),
                                                       lp, how, up, tokens.data_ptr(), logprobs.data_ptr(),
                                                       self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_forward_sample")
        return logits, tokens, logprobs

    def embed(self, tokens, table, scale: float = 1.0, dtype=None, out=None, stream=None):
        """out [n, k] = scale * table[tokens]: rows of a token table for tokens [n] int32.

        table: the blocks of an [n_rows, k] matrix in the handle's format
        (uint8, a tied head's own weights among others), or [n_rows, k] f32,
        f16 or bf16, contiguous rows any distance apart.  A token outside
        0..n_rows-1 marks a padded position: a row of zeros.  out (rows any
        distance apart) is made when not given, in `dtype`: the dense table's,
        or f32.  See muse_lmhead_embed in the C header."""
        import torch
        n = tokens.numel()
        tp = self._check(tokens, "tokens", torch.int32, (n,))
        if table.dtype == torch.uint8:
            wp, kind, ld = self._check(table, "table", torch.uint8), MUSE_DTYPE_BLOCKS, 0
            if table.numel() != self.n_rows * (self.k // 256) * self.block_bytes:
                raise ValueError("table: wrong number of bytes for this handle")
        else:
            wp, kind, rows, ld = self._rows(table, "table", self.k)
            if rows != self.n_rows:
                raise ValueError(f"table: shape {tuple(table.shape)}, need [{self.n_rows}, {self.k}]")
        if out is None:
            if dtype is None:
                dtype = torch.float32 if kind == MUSE_DTYPE_BLOCKS else table.dtype
            empty = torch.empty if stream is None else self._allocator(stream, tokens, table)
            out = empty((n, self.k), dtype=dtype, device=tokens.device)
        else:
            self._allocator(stream, tokens, table, out)
            if dtype is not None and out.dtype != dtype:
                raise ValueError("out: not of the given dtype")
        op, otype, rows, old = self._rows(out, "out", self.k)
        if rows != n:
            raise ValueError(f"out: shape {tuple(out.shape)}, need [{n}, {self.k}]")
        st = load_library().muse_lmhead_embed(self.handle, wp, kind, ld, tp, n, scale, op, otype, old,
                                              self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_embed")
        return out

    def embed_backward(self, grad, tokens, scale: float = 1.0, dtype=None, grad_table=None, accumulate: bool = False,
                       stream=None):
        """grad_table [n_rows, k]: the gradient by a dense table from grad [n, k] by embed's rows.

        grad: f32, f16 or bf16, contiguous rows any distance apart; tokens [n]
        int32 and scale as given to embed.  grad_table (rows any distance
        apart) is made when not given, in `dtype` or grad's; accumulate adds to
        the one that is given, and then only the rows of tokens that occur are
        read and written.  The same inputs give the same bits.  See
        muse_lmhead_embed_backward in the C header."""
        import torch
        gp, gtype, n, gld = self._rows(grad, "grad", self.k)
        tp = self._check(tokens, "tokens", torch.int32, (n,))
        if grad_table is None:
            if accumulate:
                raise ValueError("grad_table: needed to accumulate into")
            empty = self._allocator(stream, grad, tokens)
            grad_table = empty((self.n_rows, self.k), dtype=grad.dtype if dtype is None else dtype, device=grad.device)
        else:
            empty = self._allocator(stream, grad, tokens, grad_table)
            if dtype is not None and grad_table.dtype != dtype:
                raise ValueError("grad_table: not of the given dtype")
        op, otype, rows, old = self._rows(grad_table, "grad_table", self.k)
        if rows != self.n_rows:
            raise ValueError(f"grad_table: shape {tuple(grad_table.shape)}, need [{self.n_rows}, {self.k}]")
        need = muse_lmhead_embed_backward_workspace(self.handle, n)
        work = empty((need,), dtype=torch.uint8, device=grad.device)
        st = load_library().muse_lmhead_embed_backward(self.handle, gp, gtype, gld, tp, n, scale, op, otype, old,
                                                       1 if accumulate else 0, work.data_ptr(), need,
                                                       self._stream(stream))
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_embed_backward")
        return grad_table

    def set_argmax_key(self, key: str) -> None:
        """"capped" (the returned logit; the default) or "precap" (scale * raw, before the cap)."""
        if key not in ARGMAX_KEYS:
            raise ValueError(f"argmax key: one of {sorted(ARGMAX_KEYS)}")
        st = muse_lmhead_set_argmax_key(self.handle, ARGMAX_KEYS[key])
        if st != MUSE_OK:
            raise MuseError(st, "muse_lmhead_set_argmax_key")

    def path_name(self, batch: int) -> str | None:
        return muse_lmhead_path_name(self.handle, batch)

    def launches_per_forward(self, batch: int, with_norm: bool) -> int:
        return muse_lmhead_launches_per_forward(self.handle, batch, with_norm)

    def device_status(self) -> int:
        return muse_lmhead_device_status(self.handle)
