"""Python binding of librlk (argument marshalling only).

Every step of the computation runs in the CUDA kernels of ``librlk.so``; this
module only checks tensor placement, allocates outputs with PyTorch and passes
raw pointers plus the current CUDA stream through the C ABI declared in
``include/rlk.h``.  There is no CPU fallback: if the library is missing or the
tensors are not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librlk.so")

RLK_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace",
                4: "CUDA error", 5: "timeout", 6: "bad input"}
STATUS_BAD_TOKEN_ID = 0x1
STATUS_NONFINITE = 0x2
OP_LOGPROB_ENTROPY, OP_GRPO_LOSS, OP_LMHEAD, OP_LMHEAD_BWD, OP_LMHEAD_TOPP = 0, 1, 2, 3, 4
OP_CANONICAL = 5
OP_CANONICAL_TOPP = 6
OP_NORM_BWD = 7
OP_PREFERENCE_LOSS = 8
OP_LINEAR, OP_LINEAR_BWD = 9, 10
OP_GATED_LINEAR, OP_GATED_LINEAR_BWD = 11, 12
OP_ORTHOGONALISE = 13
ACT_NONE, ACT_GELU, ACT_SILU, ACT_RELU = 0, 1, 2, 3
PREF_SIGMOID, PREF_IPO, PREF_HINGE = 0, 1, 2
PREF_NSTATS = 6
MAX_TOKENS, MAX_ALTERNATIVES = 1024, 128   # of a row in token_logprobs
PREF_STAT_NAMES = ("loss", "pairs", "accuracy", "margin", "chosen", "rejected")
NORM_LAYER, NORM_RMS = 0, 1
CHECKPOINT_BLOCK = 32   # columns that share one checkpoint scale
SHARD_COUNTS_BYTES = 8224   # rlk_shard_counts: one row's window counts of one shard
CANONICAL_TP, CANONICAL_VOCAB = 8, 152576
SHARD_PARTIAL_WORDS = 8   # rlk_shard_partial: 32 bytes per (shard, row)
AGG_TOKEN_MEAN, AGG_SEQ_MEAN_TOKEN_MEAN, AGG_PROMPT_MEAN = 0, 1, 2
LOSS_DAPO, LOSS_IPO, LOSS_ICEPOP = 0, 1, 2
IS_NONE, IS_TIS, IS_MIS = 0, 1, 2
BASELINE_MEAN, BASELINE_LENGTH_WEIGHTED = 0, 1
NSTATS_POLICY = 9
STAT_MASK_DROPPED = 8
NSTATS = 8
class LossConfig(ctypes.Structure):
    """rlk_loss_config."""
    _fields_ = [("type", ctypes.c_int), ("eps_low", ctypes.c_float), ("eps_high", ctypes.c_float),
                ("ipo_eps", ctypes.c_float), ("band_low", ctypes.c_float),
                ("band_high", ctypes.c_float), ("is_method", ctypes.c_int),
                ("is_cap", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("baseline", ctypes.c_int), ("agg", ctypes.c_int)]


class PrefConfig(ctypes.Structure):
    """rlk_pref_config."""
    _fields_ = [("type", ctypes.c_int), ("beta", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("margin", ctypes.c_float),
                ("length_normalise", ctypes.c_int)]


class CheckpointBuffers(ctypes.Structure):
    """rlk_checkpoint."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


STAT_NAMES = ("loss", "tokens", "clip_low_frac", "clip_high_frac", "tis_mean",
              "tis_capped_frac", "k3_mean", "pg_mean")
EXPORTS = ("rlk_version", "rlk_status_string", "rlk_workspace_size", "rlk_logprob_entropy",
           "rlk_logprob_entropy_fwd", "rlk_logprob_entropy_bwd", "rlk_logprob_entropy_rows",
           "rlk_logprob_entropy_support", "rlk_logprob_entropy_support_backward",
           "rlk_grpo_loss", "rlk_policy_loss", "rlk_lmhead_logprob", "rlk_lmhead_logprob_fwd",
           "rlk_lmhead_logprob_bwd", "rlk_shard_partials", "rlk_shard_combine",
           "rlk_shard_partials_support",
           "rlk_logprob_entropy_canonical", "rlk_sample_top_p",
           "rlk_shard_window_counts", "rlk_shard_combine_topp",
           "rlk_logprob_entropy_canonical_topp",
           "rlk_grpo_loss_noalloc", "rlk_checkpoint_pack", "rlk_checkpoint_unpack",
           "rlk_norm_fwd", "rlk_norm_bwd", "rlk_preference_loss", "rlk_linear_fwd",
           "rlk_linear_bwd", "rlk_token_logprobs_fwd", "rlk_token_logprobs_bwd",
           "rlk_gated_linear_fwd", "rlk_gated_linear_bwd", "rlk_orthogonalise")
NOALLOC_MAX_SEQ = 16384
DEBUG_EXPORTS = ("rlk_lmhead_logits_debug", "rlk_debug_inject_launch_failures",
                 "rlk_debug_set_wait_limit", "rlk_debug_withhold_copy",
                 "rlk_debug_set_sampler_mode")
STATUS_TIMEOUT = 0x4
STATUS_BAD_SUPPORT = 0x8
STATUS_NO_STATE = 0x10
STATUS_BAD_PARAM = 0x20
STATUS_UNRESOLVED = 0x40
ROW_STATE_WORDS = 8   # rlk_row_state: 32 bytes per row

_lock = threading.Lock()
_lib = None


class RlkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)} ({code})")
        self.code = code


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


def load(path: str | None = None):
    """Load librlk.so (built in-tree by ``build()``) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it first (entropy_logits_bf16_gb300.build())")
        lib = ctypes.CDLL(p)
        i64, i32, f32, vp, sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                 ctypes.c_void_p, ctypes.c_size_t)
        lib.rlk_version.restype = ctypes.c_int
        lib.rlk_status_string.argtypes = [ctypes.c_int]
        lib.rlk_status_string.restype = ctypes.c_char_p
        lib.rlk_workspace_size.argtypes = [ctypes.c_int, i64, i64, i64]
        lib.rlk_workspace_size.restype = sz
        lib.rlk_logprob_entropy.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32, f32, vp,
                                            vp, vp, vp, vp, sz, vp]
        lib.rlk_logprob_entropy.restype = ctypes.c_int
        lib.rlk_logprob_entropy_fwd.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32, f32, vp,
                                                vp, vp, vp, vp, vp]
        lib.rlk_logprob_entropy_fwd.restype = ctypes.c_int
        lib.rlk_logprob_entropy_rows.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, vp, vp, vp,
                                                 vp, vp, vp, vp, vp]
        lib.rlk_logprob_entropy_rows.restype = ctypes.c_int
        lib.rlk_logprob_entropy_bwd.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32, vp, vp,
                                                vp, vp, ctypes.c_int, i64, vp, vp]
        lib.rlk_logprob_entropy_bwd.restype = ctypes.c_int
        lib.rlk_logprob_entropy_support.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32, vp,
                                                    vp, vp, vp, vp, vp]
        lib.rlk_logprob_entropy_support.restype = ctypes.c_int
        lib.rlk_logprob_entropy_support_backward.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp,
                                                             f32, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logprob_entropy_support_backward.restype = ctypes.c_int
        lib.rlk_policy_loss.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i64,
                                        ctypes.POINTER(LossConfig), vp, vp, vp, vp, sz, vp]
        lib.rlk_policy_loss.restype = ctypes.c_int
        lib.rlk_grpo_loss.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, f32, f32, f32,
                                      f32, ctypes.c_int, vp, vp, vp, vp, sz, vp]
        lib.rlk_grpo_loss.restype = ctypes.c_int
        lib.rlk_lmhead_logprob.argtypes = [vp, vp, i64, i64, i64, vp, f32, f32, vp, vp, vp, vp,
                                           sz, vp]
        lib.rlk_lmhead_logprob.restype = ctypes.c_int
        lib.rlk_sample_top_p.argtypes = [vp, ctypes.c_int, i64, i64, i64, f32, vp, vp, vp, vp, vp]
        lib.rlk_sample_top_p.restype = ctypes.c_int
        lib.rlk_debug_inject_launch_failures.argtypes = [ctypes.c_int]
        lib.rlk_debug_inject_launch_failures.restype = ctypes.c_int
        lib.rlk_debug_set_wait_limit.argtypes = [ctypes.c_longlong]
        lib.rlk_debug_set_wait_limit.restype = ctypes.c_longlong
        lib.rlk_debug_withhold_copy.argtypes = [ctypes.c_longlong]
        lib.rlk_debug_withhold_copy.restype = ctypes.c_int
        lib.rlk_debug_set_sampler_mode.argtypes = [ctypes.c_int]
        lib.rlk_debug_set_sampler_mode.restype = ctypes.c_int
        lib.rlk_shard_partials.argtypes = [vp, ctypes.c_int, i64, i64, i64, i64, i64, i32, vp, f32,
                                           vp, vp]
        lib.rlk_shard_partials.restype = ctypes.c_int
        lib.rlk_shard_partials_support.argtypes = [vp, ctypes.c_int, i64, i64, i64, i64, i64, i32,
                                                   vp, f32, vp, vp, vp, vp]
        lib.rlk_shard_partials_support.restype = ctypes.c_int
        lib.rlk_shard_combine.argtypes = [vp, i32, i64, i64, i64, vp, f32, vp, vp, vp, vp]
        lib.rlk_shard_combine.restype = ctypes.c_int
        lib.rlk_logprob_entropy_canonical.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32, i32,
                                                      i64, vp, vp, vp, vp, sz, vp]
        lib.rlk_logprob_entropy_canonical.restype = ctypes.c_int
        lib.rlk_shard_window_counts.argtypes = [vp, ctypes.c_int, i64, i64, i64, i64, i64, i32, vp,
                                                f32, f32, vp, i32, vp, vp]
        lib.rlk_shard_window_counts.restype = ctypes.c_int
        lib.rlk_shard_combine_topp.argtypes = [vp, vp, i32, i64, i64, i64, vp, f32, f32, vp, vp,
                                               vp, vp, vp]
        lib.rlk_shard_combine_topp.restype = ctypes.c_int
        lib.rlk_logprob_entropy_canonical_topp.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, f32,
                                                           f32, i32, i64, vp, vp, vp, vp, vp, sz,
                                                           vp]
        lib.rlk_logprob_entropy_canonical_topp.restype = ctypes.c_int
        lib.rlk_lmhead_logprob_fwd.argtypes = [vp, vp, i64, i64, i64, vp, f32, f32, vp, vp, vp,
                                               vp, vp, sz, vp]
        lib.rlk_lmhead_logprob_fwd.restype = ctypes.c_int
        lib.rlk_lmhead_logprob_bwd.argtypes = [vp, vp, i64, i64, i64, vp, f32, vp, vp, vp, vp, vp,
                                               vp, ctypes.c_int, vp, sz, vp]
        lib.rlk_lmhead_logprob_bwd.restype = ctypes.c_int
        lib.rlk_lmhead_logits_debug.argtypes = [vp, vp, i64, i64, i64, vp, f32, vp, vp, vp, vp,
                                                vp, sz, vp]
        lib.rlk_lmhead_logits_debug.restype = ctypes.c_int
        lib.rlk_grpo_loss_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, f32, f32,
                                              f32, f32, ctypes.c_int, vp, vp, vp, vp]
        lib.rlk_grpo_loss_noalloc.restype = ctypes.c_int
        ck = ctypes.POINTER(CheckpointBuffers)
        lib.rlk_checkpoint_pack.argtypes = [vp, ctypes.c_int, i64, i64, i64, ck, vp, vp]
        lib.rlk_checkpoint_pack.restype = ctypes.c_int
        lib.rlk_checkpoint_unpack.argtypes = [ck, i64, i64, vp, ctypes.c_int, i64, vp]
        lib.rlk_checkpoint_unpack.restype = ctypes.c_int
        lib.rlk_norm_fwd.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, vp, ctypes.c_int,
                                     ctypes.c_int, f32, vp, ctypes.c_int, i64, vp, vp, ck, vp, vp]
        lib.rlk_norm_fwd.restype = ctypes.c_int
        lib.rlk_norm_bwd.argtypes = [vp, ctypes.c_int, i64, vp, ctypes.c_int, i64, ck, i64, i64, vp,
                                     ctypes.c_int, ctypes.c_int, vp, vp, vp, ctypes.c_int, i64, vp,
                                     vp, ctypes.c_int, vp, sz, vp]
        lib.rlk_norm_bwd.restype = ctypes.c_int
        lib.rlk_preference_loss.argtypes = [vp, vp, vp, vp, i32, i64, ctypes.POINTER(PrefConfig), vp,
                                            vp, vp, vp, vp, sz, vp]
        lib.rlk_preference_loss.restype = ctypes.c_int
        lib.rlk_linear_fwd.argtypes = [vp, i64, vp, i64, vp, ctypes.c_int, vp, i64, i64, i64, i64,
                                       ctypes.c_int, vp, ctypes.c_int, i64, vp, i64, vp, sz, vp]
        lib.rlk_linear_fwd.restype = ctypes.c_int
        lib.rlk_linear_bwd.argtypes = [vp, i64, vp, i64, ck, vp, i64, vp, i64, i64, i64, i64,
                                       ctypes.c_int, vp, ctypes.c_int, i64, vp, ctypes.c_int, i64, vp,
                                       ctypes.c_int, vp, sz, vp]
        lib.rlk_linear_bwd.restype = ctypes.c_int
        lib.rlk_token_logprobs_fwd.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, f32, i32, vp, vp,
                                               vp, vp, vp, vp, vp]
        lib.rlk_token_logprobs_fwd.restype = ctypes.c_int
        lib.rlk_token_logprobs_bwd.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, f32, vp, vp, vp,
                                               vp, i32, vp, vp, ctypes.c_int, i64, vp, vp]
        lib.rlk_token_logprobs_bwd.restype = ctypes.c_int
        lib.rlk_gated_linear_fwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, ctypes.c_int, i64, i64, i64,
                                             ctypes.c_int, vp, ctypes.c_int, i64, vp, vp, i64, vp, sz, vp]
        lib.rlk_gated_linear_fwd.restype = ctypes.c_int
        lib.rlk_gated_linear_bwd.argtypes = [vp, i64, vp, i64, ck, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64,
                                             i64, ctypes.c_int, vp, ctypes.c_int, i64, vp, i64, vp, i64,
                                             ctypes.c_int, vp, vp, ctypes.c_int, vp, sz, vp]
        lib.rlk_gated_linear_bwd.restype = ctypes.c_int
        lib.rlk_orthogonalise.argtypes = [vp, ctypes.c_int, i64, i64, i64, i64, i64, i32, vp, f32, vp, i64, i64,
                                          vp, vp, sz, vp]
        lib.rlk_orthogonalise.restype = ctypes.c_int
        _lib = lib
        return lib


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a torch.cuda.Stream around it (0.1 us instead of
# 2), where this PyTorch has it: the name is private.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    """The current stream of the device as a raw handle."""
    index = torch.cuda.current_device() if device.index is None else device.index
    return torch.cuda.current_stream(index).cuda_stream if _raw_stream is None else _raw_stream(index)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("librlk operates on CUDA tensors only")


def _check(fn, code):
    if code != RLK_OK:
        raise RlkError(fn, code)


def workspace_size(op: int, T: int, V: int, H: int = 0) -> int:
    return int(load().rlk_workspace_size(op, T, V, H))


def _logits_dtype(logits):
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit stride along the vocabulary")
    dt = {torch.bfloat16: 0, torch.float32: 1}.get(logits.dtype)
    if dt is None:
        raise ValueError("logits must be bf16 or fp32")
    return dt


def new_row_state(T: int, device) -> torch.Tensor:
    """Room for the per-row state the forward saves for the backward
    (rlk_row_state[T], 32 bytes a row)."""
    return torch.empty((T, ROW_STATE_WORDS), dtype=torch.int32, device=device)


def logprob_entropy(logits: torch.Tensor, token_ids: torch.Tensor, temperature: float,
                    top_p: float, *, out_logprob=None, out_entropy=None,
                    return_nucleus_size: bool = False, status_word: torch.Tensor | None = None,
                    row_state: torch.Tensor | None = None):
    """Top-p log-probability of the selected token and entropy of the retained set.

    logits: CUDA [T, V] bf16 or fp32 (rows may be strided, unit stride along V);
    token_ids: CUDA int32 [T].  Returns (logprob, entropy) fp32 [T], plus the
    nucleus sizes int32 [T] when ``return_nucleus_size``.  ``status_word`` (CUDA
    uint32/int32 [1]) receives the STATUS_* bits of bad rows.  ``row_state``
    (from ``new_row_state``) receives what ``logprob_entropy_backward`` needs.
    """
    lib = load()
    _need_cuda(logits, token_ids)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit stride along the vocabulary")
    if logits.dtype == torch.bfloat16:
        dt = 0
    elif logits.dtype == torch.float32:
        dt = 1
    else:
        raise ValueError("logits must be bf16 or fp32")
    if token_ids.dtype != torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32")
    T, V = logits.shape
    ld = logits.stride(0) if T > 1 else V
    dev = logits.device
    lp = out_logprob if out_logprob is not None else torch.empty(T, device=dev, dtype=torch.float32)
    ent = out_entropy if out_entropy is not None else torch.empty(T, device=dev, dtype=torch.float32)
    ks = torch.empty(T, device=dev, dtype=torch.int32) if return_nucleus_size else None
    if row_state is not None:
        _need_cuda(row_state)
        if (row_state.dtype != torch.int32 or not row_state.is_contiguous()
                or row_state.numel() != T * ROW_STATE_WORDS):
            raise ValueError("row_state must come from new_row_state(T)")
        code = lib.rlk_logprob_entropy_fwd(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                           float(temperature), float(top_p), _ptr(lp), _ptr(ent),
                                           _ptr(ks), _ptr(row_state), _ptr(status_word),
                                           _stream(dev))
        _check("rlk_logprob_entropy_fwd", code)
    else:
        code = lib.rlk_logprob_entropy(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                       float(temperature), float(top_p), _ptr(lp), _ptr(ent),
                                       _ptr(ks), _ptr(status_word), None, 0, _stream(dev))
        _check("rlk_logprob_entropy", code)
    return (lp, ent, ks) if return_nucleus_size else (lp, ent)


def logprob_entropy_rows(logits: torch.Tensor, token_ids: torch.Tensor, temperatures: torch.Tensor,
                        top_ps: torch.Tensor, *, return_nucleus_size: bool = False,
                        status_word=None, row_state=None):
    """``logprob_entropy`` with per-row sampling parameters (CUDA fp32 [T]
    each).  ``row_state`` records each row's temperature for the backward and
    the sampler."""
    lib = load()
    _need_cuda(logits, token_ids, temperatures, top_ps, row_state)
    dt = _logits_dtype(logits)
    T, V = logits.shape
    for t in (temperatures, top_ps):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != T:
            raise ValueError("temperatures and top_ps must be contiguous fp32 [T]")
    if token_ids.dtype != torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32")
    if row_state is not None and (row_state.dtype != torch.int32 or not row_state.is_contiguous()
                                  or row_state.numel() != T * ROW_STATE_WORDS):
        raise ValueError("row_state must come from new_row_state(T)")
    ld = logits.stride(0) if T > 1 else V
    dev = logits.device
    lp = torch.empty(T, device=dev, dtype=torch.float32)
    ent = torch.empty(T, device=dev, dtype=torch.float32)
    ks = torch.empty(T, device=dev, dtype=torch.int32) if return_nucleus_size else None
    code = lib.rlk_logprob_entropy_rows(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                        _ptr(temperatures), _ptr(top_ps), _ptr(lp), _ptr(ent),
                                        _ptr(ks), _ptr(row_state), _ptr(status_word), _stream(dev))
    _check("rlk_logprob_entropy_rows", code)
    return (lp, ent, ks) if return_nucleus_size else (lp, ent)


def logprob_entropy_backward(logits: torch.Tensor, token_ids: torch.Tensor, temperature: float,
                             row_state: torch.Tensor, grad_logprob=None, grad_entropy=None, *,
                             out=None, grad_dtype=None, status_word=None):
    """dL/dlogits [T, V] for L = sum grad_logprob * logprob + grad_entropy * H,
    each row's retained set (saved in ``row_state`` by the forward) held fixed;
    zero outside the set.  ``grad_dtype`` (bf16 or fp32) defaults to the
    logits' dtype; ``out`` may be a strided [T, V] tensor of that dtype."""
    lib = load()
    _need_cuda(logits, token_ids, row_state, grad_logprob, grad_entropy, out)
    dt = _logits_dtype(logits)
    if token_ids.dtype != torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32")
    T, V = logits.shape
    if (row_state.dtype != torch.int32 or not row_state.is_contiguous()
            or row_state.numel() != T * ROW_STATE_WORDS):
        raise ValueError("row_state must come from new_row_state(T)")
    for g in (grad_logprob, grad_entropy):
        if g is not None and (g.dtype != torch.float32 or not g.is_contiguous() or g.numel() != T):
            raise ValueError("gradients must be contiguous fp32 [T]")
    gdt = grad_dtype or (out.dtype if out is not None else logits.dtype)
    if out is None:
        out = torch.empty((T, V), device=logits.device, dtype=gdt)
    if out.dtype != gdt or out.shape != (T, V) or out.stride(1) != 1:
        raise ValueError("out must be [T, V] of grad_dtype with unit stride along V")
    gd = {torch.bfloat16: 0, torch.float32: 1}.get(gdt)
    if gd is None:
        raise ValueError("grad_dtype must be bf16 or fp32")
    ld = logits.stride(0) if T > 1 else V
    ldg = out.stride(0) if T > 1 else V
    code = lib.rlk_logprob_entropy_bwd(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                       float(temperature), _ptr(row_state), _ptr(grad_logprob),
                                       _ptr(grad_entropy), _ptr(out), gd, ldg, _ptr(status_word),
                                       _stream(logits.device))
    _check("rlk_logprob_entropy_bwd", code)
    return out


class _LogprobEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token_ids, temperature, top_p):
        state = new_row_state(logits.shape[0], logits.device)
        lp, ent = logprob_entropy(logits, token_ids, temperature, top_p, row_state=state)
        ctx.save_for_backward(logits, token_ids, state)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return lp, ent

    @staticmethod
    @once_differentiable
    def backward(ctx, g_lp, g_ent):
        logits, token_ids, state = ctx.saved_tensors
        if g_lp is None and g_ent is None:
            return None, None, None, None
        g = logprob_entropy_backward(
            logits, token_ids, ctx.temperature, state,
            None if g_lp is None else g_lp.float().contiguous(),
            None if g_ent is None else g_ent.float().contiguous())
        return g, None, None, None


def logprob_entropy_autograd(logits: torch.Tensor, token_ids: torch.Tensor, temperature: float,
                             top_p: float):
    """``logprob_entropy`` as a differentiable op: (logprob, entropy) whose
    backward is ``rlk_logprob_entropy_bwd`` (the retained sets held fixed)."""
    return _LogprobEntropy.apply(logits, token_ids, temperature, top_p)


def logprob_entropy_support(logits: torch.Tensor, token_ids: torch.Tensor, temperature: float,
                            support_offsets: torch.Tensor, support_ids: torch.Tensor, *,
                            out_logprob=None, out_entropy=None, status_word=None):
    """Log-probability of the selected token and entropy over a retained set
    supplied by the sampler: row t keeps the ids
    support_ids[support_offsets[t]:support_offsets[t+1]] (CUDA int64 offsets
    [T+1], int32 ids).  Returns (logprob, entropy) fp32 [T]."""
    lib = load()
    _need_cuda(logits, token_ids, support_offsets, support_ids)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit stride along the vocabulary")
    if logits.dtype == torch.bfloat16:
        dt = 0
    elif logits.dtype == torch.float32:
        dt = 1
    else:
        raise ValueError("logits must be bf16 or fp32")
    if token_ids.dtype != torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32")
    if support_offsets.dtype != torch.int64 or not support_offsets.is_contiguous():
        raise ValueError("support_offsets must be contiguous int64")
    if support_ids.dtype != torch.int32 or not support_ids.is_contiguous():
        raise ValueError("support_ids must be contiguous int32")
    T, V = logits.shape
    if support_offsets.numel() != T + 1:
        raise ValueError("support_offsets must have T + 1 entries")
    ld = logits.stride(0) if T > 1 else V
    dev = logits.device
    lp = out_logprob if out_logprob is not None else torch.empty(T, device=dev, dtype=torch.float32)
    ent = out_entropy if out_entropy is not None else torch.empty(T, device=dev, dtype=torch.float32)
    code = lib.rlk_logprob_entropy_support(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                           float(temperature), _ptr(support_offsets),
                                           _ptr(support_ids), _ptr(lp), _ptr(ent),
                                           _ptr(status_word), _stream(dev))
    _check("rlk_logprob_entropy_support", code)
    return lp, ent


def logprob_entropy_support_backward(logits: torch.Tensor, token_ids: torch.Tensor,
                                     temperature: float, support_offsets: torch.Tensor,
                                     support_ids: torch.Tensor, grad_logprob=None,
                                     grad_entropy=None, *, out=None, status_word=None):
    """dL/dz for every listed id (aligned with ``support_ids``; the retained
    sets held fixed) for L = sum grad_logprob * logprob + grad_entropy * H.
    Returns a CUDA fp32 tensor shaped like ``support_ids``."""
    lib = load()
    _need_cuda(logits, token_ids, support_offsets, support_ids, grad_logprob, grad_entropy)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D with unit stride along the vocabulary")
    dt = {torch.bfloat16: 0, torch.float32: 1}.get(logits.dtype)
    if dt is None:
        raise ValueError("logits must be bf16 or fp32")
    for t, want in ((token_ids, torch.int32), (support_offsets, torch.int64),
                    (support_ids, torch.int32)):
        if t.dtype != want or not t.is_contiguous():
            raise ValueError("token_ids int32, support_offsets int64 and support_ids int32, contiguous")
    for g in (grad_logprob, grad_entropy):
        if g is not None and (g.dtype != torch.float32 or not g.is_contiguous()):
            raise ValueError("gradients must be contiguous fp32")
    T, V = logits.shape
    ld = logits.stride(0) if T > 1 else V
    grad = out if out is not None else torch.empty(support_ids.shape, device=logits.device,
                                                   dtype=torch.float32)
    code = lib.rlk_logprob_entropy_support_backward(
        _ptr(logits), dt, T, V, ld, _ptr(token_ids), float(temperature), _ptr(support_offsets),
        _ptr(support_ids), _ptr(grad_logprob), _ptr(grad_entropy), _ptr(grad), _ptr(status_word),
        _stream(logits.device))
    _check("rlk_logprob_entropy_support_backward", code)
    return grad


def grpo_loss(logp_new, logp_old, logp_rollout, logp_ref, rewards, seq_offsets, group_size, *,
              loss_mask=None, eps_low=0.2, eps_high=0.28, tis_cap=2.0, kl_coef=0.01,
              agg=AGG_TOKEN_MEAN, want_grad=True, want_stats=True, workspace=None):
    """GRPO/DAPO loss with TIS and k3 KL.  Returns (loss[1], grad[T] or None,
    stats[NSTATS] or None), all CUDA fp32 tensors."""
    lib = load()
    _need_cuda(logp_new, logp_old, logp_rollout, logp_ref, rewards, seq_offsets, loss_mask)
    for t in (logp_new, logp_old, logp_rollout, logp_ref, rewards):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("log-probs and rewards must be contiguous fp32")
    if seq_offsets.dtype != torch.int32:
        raise ValueError("seq_offsets must be int32")
    if loss_mask is not None and loss_mask.dtype != torch.uint8:
        raise ValueError("loss_mask must be uint8")
    n_seq = seq_offsets.numel() - 1
    n_tok = logp_new.numel()
    dev = logp_new.device
    need = int(lib.rlk_workspace_size(OP_GRPO_LOSS, n_tok, n_seq, 0))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    loss = torch.empty(1, device=dev, dtype=torch.float32)
    grad = torch.empty(n_tok, device=dev, dtype=torch.float32) if want_grad else None
    stats = torch.empty(NSTATS, device=dev, dtype=torch.float32) if want_stats else None
    code = lib.rlk_grpo_loss(_ptr(logp_new), _ptr(logp_old), _ptr(logp_rollout), _ptr(logp_ref),
                             _ptr(loss_mask), _ptr(rewards), _ptr(seq_offsets), n_seq,
                             int(group_size), n_tok, float(eps_low), float(eps_high),
                             float(tis_cap), float(kl_coef), int(agg), _ptr(loss), _ptr(grad),
                             _ptr(stats), _ptr(workspace), workspace.numel(), _stream(dev))
    _check("rlk_grpo_loss", code)
    return loss, grad, stats


def policy_loss(logp_new, logp_old, logp_rollout, logp_ref, rewards, seq_offsets, group_size, *,
                loss_mask=None, loss_type=LOSS_DAPO, eps_low=0.2, eps_high=0.28, ipo_eps=0.3,
                band_low=0.5, band_high=2.0, is_method=IS_TIS, is_cap=2.0, kl_coef=0.01,
                baseline=BASELINE_MEAN, agg=AGG_TOKEN_MEAN, want_grad=True, want_stats=True,
                workspace=None):
    """rlk_policy_loss: the GRPO/DAPO loss with the IPO / IcePop policy terms,
    none / TIS / MIS weights, a mean or length-weighted baseline and token /
    sequence / prompt aggregation.  Returns (loss[1], grad[T] or None,
    stats[NSTATS_POLICY] or None), CUDA fp32 tensors."""
    lib = load()
    _need_cuda(logp_new, logp_old, logp_rollout, logp_ref, rewards, seq_offsets, loss_mask)
    for t in (logp_new, logp_old, logp_rollout, logp_ref, rewards):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("log-probs and rewards must be contiguous fp32")
    if seq_offsets.dtype != torch.int32:
        raise ValueError("seq_offsets must be int32")
    if loss_mask is not None and loss_mask.dtype != torch.uint8:
        raise ValueError("loss_mask must be uint8")
    n_seq = seq_offsets.numel() - 1
    n_tok = logp_new.numel()
    dev = logp_new.device
    need = int(lib.rlk_workspace_size(OP_GRPO_LOSS, n_tok, n_seq, 0))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    cfg = LossConfig(int(loss_type), float(eps_low), float(eps_high), float(ipo_eps),
                     float(band_low), float(band_high), int(is_method), float(is_cap),
                     float(kl_coef), int(baseline), int(agg))
    loss = torch.empty(1, device=dev, dtype=torch.float32)
    grad = torch.empty(n_tok, device=dev, dtype=torch.float32) if want_grad else None
    stats = torch.empty(NSTATS_POLICY, device=dev, dtype=torch.float32) if want_stats else None
    code = lib.rlk_policy_loss(_ptr(logp_new), _ptr(logp_old), _ptr(logp_rollout),
                               _ptr(logp_ref), _ptr(loss_mask), _ptr(rewards), _ptr(seq_offsets),
                               n_seq, int(group_size), n_tok, ctypes.byref(cfg), _ptr(loss),
                               _ptr(grad), _ptr(stats), _ptr(workspace), workspace.numel(),
                               _stream(dev))
    _check("rlk_policy_loss", code)
    return loss, grad, stats


def lmhead_logprob(hidden, w_vocab, token_ids, temperature, top_p=1.0, *, status_word=None,
                   workspace=None, out_lse=None):
    """Fused LM-head log-probability and entropy.  At top_p = 1 the logits never
    reach memory; at top_p < 1 they are emitted as bf16 4096 rows at a time
    and scored by the top-p path.  ``out_lse`` (CUDA fp32 [T], top_p = 1)
    receives each row's log-normaliser for ``lmhead_backward``."""
    lib = load()
    _need_cuda(hidden, w_vocab, token_ids)
    if hidden.dtype != torch.bfloat16 or w_vocab.dtype != torch.bfloat16:
        raise ValueError("hidden and w_vocab must be bf16")
    if not (hidden.is_contiguous() and w_vocab.is_contiguous()):
        raise ValueError("hidden and w_vocab must be contiguous")
    T, H = hidden.shape
    V, H2 = w_vocab.shape
    if H != H2:
        raise ValueError("hidden and w_vocab disagree on H")
    dev = hidden.device
    need = int(lib.rlk_workspace_size(OP_LMHEAD if top_p == 1.0 else OP_LMHEAD_TOPP, T, V, H))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    lp = torch.empty(T, device=dev, dtype=torch.float32)
    ent = torch.empty(T, device=dev, dtype=torch.float32)
    wsb = 0 if workspace is None else workspace.numel()
    if out_lse is not None:
        _need_cuda(out_lse)
        if out_lse.dtype != torch.float32 or out_lse.numel() != T or not out_lse.is_contiguous():
            raise ValueError("out_lse must be contiguous fp32 [T]")
        code = lib.rlk_lmhead_logprob_fwd(_ptr(hidden), _ptr(w_vocab), T, H, V, _ptr(token_ids),
                                          float(temperature), float(top_p), _ptr(lp), _ptr(ent),
                                          _ptr(out_lse), _ptr(status_word), _ptr(workspace), wsb,
                                          _stream(dev))
        _check("rlk_lmhead_logprob_fwd", code)
    else:
        code = lib.rlk_lmhead_logprob(_ptr(hidden), _ptr(w_vocab), T, H, V, _ptr(token_ids),
                                      float(temperature), float(top_p), _ptr(lp), _ptr(ent),
                                      _ptr(status_word), _ptr(workspace), wsb, _stream(dev))
        _check("rlk_lmhead_logprob", code)
    return lp, ent


def lmhead_backward(hidden, w_vocab, token_ids, temperature, lse, entropy, grad_logprob=None,
                    grad_entropy=None, *, grad_hidden=None, grad_w=None, accumulate_grad_w=False,
                    workspace=None):
    """Gradients of the fused LM-head path: (dL/dhidden fp32 [T, H],
    dL/dW fp32 [V, H]); ``lse`` and ``entropy`` from the forward."""
    lib = load()
    _need_cuda(hidden, w_vocab, token_ids, lse, entropy, grad_logprob, grad_entropy, grad_hidden,
               grad_w)
    if hidden.dtype != torch.bfloat16 or w_vocab.dtype != torch.bfloat16:
        raise ValueError("hidden and w_vocab must be bf16")
    if not (hidden.is_contiguous() and w_vocab.is_contiguous()):
        raise ValueError("hidden and w_vocab must be contiguous")
    T, H = hidden.shape
    V, H2 = w_vocab.shape
    if H != H2:
        raise ValueError("hidden and w_vocab disagree on H")
    for t in (lse, entropy, grad_logprob, grad_entropy):
        if t is not None and (t.dtype != torch.float32 or t.numel() != T or not t.is_contiguous()):
            raise ValueError("lse, entropy and the gradients must be contiguous fp32 [T]")
    dev = hidden.device
    if grad_hidden is None:
        grad_hidden = torch.empty((T, H), device=dev, dtype=torch.float32)
    if grad_w is None:
        if accumulate_grad_w:
            raise ValueError("accumulate_grad_w needs grad_w")
        grad_w = torch.empty((V, H), device=dev, dtype=torch.float32)
    for t, shp in ((grad_hidden, (T, H)), (grad_w, (V, H))):
        if t.dtype != torch.float32 or tuple(t.shape) != shp or not t.is_contiguous():
            raise ValueError("grad_hidden / grad_w must be contiguous fp32 [T, H] / [V, H]")
    need = int(lib.rlk_workspace_size(OP_LMHEAD_BWD, T, V, H))
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dev, dtype=torch.uint8)
    code = lib.rlk_lmhead_logprob_bwd(_ptr(hidden), _ptr(w_vocab), T, H, V, _ptr(token_ids),
                                      float(temperature), _ptr(lse), _ptr(entropy),
                                      _ptr(grad_logprob), _ptr(grad_entropy), _ptr(grad_hidden),
                                      _ptr(grad_w), int(bool(accumulate_grad_w)), _ptr(workspace),
                                      workspace.numel(), _stream(dev))
    _check("rlk_lmhead_logprob_bwd", code)
    return grad_hidden, grad_w


def lmhead_logits_debug(hidden, w_vocab, token_ids, temperature):
    """Validation aid: the fused LM-head path that also returns the fp32 logits
    it computed ([T, V]); for small sizes only."""
    lib = load()
    _need_cuda(hidden, w_vocab, token_ids)
    T, H = hidden.shape
    V = w_vocab.shape[0]
    dev = hidden.device
    need = int(lib.rlk_workspace_size(OP_LMHEAD, T, V, H))
    ws = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    logits = torch.empty(T, V, device=dev, dtype=torch.float32)
    lp = torch.empty(T, device=dev, dtype=torch.float32)
    ent = torch.empty(T, device=dev, dtype=torch.float32)
    code = lib.rlk_lmhead_logits_debug(_ptr(hidden), _ptr(w_vocab), T, H, V, _ptr(token_ids),
                                       float(temperature), _ptr(logits), _ptr(lp), _ptr(ent),
                                       None, _ptr(ws), ws.numel(), _stream(dev))
    _check("rlk_lmhead_logits_debug", code)
    return logits, lp, ent


# ------------------------------------------------------------ canonical partition
def canonical_plan(tp_size: int, tp_rank: int, n_virtual: int = CANONICAL_TP,
                   padded_vocab: int = CANONICAL_VOCAB):
    """The virtual shards a physical tensor-parallel rank holds: (first shard,
    number of shards, first global column, shard width).  Rank k of tp_size
    holds the adjacent shards [k n, (k + 1) n), n = n_virtual / tp_size."""
    if n_virtual % tp_size != 0 or not 0 <= tp_rank < tp_size:
        raise ValueError("tp_size must divide the virtual degree; 0 <= tp_rank < tp_size")
    if padded_vocab % n_virtual != 0:
        raise ValueError("the padded vocabulary must be a multiple of the virtual degree")
    n = n_virtual // tp_size
    width = padded_vocab // n_virtual
    return tp_rank * n, n, tp_rank * n * width, width


def shard_partials(logits, token_ids, temperature, V, first_col, shard_width, n_shards):
    """rlk_shard_partials: [n_shards, T, 8] fp32 partials of the shards whose
    columns ``logits`` ([T, cols], unit stride along the vocabulary) holds."""
    lib = load()
    _need_cuda(logits, token_ids)
    dt = _logits_dtype(logits)
    T = logits.shape[0]
    ld = logits.stride(0) if T > 1 else logits.shape[1]
    out = torch.empty((n_shards, T, SHARD_PARTIAL_WORDS), device=logits.device,
                      dtype=torch.float32)
    code = lib.rlk_shard_partials(_ptr(logits), dt, T, int(V), ld, int(first_col),
                                  int(shard_width), int(n_shards), _ptr(token_ids),
                                  float(temperature), _ptr(out), _stream(logits.device))
    _check("rlk_shard_partials", code)
    return out


def shard_partials_support(logits, token_ids, temperature, V, first_col, shard_width, n_shards,
                           support_offsets, support_ids):
    """rlk_shard_partials_support: [n_shards, T, 8] partials of a supplied
    retained set (CSR over global ids) restricted to this rank's shards."""
    lib = load()
    _need_cuda(logits, token_ids, support_offsets, support_ids)
    dt = _logits_dtype(logits)
    if support_offsets.dtype != torch.int64 or support_ids.dtype != torch.int32:
        raise ValueError("support_offsets int64, support_ids int32")
    T = logits.shape[0]
    ld = logits.stride(0) if T > 1 else logits.shape[1]
    out = torch.empty((n_shards, T, SHARD_PARTIAL_WORDS), device=logits.device,
                      dtype=torch.float32)
    code = lib.rlk_shard_partials_support(_ptr(logits), dt, T, int(V), ld, int(first_col),
                                          int(shard_width), int(n_shards), _ptr(token_ids),
                                          float(temperature), _ptr(support_offsets),
                                          _ptr(support_ids), _ptr(out), _stream(logits.device))
    _check("rlk_shard_partials_support", code)
    return out


def shard_combine(partials, token_ids, temperature, V, shard_width, *, status_word=None):
    """rlk_shard_combine: (logprob, entropy) from all shards' partials
    ([n_shards, T, 8], canonical order)."""
    lib = load()
    _need_cuda(partials, token_ids)
    if partials.dtype != torch.float32 or not partials.is_contiguous() or partials.dim() != 3:
        raise ValueError("partials must be contiguous fp32 [n_shards, T, 8]")
    n_shards, T = partials.shape[0], partials.shape[1]
    lp = torch.empty(T, device=partials.device, dtype=torch.float32)
    ent = torch.empty(T, device=partials.device, dtype=torch.float32)
    code = lib.rlk_shard_combine(_ptr(partials), n_shards, T, int(V), int(shard_width),
                                 _ptr(token_ids), float(temperature), _ptr(lp), _ptr(ent),
                                 _ptr(status_word), _stream(partials.device))
    _check("rlk_shard_combine", code)
    return lp, ent


def shard_window_counts(logits, token_ids, temperature, top_p, V, first_col, shard_width,
                        n_shards, all_partials):
    """rlk_shard_window_counts: [n_shards, T, 8224] uint8 window counts of this
    rank's shards (bf16 ``logits`` [T, cols]), given every shard's partial
    ([n_all, T, 8], canonical order)."""
    lib = load()
    _need_cuda(logits, token_ids, all_partials)
    dt = _logits_dtype(logits)
    T = logits.shape[0]
    ld = logits.stride(0) if T > 1 else logits.shape[1]
    if all_partials.dtype != torch.float32 or not all_partials.is_contiguous():
        raise ValueError("all_partials must be contiguous fp32 [n_all, T, 8]")
    out = torch.empty((n_shards, T, SHARD_COUNTS_BYTES), device=logits.device, dtype=torch.uint8)
    code = lib.rlk_shard_window_counts(_ptr(logits), dt, T, int(V), ld, int(first_col),
                                       int(shard_width), int(n_shards), _ptr(token_ids),
                                       float(temperature), float(top_p), _ptr(all_partials),
                                       int(all_partials.shape[0]), _ptr(out), _stream(logits.device))
    _check("rlk_shard_window_counts", code)
    return out


def shard_combine_topp(partials, counts, token_ids, temperature, top_p, V, shard_width, *,
                       status_word=None):
    """rlk_shard_combine_topp: (logprob, entropy, nucleus size) from all shards'
    partials and window counts (canonical order)."""
    lib = load()
    _need_cuda(partials, counts, token_ids)
    n_shards, T = partials.shape[0], partials.shape[1]
    if counts.shape[:2] != (n_shards, T) or not counts.is_contiguous():
        raise ValueError("counts must be contiguous [n_shards, T, 8224]")
    lp = torch.empty(T, device=partials.device, dtype=torch.float32)
    ent = torch.empty(T, device=partials.device, dtype=torch.float32)
    k = torch.empty(T, device=partials.device, dtype=torch.int32)
    code = lib.rlk_shard_combine_topp(_ptr(partials), _ptr(counts), n_shards, T, int(V),
                                      int(shard_width), _ptr(token_ids), float(temperature),
                                      float(top_p), _ptr(lp), _ptr(ent), _ptr(k), _ptr(status_word),
                                      _stream(partials.device))
    _check("rlk_shard_combine_topp", code)
    return lp, ent, k


def logprob_entropy_canonical_topp(logits, token_ids, temperature, top_p, n_virtual=CANONICAL_TP,
                                   padded_vocab=CANONICAL_VOCAB, *, status_word=None):
    """The canonical partition on one device at top_p < 1: (logprob, entropy,
    nucleus size)."""
    lib = load()
    _need_cuda(logits, token_ids)
    dt = _logits_dtype(logits)
    T, V = logits.shape
    ld = logits.stride(0) if T > 1 else V
    ws = torch.empty(max(int(lib.rlk_workspace_size(OP_CANONICAL_TOPP, T, n_virtual, 0)), 16),
                     device=logits.device, dtype=torch.uint8)
    lp = torch.empty(T, device=logits.device, dtype=torch.float32)
    ent = torch.empty(T, device=logits.device, dtype=torch.float32)
    k = torch.empty(T, device=logits.device, dtype=torch.int32)
    code = lib.rlk_logprob_entropy_canonical_topp(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                                  float(temperature), float(top_p), int(n_virtual),
                                                  int(padded_vocab), _ptr(lp), _ptr(ent), _ptr(k),
                                                  _ptr(status_word), _ptr(ws), ws.numel(),
                                                  _stream(logits.device))
    _check("rlk_logprob_entropy_canonical_topp", code)
    return lp, ent, k


def logprob_entropy_canonical(logits, token_ids, temperature, n_virtual=CANONICAL_TP,
                              padded_vocab=CANONICAL_VOCAB, *, status_word=None):
    """The canonical partition on one device (top_p = 1)."""
    lib = load()
    _need_cuda(logits, token_ids)
    dt = _logits_dtype(logits)
    T, V = logits.shape
    ld = logits.stride(0) if T > 1 else V
    ws = torch.empty(max(int(lib.rlk_workspace_size(OP_CANONICAL, T, n_virtual, 0)), 16),
                     device=logits.device, dtype=torch.uint8)
    lp = torch.empty(T, device=logits.device, dtype=torch.float32)
    ent = torch.empty(T, device=logits.device, dtype=torch.float32)
    code = lib.rlk_logprob_entropy_canonical(_ptr(logits), dt, T, V, ld, _ptr(token_ids),
                                             float(temperature), int(n_virtual), int(padded_vocab),
                                             _ptr(lp), _ptr(ent), _ptr(status_word), _ptr(ws),
                                             ws.numel(), _stream(logits.device))
    _check("rlk_logprob_entropy_canonical", code)
    return lp, ent


def gather_shard_partials(local_partials, group=None):
    """All ranks' per-shard tensors ([n_local, T, ...] each: partials, or window
    counts) gathered in rank order, which is canonical shard order:
    [n_local * world, T, ...].  The exchange of the vocabulary-parallel path
    (once at top_p = 1, twice at top_p < 1)."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    parts = [torch.empty_like(local_partials) for _ in range(world)]
    dist.all_gather(parts, local_partials.contiguous(), group=group)
    return torch.cat(parts, 0)


def vocab_parallel_logprob_entropy(local_logits, token_ids, temperature, V, group=None,
                                   n_virtual=CANONICAL_TP, padded_vocab=CANONICAL_VOCAB,
                                   top_p=1.0):
    """Tensor-parallel log-probability and entropy: this rank's canonical
    shards -> partials -> gather in rank order -> combine; at top_p < 1 the
    gathered partials set every shard's window, whose counts are gathered too
    and combined (returns (logprob, entropy, nucleus size) then).  The result is
    bitwise the same for every tensor-parallel degree."""
    import torch.distributed as dist
    world = dist.get_world_size(group) if dist.is_initialized() else 1
    rank = dist.get_rank(group) if dist.is_initialized() else 0
    _, n, first_col, width = canonical_plan(world, rank, n_virtual, padded_vocab)
    part = shard_partials(local_logits, token_ids, temperature, V, first_col, width, n)
    allp = gather_shard_partials(part, group) if world > 1 else part
    if top_p >= 1.0:
        return shard_combine(allp, token_ids, temperature, V, width)
    cnt = shard_window_counts(local_logits, token_ids, temperature, top_p, V, first_col, width, n,
                              allp)
    allc = gather_shard_partials(cnt, group) if world > 1 else cnt
    return shard_combine_topp(allp, allc, token_ids, temperature, top_p, V, width)


def sample_top_p(logits, temperature, top_p, uniforms, *, row_state=None, status_word=None):
    """Deterministic top-p draw per row (rlk_sample_top_p): the id where the
    cumulative renormalised probability over the retained set, in ranking
    order, first reaches ``uniforms`` (CUDA fp32 [T]).  Without ``row_state``
    the forward runs first to select the sets; ``temperature`` and ``top_p``
    may then be CUDA fp32 [T] tensors (per-row parameters)."""
    lib = load()
    _need_cuda(logits, uniforms, row_state)
    if logits.dtype != torch.bfloat16:
        raise ValueError("the sampler takes bf16 logits")
    _logits_dtype(logits)
    if uniforms.dtype != torch.float32 or not uniforms.is_contiguous():
        raise ValueError("uniforms must be contiguous fp32")
    T, V = logits.shape
    if row_state is None:
        row_state = new_row_state(T, logits.device)
        zeros = torch.zeros(T, dtype=torch.int32, device=logits.device)
        if torch.is_tensor(temperature) or torch.is_tensor(top_p):   # per-row parameters
            full = lambda v: v if torch.is_tensor(v) else torch.full(
                (T,), float(v), device=logits.device, dtype=torch.float32)
            logprob_entropy_rows(logits, zeros, full(temperature), full(top_p),
                                 row_state=row_state)
            temperature = 1.0   # each state carries its row's
        else:
            logprob_entropy(logits, zeros, temperature, top_p, row_state=row_state)
    out = torch.empty(T, dtype=torch.int32, device=logits.device)
    ld = logits.stride(0) if T > 1 else V
    code = lib.rlk_sample_top_p(_ptr(logits), 0, T, V, ld, float(temperature), _ptr(row_state),
                                _ptr(uniforms), _ptr(out), _ptr(status_word),
                                _stream(logits.device))
    _check("rlk_sample_top_p", code)
    return out


# ------------------------------------------- norm and activation checkpoints
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _dtype(dtype, name):
    """dtype index of a bf16 / fp32 output asked for."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"{name} must be bf16 or fp32")
    return dt


def _matrix(t, name, shape=None):
    """dtype index and row stride of a 2-D bf16 / fp32 tensor (of ``shape``) with
    unit stride along its rows."""
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{name} must be 2-D")
    ld, unit = t.stride()
    if unit != 1 and size[1] > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bf16 or fp32")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return dt, (ld if size[0] > 1 else size[1])


def _param(t, H, name):
    """dtype index of a contiguous [H] parameter vector."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or t.shape != (H,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous bf16 or fp32 [{H}]")
    return dt


def _params(H, weight, bias, name="weight", name_bias="bias"):
    """dtype index of the parameter vectors given (fp32 when none is)."""
    dt = 1 if weight is None else _param(weight, H, name)
    if bias is not None:
        db = _param(bias, H, name_bias)
        if weight is not None and db != dt:
            raise ValueError(f"{name} and {name_bias} must have one dtype")
        dt = db
    return dt


def _vector(t, n, name):
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous fp32 [{n}]")


class Checkpoint:
    """An activation [T, H] kept in 8 bits (rlk_checkpoint): int8 ``codes``
    [T, >= H] and uint8 ``scales`` [T, >= ceil(H / 32)].  Both may be replaced
    (moved off the device and back, say): a call takes the tensors that are there."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, T: int, H: int):
        self.codes, self.scales, self.shape = codes, scales, (T, H)
        self.buffers()

    def buffers(self):
        """A reference to the rlk_checkpoint of the tensors as they are now."""
        codes, scales, (T, H) = self.codes, self.scales, self.shape
        if not (codes.is_cuda and scales.is_cuda):
            raise ValueError("librlk operates on CUDA tensors only")
        if codes.dtype is not torch.int8 or scales.dtype is not torch.uint8:
            raise ValueError("codes must be int8, scales uint8")
        a, b = codes.shape, scales.shape
        if (len(a) != 2 or len(b) != 2 or a[0] != T or b[0] != T or a[1] < H or b[1] * CHECKPOINT_BLOCK < H
                or not codes.is_contiguous() or not scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous [T, >= H] and [T, >= ceil(H / 32)]")
        return ctypes.byref(CheckpointBuffers(codes.data_ptr(), scales.data_ptr(), a[1], b[1]))


def new_checkpoint(T: int, H: int, device) -> Checkpoint:
    """Room for the 8-bit checkpoint of an activation [T, H] on a CUDA device."""
    if torch.device(device).type != "cuda":
        raise ValueError("librlk operates on CUDA tensors only")
    ck = Checkpoint.__new__(Checkpoint)   # its tensors are looked at when they are used
    ck.codes = torch.empty((T, (H + 15) // 16 * 16), dtype=torch.int8, device=device)
    ck.scales = torch.empty((T, (H + 511) // 512 * 16), dtype=torch.uint8, device=device)
    ck.shape = (T, H)
    return ck


def checkpoint_pack(x: torch.Tensor, *, out: Checkpoint | None = None, status_word=None) -> Checkpoint:
    """The 8-bit checkpoint of x (CUDA [T, H] bf16 or fp32, rows may be strided)."""
    lib = load()
    _need_cuda(x, status_word)
    dt, ld = _matrix(x, "x")
    T, H = x.shape
    if out is None:
        out = new_checkpoint(T, H, x.device)
    if out.shape != (T, H):
        raise ValueError("out must be a checkpoint of x's shape")
    _check("rlk_checkpoint_pack",
           lib.rlk_checkpoint_pack(x.data_ptr(), dt, T, H, ld, out.buffers(), _ptr(status_word),
                                   _stream(x.device)))
    return out


def checkpoint_unpack(checkpoint: Checkpoint, *, dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """The values a checkpoint stands for (exact in bf16 and fp32)."""
    lib = load()
    T, H = checkpoint.shape
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=checkpoint.codes.device)
    _need_cuda(out)
    dt, ld = _matrix(out, "out", (T, H))
    _check("rlk_checkpoint_unpack",
           lib.rlk_checkpoint_unpack(checkpoint.buffers(), T, H, out.data_ptr(), dt, ld, _stream(out.device)))
    return out


def norm(x: torch.Tensor, weight=None, bias=None, *, kind: int = NORM_LAYER, eps: float = 1e-5,
         out=None, out_dtype=None, checkpoint: Checkpoint | None = None, status_word=None):
    """Layer or RMS norm of each row of x (CUDA [T, H] bf16 or fp32).  Returns
    (y, mean, rstd); mean is None for NORM_RMS.  ``checkpoint`` (from
    ``new_checkpoint``) receives x in 8 bits for ``norm_backward``."""
    lib = load()
    _need_cuda(x, weight, bias, out, status_word)
    dt, ld = _matrix(x, "x")
    T, H = x.shape
    pdt = _params(H, weight, bias)
    dev = x.device
    if out is None:
        ydt, ldy = (dt if out_dtype is None else _dtype(out_dtype, "out_dtype")), H
        out = torch.empty_like(x) if out_dtype is None and ld == H else torch.empty(
            (T, H), dtype=out_dtype or x.dtype, device=dev)
    else:
        ydt, ldy = _matrix(out, "out", (T, H))
    ck = None
    if checkpoint is not None:
        if checkpoint.shape != (T, H):
            raise ValueError("checkpoint must be of x's shape")
        ck = checkpoint.buffers()
    mean = None if kind == NORM_RMS else torch.empty(T, dtype=torch.float32, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    code = lib.rlk_norm_fwd(x.data_ptr(), dt, T, H, ld, _ptr(weight), _ptr(bias), pdt, kind, eps,
                            out.data_ptr(), ydt, ldy, _ptr(mean), rstd.data_ptr(), ck,
                            _ptr(status_word), _stream(dev))
    _check("rlk_norm_fwd", code)
    return out, mean, rstd


def norm_backward(dy: torch.Tensor, x, weight, mean, rstd, *, kind: int = NORM_LAYER,
                  grad_dtype=None, out=None, want_weight_grad: bool = True,
                  want_bias_grad: bool = True, grad_weight=None, grad_bias=None,
                  accumulate: bool = False, workspace=None):
    """Gradients of ``norm``: (dL/dx, dL/dweight fp32 [H] or None, dL/dbias
    fp32 [H] or None).  ``x`` is the forward's input or its ``Checkpoint``;
    ``dy`` bf16 or fp32 (``lmhead_backward``'s grad_hidden).  ``accumulate``
    adds into ``grad_weight`` / ``grad_bias``."""
    lib = load()
    kept = x if isinstance(x, Checkpoint) else None
    _need_cuda(dy, None if kept else x, weight, mean, rstd, out, grad_weight, grad_bias, workspace)
    gdt, ldg = _matrix(dy, "dy")
    T, H = dy.shape
    dev = dy.device
    if tuple(x.shape) != (T, H):
        raise ValueError("x must have dy's shape")
    dt, ld = (0, H) if kept else _matrix(x, "x")
    pdt = _params(H, weight, None)
    if mean is not None:
        _vector(mean, T, "mean")
    _vector(rstd, T, "rstd")
    if out is None:
        out = torch.empty((T, H), dtype=grad_dtype or (torch.bfloat16 if kept else x.dtype), device=dev)
    odt, ldo = _matrix(out, "out", (T, H))
    if accumulate and ((want_weight_grad and grad_weight is None) or (want_bias_grad and grad_bias is None)):
        raise ValueError("accumulate needs grad_weight and grad_bias")
    if grad_weight is not None:
        _vector(grad_weight, H, "grad_weight")
    elif want_weight_grad:
        grad_weight = torch.empty(H, dtype=torch.float32, device=dev)
    if grad_bias is not None:
        _vector(grad_bias, H, "grad_bias")
    elif want_bias_grad:
        grad_bias = torch.empty(H, dtype=torch.float32, device=dev)
    if workspace is None and (grad_weight is not None or grad_bias is not None):
        workspace = torch.empty(max(lib.rlk_workspace_size(OP_NORM_BWD, T, H, 0), 16), dtype=torch.uint8,
                                device=dev)
    ck = None if kept is None else kept.buffers()
    code = lib.rlk_norm_bwd(dy.data_ptr(), gdt, ldg, None if kept else x.data_ptr(), dt, ld, ck, T, H,
                            _ptr(weight), pdt, kind, _ptr(mean), rstd.data_ptr(), out.data_ptr(), odt,
                            ldo, _ptr(grad_weight), _ptr(grad_bias), int(bool(accumulate)),
                            _ptr(workspace), 0 if workspace is None else workspace.numel(),
                            _stream(dev))
    _check("rlk_norm_bwd", code)
    return out, grad_weight, grad_bias


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, kind, eps, keep8):
        ck = new_checkpoint(x.shape[0], x.shape[1], x.device) if keep8 else None
        y, mean, rstd = norm(x, weight, bias, kind=kind, eps=eps, checkpoint=ck)
        ctx.save_for_backward(ck.codes if keep8 else x, ck.scales if keep8 else None, weight, mean, rstd)
        ctx.kind, ctx.H, ctx.x_dtype = kind, x.shape[1], x.dtype
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        kept, scales, weight, mean, rstd = ctx.saved_tensors
        x = kept if scales is None else Checkpoint(kept, scales, kept.shape[0], ctx.H)
        dx, dw, db = norm_backward(dy.contiguous(), x, weight, mean, rstd, kind=ctx.kind,
                                   grad_dtype=ctx.x_dtype,
                                   want_weight_grad=weight is not None and ctx.needs_input_grad[1],
                                   want_bias_grad=ctx.bias_dtype is not None and ctx.needs_input_grad[2])
        return (dx, None if dw is None else dw.to(weight.dtype),
                None if db is None else db.to(ctx.bias_dtype), None, None, None)


def norm_autograd(x: torch.Tensor, weight=None, bias=None, *, kind: int = NORM_LAYER,
                  eps: float = 1e-5, keep_8bit: bool = False):
    """``norm`` as a differentiable op; ``keep_8bit`` keeps x for the backward as
    its 8-bit checkpoint instead of the tensor."""
    return _Norm.apply(x, weight, bias, kind, eps, keep_8bit)


# ------------------------------------------------------------ linear
def _bf16(t, name, shape=None):
    """Row stride of a 2-D bf16 tensor (of ``shape``) with unit stride along its rows."""
    dt, ld = _matrix(t, name, shape)
    if dt != 0:
        raise ValueError(f"{name} must be bf16")
    return ld


def _copied(rows, cols, ptr, ld):
    """Bytes of the workspace for the copy that a product's bf16 operand needs when
    its rows do not start on 16-byte boundaries."""
    return 0 if ptr % 16 == 0 and ld % 8 == 0 else -(-rows * (-(-cols // 8) * 16) // 256) * 256


def linear(x: torch.Tensor, weight: torch.Tensor, bias=None, residual=None, *,
           activation: int = ACT_NONE, return_preact: bool = False, out=None, out_dtype=None,
           workspace=None):
    """act(x weight^T + bias) + residual: x [M, K], weight [N, K], residual
    [M, N] CUDA bf16 (rows may be strided), bias [N] bf16 or fp32.  Returns y
    (bf16, or ``out_dtype`` fp32; ``out`` may be the residual itself), or
    (y, z) with the bf16 pre-activation for ``linear_backward``."""
    lib = load()
    _need_cuda(x, weight, bias, residual, out, workspace)
    ldx, ldw = _bf16(x, "x"), _bf16(weight, "weight")
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError("x and weight disagree on K")
    bdt = 1 if bias is None else _param(bias, N, "bias")
    dev = x.device
    ldr = 0 if residual is None else _bf16(residual, "residual", (M, N))
    if out is None:
        ydt, ldy = (0 if out_dtype is None else _dtype(out_dtype, "out_dtype")), N
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=dev)
    else:
        ydt, ldy = _matrix(out, "out", (M, N))
    z = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if return_preact else None
    px, pw = x.data_ptr(), weight.data_ptr()
    if workspace is None and M > 4:   # fewer rows are not copied
        need = _copied(M, K, px, ldx) + _copied(N, K, pw, ldw)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    code = lib.rlk_linear_fwd(px, ldx, pw, ldw, _ptr(bias), bdt, _ptr(residual), ldr, M, N, K, activation,
                              out.data_ptr(), ydt, ldy, _ptr(z), N, _ptr(workspace),
                              0 if workspace is None else workspace.numel(), _stream(dev))
    _check("rlk_linear_fwd", code)
    return (out, z) if return_preact else out


def linear_backward(dy: torch.Tensor, x, weight: torch.Tensor, preact=None, *,
                    activation: int = ACT_NONE, grad_dtype=torch.bfloat16,
                    weight_grad_dtype=torch.float32, want_x_grad: bool = True,
                    want_weight_grad: bool = True, want_bias_grad: bool = True, grad_weight=None,
                    grad_bias=None, accumulate: bool = False, workspace=None):
    """Gradients of ``linear``: (dL/dx [M, K], dL/dweight [N, K], dL/dbias fp32
    [N]), None where not wanted; the residual's gradient is dy.  ``x`` is the
    forward's input or its ``Checkpoint``.  ``accumulate`` adds into
    ``grad_weight`` (fp32) and ``grad_bias``."""
    lib = load()
    kept = x if isinstance(x, Checkpoint) else None
    _need_cuda(dy, None if kept else x, weight, preact, grad_weight, grad_bias, workspace)
    lddy, ldw = _bf16(dy, "dy"), _bf16(weight, "weight")
    M, N = dy.shape
    K = weight.shape[1]
    if weight.shape[0] != N or (x is not None and tuple(x.shape) != (M, K)):
        raise ValueError("dy, x and weight disagree on M, N or K")
    ldx = 0 if x is None or kept else _bf16(x, "x")
    ldz = 0 if preact is None else _bf16(preact, "preact", (M, N))
    if accumulate and ((want_weight_grad and grad_weight is None) or (want_bias_grad and grad_bias is None)):
        raise ValueError("accumulate needs grad_weight and grad_bias")
    dev = dy.device
    dx = torch.empty((M, K), device=dev, dtype=grad_dtype) if want_x_grad else None
    if grad_weight is None and want_weight_grad:
        grad_weight = torch.empty((N, K), device=dev, dtype=weight_grad_dtype)
    if grad_bias is None and want_bias_grad:
        grad_bias = torch.empty(N, device=dev, dtype=torch.float32)
    xdt = 0 if dx is None else _matrix(dx, "dx")[0]
    wdt, ldgw = (1, K) if grad_weight is None else _matrix(grad_weight, "grad_weight")
    if grad_weight is not None and tuple(grad_weight.shape) != (N, K):
        raise ValueError("grad_weight must be [N, K]")
    if grad_bias is not None and (grad_bias.dtype != torch.float32 or grad_bias.numel() != N
                                  or not grad_bias.is_contiguous()):
        raise ValueError("grad_bias must be contiguous fp32 [N]")
    px = None if x is None or kept else x.data_ptr()
    if workspace is None and M > 0:   # what this call uses: copies of operands, partial sums of the bias gradient
        all_copies = _copied(M, N, 1, 0) + _copied(N, K, 1, 0) + _copied(M, K, 1, 0)
        need = 0
        if grad_bias is not None:
            need += lib.rlk_workspace_size(OP_LINEAR_BWD, M, N, K) - all_copies
        if dx is not None or grad_weight is not None:
            need += _copied(M, N, dy.data_ptr() if activation == ACT_NONE else 1, lddy)
        if dx is not None:
            need += _copied(N, K, weight.data_ptr(), ldw)
        if grad_weight is not None:
            need += _copied(M, K, px or 1, ldx)
        workspace = torch.empty(need, device=dev, dtype=torch.uint8) if need else None
    ck = None if kept is None else kept.buffers()
    _check("rlk_linear_bwd",
           lib.rlk_linear_bwd(_ptr(dy), lddy, px, ldx, ck, _ptr(weight), ldw,
                              _ptr(preact), ldz, M, N, K, int(activation), _ptr(dx), xdt, K,
                              _ptr(grad_weight), wdt, ldgw, _ptr(grad_bias), int(bool(accumulate)),
                              _ptr(workspace), 0 if workspace is None else workspace.numel(),
                              _stream(dev)))
    return dx, grad_weight, grad_bias


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, keep8):
        if activation == ACT_NONE:
            y, z = linear(x, weight, bias, residual), None
        else:
            y, z = linear(x, weight, bias, residual, activation=activation, return_preact=True)
        ck = checkpoint_pack(x) if keep8 else None
        ctx.save_for_backward(ck.codes if keep8 else x, ck.scales if keep8 else None, weight, z)
        ctx.activation, ctx.bias_dtype = activation, None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        kept, scales, weight, z = ctx.saved_tensors
        x = kept if scales is None else Checkpoint(kept, scales, kept.shape[0], weight.shape[1])
        dy = dy.contiguous()
        dx, dw, db = linear_backward(dy, x, weight, z, activation=ctx.activation,
                                     weight_grad_dtype=weight.dtype,
                                     want_x_grad=ctx.needs_input_grad[0],
                                     want_weight_grad=ctx.needs_input_grad[1],
                                     want_bias_grad=ctx.needs_input_grad[2])
        return (dx, dw, None if db is None else db.to(ctx.bias_dtype),
                dy if ctx.needs_input_grad[3] else None, None, None)


def linear_autograd(x: torch.Tensor, weight: torch.Tensor, bias=None, residual=None, *,
                    activation: int = ACT_NONE, keep_8bit: bool = False):
    """``linear`` as a differentiable op; ``keep_8bit`` keeps x for the backward
    as its 8-bit checkpoint instead of the tensor."""
    return _Linear.apply(x, weight, bias, residual, activation, keep_8bit)


# ------------------------------------------------------------ gated linear
def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, bias_gate=None, bias_up=None, *,
                 activation: int = ACT_SILU, return_preact: bool = False, out=None, out_dtype=None,
                 workspace=None):
    """act(x w_gate^T + bias_gate) * (x w_up^T + bias_up): x [M, K], weights
    [N, K] CUDA bf16 (rows may be strided), biases [N] bf16 or fp32.  Returns y
    (bf16, or ``out_dtype`` fp32), or (y, gate, up) with the bf16 projections
    for ``gated_linear_backward``."""
    lib = load()
    _need_cuda(x, w_gate, w_up, bias_gate, bias_up, out, workspace)
    ldx, ldg, ldu = _bf16(x, "x"), _bf16(w_gate, "w_gate"), _bf16(w_up, "w_up")
    M, K = x.shape
    N = w_gate.shape[0]
    if w_gate.shape[1] != K or w_up.shape != w_gate.shape:
        raise ValueError("x, w_gate and w_up disagree on K or N")
    bdt = _params(N, bias_gate, bias_up, "bias_gate", "bias_up")
    dev = x.device
    if out is None:
        ydt, ldy = (0 if out_dtype is None else _dtype(out_dtype, "out_dtype")), N
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=dev)
    else:
        ydt, ldy = _matrix(out, "out", (M, N))
    gate = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if return_preact else None
    up = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if return_preact else None
    px, pg, pu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    if workspace is None and M > 4:   # fewer rows are not copied
        need = _copied(M, K, px, ldx) + _copied(N, K, pg, ldg) + _copied(N, K, pu, ldu)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    code = lib.rlk_gated_linear_fwd(px, ldx, pg, ldg, pu, ldu, _ptr(bias_gate), _ptr(bias_up), bdt, M, N, K,
                                    activation, out.data_ptr(), ydt, ldy, _ptr(gate), _ptr(up), N,
                                    _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev))
    _check("rlk_gated_linear_fwd", code)
    return (out, gate, up) if return_preact else out


def gated_linear_backward(dy: torch.Tensor, x, w_gate: torch.Tensor, w_up: torch.Tensor, gate: torch.Tensor,
                          up: torch.Tensor, *, activation: int = ACT_SILU, grad_dtype=torch.bfloat16,
                          weight_grad_dtype=torch.float32, want_x_grad: bool = True,
                          want_weight_grad: bool = True, want_bias_grad: bool = True, grad_w_gate=None,
                          grad_w_up=None, grad_bias_gate=None, grad_bias_up=None, accumulate: bool = False,
                          workspace=None):
    """Gradients of ``gated_linear``: (dL/dx [M, K], dL/dw_gate, dL/dw_up [N, K],
    dL/dbias_gate, dL/dbias_up fp32 [N]), None where not wanted.  ``gate`` and
    ``up`` from the forward; ``x`` its input or that one's ``Checkpoint``.
    ``accumulate`` adds into the weights' (fp32) and biases' gradients given."""
    lib = load()
    kept = x if isinstance(x, Checkpoint) else None
    _need_cuda(dy, None if kept else x, w_gate, w_up, gate, up, grad_w_gate, grad_w_up, grad_bias_gate,
               grad_bias_up, workspace)
    lddy, ldwg, ldwu = _bf16(dy, "dy"), _bf16(w_gate, "w_gate"), _bf16(w_up, "w_up")
    M, N = dy.shape
    K = w_gate.shape[1]
    if w_gate.shape[0] != N or w_up.shape != w_gate.shape or (x is not None and tuple(x.shape) != (M, K)):
        raise ValueError("dy, x, w_gate and w_up disagree on M, N or K")
    ldg, ldu = _bf16(gate, "gate", (M, N)), _bf16(up, "up", (M, N))
    ldx = 0 if x is None or kept else _bf16(x, "x")
    if accumulate and ((want_weight_grad and (grad_w_gate is None or grad_w_up is None))
                       or (want_bias_grad and (grad_bias_gate is None or grad_bias_up is None))):
        raise ValueError("accumulate needs the gradients to add to")
    for a, b in ((grad_w_gate, grad_w_up), (grad_bias_gate, grad_bias_up)):
        if a is not None and b is not None and a.data_ptr() == b.data_ptr():
            raise ValueError("the gate's and up's gradients must be tensors of their own")
    dev = dy.device
    dx = torch.empty((M, K), device=dev, dtype=grad_dtype) if want_x_grad else None
    xdt = 0 if dx is None else _matrix(dx, "dx")[0]
    wdt, ldgwg, ldgwu = 1, K, K
    if want_weight_grad or grad_w_gate is not None or grad_w_up is not None:
        like = grad_w_gate if grad_w_gate is not None else grad_w_up
        dt = weight_grad_dtype if like is None else like.dtype
        if grad_w_gate is None:
            grad_w_gate = torch.empty((N, K), device=dev, dtype=dt)
        if grad_w_up is None:
            grad_w_up = torch.empty((N, K), device=dev, dtype=dt)
        wdt, ldgwg = _matrix(grad_w_gate, "grad_w_gate", (N, K))
        other, ldgwu = _matrix(grad_w_up, "grad_w_up", (N, K))
        if other != wdt:
            raise ValueError("grad_w_gate and grad_w_up must have one dtype")
    if want_bias_grad or grad_bias_gate is not None or grad_bias_up is not None:
        if grad_bias_gate is None:
            grad_bias_gate = torch.empty(N, device=dev, dtype=torch.float32)
        if grad_bias_up is None:
            grad_bias_up = torch.empty(N, device=dev, dtype=torch.float32)
        _vector(grad_bias_gate, N, "grad_bias_gate")
        _vector(grad_bias_up, N, "grad_bias_up")
    px = None if x is None or kept else x.data_ptr()
    if workspace is None and M > 0:   # what this call uses: dg and du, copies of operands, partial sums
        need = 0
        if grad_bias_gate is not None:
            need += (lib.rlk_workspace_size(OP_GATED_LINEAR_BWD, M, N, K) - 2 * _copied(M, N, 1, 0)
                     - 2 * _copied(N, K, 1, 0) - _copied(M, K, 1, 0))
        if dx is not None or grad_w_gate is not None:
            need += 2 * _copied(M, N, 1, 0)
        if dx is not None:
            need += _copied(N, K, w_gate.data_ptr(), ldwg) + _copied(N, K, w_up.data_ptr(), ldwu)
        if grad_w_gate is not None:
            need += _copied(M, K, px or 1, ldx)
        workspace = torch.empty(need, device=dev, dtype=torch.uint8) if need else None
    ck = None if kept is None else kept.buffers()
    _check("rlk_gated_linear_bwd",
           lib.rlk_gated_linear_bwd(_ptr(dy), lddy, px, ldx, ck, _ptr(w_gate), ldwg, _ptr(w_up), ldwu, _ptr(gate),
                                    ldg, _ptr(up), ldu, M, N, K, int(activation), _ptr(dx), xdt, K,
                                    _ptr(grad_w_gate), ldgwg, _ptr(grad_w_up), ldgwu, wdt,
                                    _ptr(grad_bias_gate), _ptr(grad_bias_up), int(bool(accumulate)),
                                    _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                    _stream(dev)))
    return dx, grad_w_gate, grad_w_up, grad_bias_gate, grad_bias_up


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, bias_gate, bias_up, activation, keep8):
        y, gate, up = gated_linear(x, w_gate, w_up, bias_gate, bias_up, activation=activation, return_preact=True)
        ck = checkpoint_pack(x) if keep8 else None
        ctx.save_for_backward(ck.codes if keep8 else x, ck.scales if keep8 else None, w_gate, w_up, gate, up)
        ctx.activation = activation
        ctx.bias_dtypes = [None if b is None else b.dtype for b in (bias_gate, bias_up)]
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        kept, scales, w_gate, w_up, gate, up = ctx.saved_tensors
        x = kept if scales is None else Checkpoint(kept, scales, kept.shape[0], w_gate.shape[1])
        need = ctx.needs_input_grad
        dx, dwg, dwu, dbg, dbu = gated_linear_backward(
            dy.contiguous(), x, w_gate, w_up, gate, up, activation=ctx.activation, weight_grad_dtype=w_gate.dtype,
            want_x_grad=need[0], want_weight_grad=need[1] or need[2], want_bias_grad=need[3] or need[4])
        of = lambda g, want, dtype: g.to(dtype) if want and g is not None else None
        return (dx, dwg if need[1] else None, dwu if need[2] else None, of(dbg, need[3], ctx.bias_dtypes[0]),
                of(dbu, need[4], ctx.bias_dtypes[1]), None, None)


def gated_linear_autograd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, bias_gate=None, bias_up=None, *,
                          activation: int = ACT_SILU, keep_8bit: bool = False):
    """``gated_linear`` as a differentiable op; ``keep_8bit`` keeps x for the
    backward as its 8-bit checkpoint instead of the tensor."""
    return _GatedLinear.apply(x, w_gate, w_up, bias_gate, bias_up, activation, keep_8bit)


# ------------------------------------------------------------ orthogonalised updates
MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=64)
def _coefficients(a, b, c):
    return (ctypes.c_float * 3)(a, b, c)


def _stacked(t, name):
    """(matrices, rows, columns, row stride, matrix stride) of a [m, n] or [B, m, n] tensor."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [m, n] or [B, m, n]")
    m, n = t.shape[-2:]
    ld, unit = t.stride()[-2:]
    if unit != 1 and n > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    B, matrix = (1, 0) if t.dim() == 2 else (t.shape[0], t.stride(0))
    return B, m, n, (ld if m > 1 else n), matrix


def orthogonalise(update: torch.Tensor, *, steps: int = 5, coefficients=MUON_COEFFICIENTS, eps: float = 1e-7, out=None,
                  workspace=None, status_word=None):
    """``update`` ([m, n], or a stack [B, m, n]; CUDA bf16 or fp32, rows and
    matrices may be strided) made nearly orthogonal by ``steps`` Newton-Schulz
    products, bf16 (as an optimiser does between the momentum and the weights).
    ``out`` may be a bf16 ``update`` itself."""
    lib = load()
    _need_cuda(update, out, workspace, status_word)
    dt = _DTYPES.get(update.dtype)
    if dt is None:
        raise ValueError("update must be bf16 or fp32")
    B, m, n, ld, matrix = _stacked(update, "update")
    dev = update.device
    if out is None:
        out = torch.empty(update.shape, dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or out.shape != update.shape:
        raise ValueError("out must be bf16, shaped like update")
    ldo, out_matrix = _stacked(out, "out")[3:]
    if workspace is None and B > 0:
        workspace = torch.empty(lib.rlk_workspace_size(OP_ORTHOGONALISE, B, m, n), dtype=torch.uint8, device=dev)
    code = lib.rlk_orthogonalise(update.data_ptr(), dt, B, m, n, ld, matrix, steps, _coefficients(*coefficients), eps,
                                 out.data_ptr(), ldo, out_matrix, _ptr(status_word), _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), _stream(dev))
    _check("rlk_orthogonalise", code)
    return out


# ------------------------------------------------------------ preference loss
@functools.lru_cache(maxsize=64)
def _pref_config(*fields):
    """A reference to an rlk_pref_config of these fields (the entry point only reads it)."""
    return ctypes.byref(PrefConfig(*fields))


def preference_loss(logp, logp_ref, seq_offsets, *, loss_mask=None, loss_type: int = PREF_SIGMOID,
                    beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                    length_normalise: bool = False, want_grad: bool = True,
                    want_reward: bool = True, want_stats: bool = True, workspace=None):
    """Paired preference loss over packed per-token log-probabilities (CUDA
    fp32); sequences 2 i and 2 i + 1 are pair i's chosen and rejected response.
    ``logp_ref`` None: reference-free.  Returns (loss[1], dL/dlogp or None,
    rewards [2 pairs] or None, stats[PREF_NSTATS] or None)."""
    lib = load()
    _need_cuda(logp, logp_ref, seq_offsets, loss_mask, workspace)
    n_tok, offsets = logp.numel(), seq_offsets.numel()
    _vector(logp, n_tok, "logp")
    if logp_ref is not None:
        _vector(logp_ref, n_tok, "logp_ref")
    if seq_offsets.dtype != torch.int32 or not seq_offsets.is_contiguous() or offsets % 2 != 1:
        raise ValueError("seq_offsets must be contiguous int32 [2 pairs + 1]")
    if loss_mask is not None and (loss_mask.dtype != torch.uint8 or not loss_mask.is_contiguous()
                                  or loss_mask.numel() != n_tok):
        raise ValueError("loss_mask must be contiguous uint8 [n_tok]")
    P, dev = offsets // 2, logp.device
    if workspace is None:
        workspace = torch.empty(lib.rlk_workspace_size(OP_PREFERENCE_LOSS, n_tok, P, 0),
                                dtype=torch.uint8, device=dev)
    cfg = _pref_config(loss_type, beta, label_smoothing, margin, bool(length_normalise))
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    grad = torch.empty_like(logp) if want_grad else None
    reward = torch.empty(2 * P, dtype=torch.float32, device=dev) if want_reward else None
    stats = torch.empty(PREF_NSTATS, dtype=torch.float32, device=dev) if want_stats else None
    code = lib.rlk_preference_loss(logp.data_ptr(), _ptr(logp_ref), _ptr(loss_mask), seq_offsets.data_ptr(),
                                   P, n_tok, cfg, loss.data_ptr(), _ptr(grad), _ptr(reward),
                                   _ptr(stats), workspace.data_ptr(), workspace.numel(),
                                   _stream(dev))
    _check("rlk_preference_loss", code)
    return loss, grad, reward, stats


# ------------------------------------------------------------ given tokens and alternatives
def new_token_state(T: int, device) -> torch.Tensor:
    """Room for what ``token_logprobs`` keeps for its backward (rlk_token_state[T])."""
    return torch.empty((T, 4), dtype=torch.float32, device=device)


def _token_state(state, T):
    if state.dtype != torch.float32 or state.shape != (T, 4) or not state.is_contiguous():
        raise ValueError("state must come from new_token_state(T)")


def _token_ids(token_ids, T):
    """Tokens a row of contiguous int32 [T] or [T, C] ids."""
    if token_ids is None:
        return 0
    if (token_ids.dtype != torch.int32 or not token_ids.is_contiguous() or token_ids.dim() not in (1, 2)
            or token_ids.shape[0] != T):
        raise ValueError("token_ids must be contiguous int32 [T] or [T, C]")
    return 1 if token_ids.dim() == 1 else token_ids.shape[1]


def token_logprobs(logits: torch.Tensor, token_ids, temperature: float = 1.0, *, n_top: int = 0,
                   state: torch.Tensor | None = None, status_word=None):
    """Log-probabilities of given tokens over the whole vocabulary, the entropy
    and the ``n_top`` largest alternatives of each row of logits (CUDA [T, V]
    bf16 or fp32, rows may be strided; -inf rules a token out).  ``token_ids``:
    CUDA int32 [T], [T, C] (-1: an empty place) or None.  Returns (logprob shaped
    like token_ids or None, entropy [T], top_ids int32 [T, n_top] or None, their
    log-probabilities or None).  ``state`` (from ``new_token_state``) receives
    what ``token_logprobs_backward`` needs."""
    lib = load()
    _need_cuda(logits, token_ids, state, status_word)
    dt = _logits_dtype(logits)
    T, V = logits.shape
    C = _token_ids(token_ids, T)
    if not 0 <= n_top <= MAX_ALTERNATIVES or C > MAX_TOKENS:
        raise ValueError(f"at most {MAX_TOKENS} tokens and {MAX_ALTERNATIVES} alternatives a row")
    if state is not None:
        _token_state(state, T)
    dev = logits.device
    f32 = torch.float32
    lp = None if token_ids is None else torch.empty(token_ids.shape, dtype=f32, device=dev)
    ent = torch.empty(T, dtype=f32, device=dev)
    ids = torch.empty((T, n_top), dtype=torch.int32, device=dev) if n_top else None
    top = torch.empty((T, n_top), dtype=f32, device=dev) if n_top else None
    code = lib.rlk_token_logprobs_fwd(logits.data_ptr(), dt, T, V, logits.stride(0) if T > 1 else V,
                                      _ptr(token_ids), C, temperature, n_top, _ptr(lp), ent.data_ptr(),
                                      _ptr(ids), _ptr(top), _ptr(state), _ptr(status_word), _stream(dev))
    _check("rlk_token_logprobs_fwd", code)
    return lp, ent, ids, top


def token_logprobs_backward(logits: torch.Tensor, token_ids, temperature: float, state: torch.Tensor,
                            grad_logprob=None, grad_entropy=None, *, top_ids=None, grad_top=None,
                            out=None, grad_dtype=None, status_word=None):
    """dL/dlogits [T, V] of ``token_logprobs`` for the gradients of its outputs
    (fp32, each or None); ``top_ids`` from the forward with ``grad_top``.
    ``grad_dtype`` (bf16 or fp32) defaults to the logits' dtype; ``out`` may be
    a strided [T, V] tensor."""
    lib = load()
    _need_cuda(logits, token_ids, state, grad_logprob, grad_entropy, top_ids, grad_top, out, status_word)
    dt = _logits_dtype(logits)
    T, V = logits.shape
    C = _token_ids(token_ids, T)
    _token_state(state, T)
    if grad_logprob is not None and (token_ids is None or grad_logprob.dtype != torch.float32
                                     or grad_logprob.shape != token_ids.shape or not grad_logprob.is_contiguous()):
        raise ValueError("grad_logprob must be contiguous fp32, shaped like token_ids")
    if grad_entropy is not None:
        _vector(grad_entropy, T, "grad_entropy")
    n_top = 0
    if grad_top is not None:
        if (top_ids is None or top_ids.dtype != torch.int32 or top_ids.dim() != 2 or top_ids.shape[0] != T
                or not top_ids.is_contiguous()):
            raise ValueError("grad_top needs top_ids, contiguous int32 [T, n_top]")
        if grad_top.dtype != torch.float32 or grad_top.shape != top_ids.shape or not grad_top.is_contiguous():
            raise ValueError("grad_top must be contiguous fp32, shaped like top_ids")
        n_top = top_ids.shape[1]
    if out is None:
        out = torch.empty((T, V), dtype=grad_dtype or logits.dtype, device=logits.device)
    elif grad_dtype is not None and out.dtype != grad_dtype:
        raise ValueError("out must be of grad_dtype")
    gd, ldg = _matrix(out, "out", (T, V))
    code = lib.rlk_token_logprobs_bwd(logits.data_ptr(), dt, T, V, logits.stride(0) if T > 1 else V,
                                      _ptr(token_ids), C, temperature, state.data_ptr(), _ptr(grad_logprob),
                                      _ptr(grad_entropy), _ptr(top_ids) if n_top else None, n_top,
                                      _ptr(grad_top), out.data_ptr(), gd, ldg, _ptr(status_word),
                                      _stream(logits.device))
    _check("rlk_token_logprobs_bwd", code)
    return out


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token_ids, temperature, n_top):
        state = new_token_state(logits.shape[0], logits.device)
        lp, ent, ids, top = token_logprobs(logits, token_ids, temperature, n_top=n_top, state=state)
        ctx.save_for_backward(logits, token_ids, state, ids)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        if ids is not None:
            ctx.mark_non_differentiable(ids)
        return lp, ent, ids, top

    @staticmethod
    @once_differentiable
    def backward(ctx, g_lp, g_ent, _, g_top):
        logits, token_ids, state, ids = ctx.saved_tensors
        if g_lp is None and g_ent is None and g_top is None:
            return None, None, None, None
        flat = lambda g: None if g is None else g.contiguous()
        g = token_logprobs_backward(logits, token_ids, ctx.temperature, state, flat(g_lp), flat(g_ent),
                                    top_ids=ids, grad_top=flat(g_top))
        return g, None, None, None


def token_logprobs_autograd(logits: torch.Tensor, token_ids, temperature: float = 1.0, *, n_top: int = 0):
    """``token_logprobs`` as a differentiable op."""
    return _TokenLogprobs.apply(logits, token_ids, temperature, n_top)


def inject_launch_failures(n: int) -> int:
    """Host-side fault injection: the next ``n`` entry points that would launch
    return RLK_ERR_CUDA (raised as RlkError) without launching.  Returns the
    count that was pending."""
    return int(load().rlk_debug_inject_launch_failures(int(n)))


def set_wait_limit(cycles: int) -> int:
    """Debug: the clock cycles a bounded device wait may take before it gives
    up (<= 0 restores the default of about a second).  Returns the previous
    limit."""
    return int(load().rlk_debug_set_wait_limit(int(cycles)))


def withhold_copy(stage: int) -> None:
    """Debug: the next scorer (or LM-head forward) launch skips the bulk copy
    of the given stage in its first CTA, so the wait on it runs out; < 0
    clears it."""
    load().rlk_debug_withhold_copy(int(stage))


def set_sampler_mode(mode: int) -> int:
    """Debug: the ways rlk_sample_top_p may take to a draw: 1 the direct mode
    with its member list (default), 2 the direct mode without the list, 0 the
    radix descent only.  Returns the previous mode."""
    return int(load().rlk_debug_set_sampler_mode(int(mode)))
