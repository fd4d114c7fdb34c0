"""GB300 (sm_103a) fused selected-token logprob and train/rollout mismatch statistics.

A thin ctypes binding over ``libtim.so`` (C ABI in ``include/tim.h``).  The
functions named like the C entry points (``tim_token_logprob``,
``tim_mismatch_stats``, ``tim_check``) take raw device pointers and sizes;
``token_logprob`` and ``mismatch_stats`` take torch CUDA tensors and only
marshal them.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU fallback: if ``libtim.so`` is missing, importing the
binding succeeds but every call raises ``TimError``.

Method: the trainer recomputes l_t = log softmax(h_t W^T)[a_t] from its final
hidden states (icarus "RL: Training Inference Mismatch", section "log p") and
compares it with the rollout engine's logprob through delta = l_train -
l_rollout, r = e^delta, the k1/k2/k3 KL estimators, the truncated importance
weight min(r, C) and masked per-sequence / per-batch means with a sequence
rejection flag (VeXact summary, eq. (1) and "Algorithmic TIM Compensation";
LoongSage "Train-Inference Consistency", sections 4-5).  ``tis_ppo`` gives the
clipped PPO surrogate weighted by the truncated importance weight, its
gradient and masked means (VeXact summary eq. (2)-(3)).

Where a program holds the logits themselves, ``process_logits`` applies the
sampler's rules (biases, penalties for repeated tokens, temperature, grammar
masks), ``processed_logprob`` gives the chosen token's log-probability under them
(with its gradient), and ``distill_topk`` distils from a teacher's top logits
(icarus page, section "logits processor"; no formulas there).
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import math
import os
import threading

__all__ = [
    "TimError", "SEQ_FIELDS", "BATCH_FIELDS", "PPO_FIELDS", "MONITOR_FIELDS", "tim_mismatch_out", "tim_ppo_out", "lib_path", "load",
    "tim_token_logprob", "tim_token_logprob_temperature", "tim_token_logprob_noalloc", "tim_mismatch_stats",
    "tim_mismatch_fold", "SEQ_RECORD_WORDS", "mismatch_fold",
    "tim_tis_ppo", "tim_mismatch_monitor", "tim_split_weight_bytes", "tim_split_weight_fp32",
    "tim_token_logprob_fp32_head", "tim_token_logprob_backward", "tim_selftest_wait_timeout", "tim_check", "tim_last_error", "tim_version",
    "tim_debug_violation", "tim_debug_build", "load_debug", "checked", "CHECKS",
    "token_logprob", "token_logprob_backward", "split_weight_fp32", "token_logprob_fp32_head", "mismatch_stats", "mismatch_monitor", "tis_ppo", "check",
    "LogitsRules", "tim_logits_rules", "tim_process_logits", "tim_processed_logprob", "tim_processed_logprob_backward",
    "tim_distill_topk", "tim_distill_topk_backward", "tim_distill_topk_step", "process_logits", "processed_logprob",
    "processed_logprob_backward", "distill_topk", "distill_topk_backward", "distill_topk_step", "packed_spans",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libtim.so")
_DEBUG_LIB_PATH = os.path.join(_PKG, "libtim_debug.so")

TIM_OK = 0
TIM_ERR_INVALID_ARG = -1
TIM_ERR_UNSUPPORTED_DEVICE = -2
TIM_ERR_CUDA = -3
TIM_ERR_TIMEOUT = -4
TIM_ERR_BAD_INPUT = -5
NOALLOC_SCRATCH_BYTES = 16 << 20   # TIM_NOALLOC_SCRATCH_BYTES in include/tim.h

# TIM_CHECK_* of include/tim.h: what the checked build (libtim_debug.so) records
CHECKS = {0: "none", 1: "target", 2: "mask", 3: "logit", 4: "backward_input", 5: "advantage",
          6: "tma_coord", 7: "store", 8: "unit", 9: "bulk"}

SEQ_RECORD_WORDS = 16   # TIM_SEQ_RECORD_WORDS
TIM_F32, TIM_BF16, TIM_F16 = 0, 1, 2   # enum tim_dtype
DISTILL_MAX_K = 1024    # TIM_DISTILL_MAX_K
SEQ_FIELDS = ("n_mask", "n_used", "n_nan", "n_clip", "mean_delta", "mean_abs_delta",
              "max_abs_delta", "mean_k1", "mean_k2", "mean_k3", "mean_w", "mean_rel")
BATCH_FIELDS = ("n_mask", "n_used", "n_nan", "n_clip", "mean_delta", "mean_abs_delta",
                "max_abs_delta", "mean_k1", "mean_k2", "mean_k3", "mean_w", "mean_rel",
                "seqmean_k1", "seqmean_k2", "seqmean_k3", "clip_ratio", "nan_ratio",
                "reject_ratio", "n_seqs_nonempty", "n_rejected")

PPO_FIELDS = ("n_mask", "n_used", "n_ppo_clipped", "n_tis_clipped", "mean_loss", "seqmean_loss",
              "ppo_clip_ratio", "tis_clip_ratio", "n_seqs_nonempty")

MONITOR_FIELDS = ("n_used", "p95_abs_delta", "ratio_q01", "ratio_q50", "ratio_q99", "n_extreme",
                  "frac_extreme")


class TimError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("tim error %d: %s" % (code, msg))
        self.code = code


class tim_mismatch_out(ctypes.Structure):
    """Mirror of the C struct tim_mismatch_out (host struct of device pointers)."""
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("num_tokens", ctypes.c_int64),
        ("tau_seq", ctypes.c_float),
        ("seq_estimator", ctypes.c_int32),
        ("token_weight", ctypes.c_void_p),
        ("seq_stats", ctypes.c_void_p),
        ("seq_flags", ctypes.c_void_p),
        ("batch_stats", ctypes.c_void_p),
        ("seq_records", ctypes.c_void_p),
    ]


class tim_ppo_out(ctypes.Structure):
    """Mirror of the C struct tim_ppo_out (host struct of device pointers)."""
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("num_tokens", ctypes.c_int64),
        ("token_loss", ctypes.c_void_p),
        ("token_grad", ctypes.c_void_p),
        ("seq_loss", ctypes.c_void_p),
        ("batch_stats", ctypes.c_void_p),
    ]


class tim_logits_rules(ctypes.Structure):
    """Mirror of the C struct tim_logits_rules (host struct of device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("temperature", "repetition", "presence", "frequency", "history", "history_spans", "bias_offsets",
                 "bias_ids", "bias_values", "allowed", "allowed_rows")] + [
        ("allowed_stride", ctypes.c_int64),
        ("num_history", ctypes.c_int32),
        ("num_bias", ctypes.c_int32),
        ("num_allowed", ctypes.c_int32),
    ]


_lock = threading.Lock()
_lib = None          # the library calls go to (libtim.so, or libtim_debug.so inside `checked()`)
_release = None
_debug = None


def lib_path() -> str:
    return _LIB_PATH


def _open(path: str, what: str):
    if not os.path.exists(path):
        raise TimError(TIM_ERR_CUDA, "%s is not built (%s); run "
                       "`python -m rollout_logprob_mismatch_gb300.build`" % (what, path))
    lib = ctypes.CDLL(path)
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    lib.tim_token_logprob.argtypes = [P, P, P, I64, I64, I64, P, P, P]
    lib.tim_token_logprob.restype = ctypes.c_int
    lib.tim_token_logprob_temperature.argtypes = [P, P, P, I64, I64, I64, ctypes.c_float, P, P, P]
    lib.tim_token_logprob_temperature.restype = ctypes.c_int
    lib.tim_token_logprob_noalloc.argtypes = [P, P, P, I64, I64, I64, P, P, P]
    lib.tim_token_logprob_noalloc.restype = ctypes.c_int
    lib.tim_mismatch_stats.argtypes = [P, P, P, P, ctypes.c_float, ctypes.POINTER(tim_mismatch_out), P]
    lib.tim_mismatch_stats.restype = ctypes.c_int
    lib.tim_mismatch_fold.argtypes = [P, ctypes.c_int32, P, P]
    lib.tim_mismatch_fold.restype = ctypes.c_int
    F = ctypes.c_float
    lib.tim_tis_ppo.argtypes = [P, P, P, P, P, P, F, F, F, ctypes.POINTER(tim_ppo_out), P]
    lib.tim_tis_ppo.restype = ctypes.c_int
    lib.tim_split_weight_bytes.argtypes = [I64, I64]
    lib.tim_split_weight_bytes.restype = ctypes.c_int64
    lib.tim_split_weight_fp32.argtypes = [P, I64, I64, P, P]
    lib.tim_split_weight_fp32.restype = ctypes.c_int
    lib.tim_token_logprob_fp32_head.argtypes = [P, P, P, I64, I64, I64, ctypes.c_float, P, P, P]
    lib.tim_token_logprob_fp32_head.restype = ctypes.c_int
    lib.tim_token_logprob_backward.argtypes = [P, P, P, P, P, I64, I64, I64, ctypes.c_float, P, P,
                                               ctypes.c_int, P]
    lib.tim_token_logprob_backward.restype = ctypes.c_int
    lib.tim_mismatch_monitor.argtypes = [P, P, P, I64, F, P, P, P]
    lib.tim_mismatch_monitor.restype = ctypes.c_int
    head = [P, ctypes.c_int, I64, I64, I64]   # logits, dtype, N, V, stride
    RP = ctypes.POINTER(tim_logits_rules)
    teacher = [P, P, P, I64, F]               # ids, logits, lse, K, temperature
    for name, args in (("tim_process_logits", head + [RP, P, ctypes.c_int, I64, P]),
                       ("tim_processed_logprob", head + [RP, P, P, P, P]),
                       ("tim_processed_logprob_backward", head + [RP, P, P, P, P, I64, P]),
                       ("tim_distill_topk", head + teacher + [P, P, P, P]),
                       ("tim_distill_topk_backward", head + teacher + [P, P, P, P, I64, P]),
                       ("tim_distill_topk_step", head + teacher + [P, P, P, P, P, I64, P])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    lib.tim_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
    lib.tim_selftest_wait_timeout.restype = ctypes.c_int
    lib.tim_check.argtypes = [P]
    lib.tim_check.restype = ctypes.c_int
    lib.tim_debug_violation.argtypes = [ctypes.POINTER(ctypes.c_int64), P]
    lib.tim_debug_violation.restype = ctypes.c_int
    lib.tim_debug_build.argtypes = []
    lib.tim_debug_build.restype = ctypes.c_int
    lib.tim_last_error.argtypes = []
    lib.tim_last_error.restype = ctypes.c_char_p
    lib.tim_version.argtypes = []
    lib.tim_version.restype = ctypes.c_int
    return lib


def load():
    """The library calls go to: libtim.so (libtim_debug.so inside `checked()`);
    raises TimError when it has not been built."""
    global _lib, _release
    with _lock:
        if _lib is None:
            if _release is None:
                _release = _open(_LIB_PATH, "libtim.so")
            _lib = _release
    return _lib


def load_debug():
    """libtim_debug.so: the same library built with TIM_DEBUG (its kernels also
    check indices, TMA coordinates and input contracts; see include/tim.h)."""
    global _debug
    with _lock:
        if _debug is None:
            _debug = _open(_DEBUG_LIB_PATH, "libtim_debug.so")
    return _debug


@contextlib.contextmanager
def checked():
    """Within the block every call of this module goes to libtim_debug.so
    (one thread at a time); tim_debug_violation() then reports the first
    violation its kernels found."""
    global _lib
    dbg = load_debug()
    prev = load()
    _lib = dbg
    try:
        yield dbg
    finally:
        _lib = prev


# ----------------------------------------------------------------------------- raw C ABI
def tim_token_logprob(h, W, targets, N, D, V, out_logp, out_lse, stream) -> int:
    """C ABI call with integer device addresses; returns the tim_status code."""
    return load().tim_token_logprob(h, W, targets, N, D, V, out_logp, out_lse, stream)


def tim_token_logprob_temperature(h, W, targets, N, D, V, temperature, out_logp, out_lse, stream) -> int:
    """C ABI call of the token logprob at a sampling temperature; returns the tim_status code."""
    return load().tim_token_logprob_temperature(h, W, targets, N, D, V, float(temperature), out_logp,
                                                out_lse, stream)


def tim_token_logprob_noalloc(h, W, targets, N, D, V, out_logp, out_lse, stream) -> int:
    """C ABI call of the variant that allocates nothing (its scratch is a fixed
    NOALLOC_SCRATCH_BYTES device array of the library); returns the tim_status code."""
    return load().tim_token_logprob_noalloc(h, W, targets, N, D, V, out_logp, out_lse, stream)


def tim_mismatch_stats(logp_train, logp_rollout, mask, seq_offsets, C, out: tim_mismatch_out,
                       stream) -> int:
    return load().tim_mismatch_stats(logp_train, logp_rollout, mask, seq_offsets, float(C),
                                     ctypes.byref(out), stream)


def tim_mismatch_fold(seq_records, num_seqs, batch_stats, stream) -> int:
    return load().tim_mismatch_fold(seq_records, int(num_seqs), batch_stats, stream)


def tim_tis_ppo(logp_theta, logp_old, logp_rollout, advantages, mask, seq_offsets, eps_low, eps_high, C,
                out: tim_ppo_out, stream) -> int:
    return load().tim_tis_ppo(logp_theta, logp_old, logp_rollout, advantages, mask, seq_offsets,
                              float(eps_low), float(eps_high), float(C), ctypes.byref(out), stream)


def tim_token_logprob_backward(h, W, targets, grad_logp, lse, N, D, V, temperature, dh, dW, accumulate_dW,
                               stream) -> int:
    return load().tim_token_logprob_backward(h, W, targets, grad_logp, lse, N, D, V, float(temperature), dh, dW,
                                             int(accumulate_dW), stream)


def tim_split_weight_bytes(V, D) -> int:
    return load().tim_split_weight_bytes(V, D)


def tim_split_weight_fp32(W, V, D, W_split, stream) -> int:
    return load().tim_split_weight_fp32(W, V, D, W_split, stream)


def tim_token_logprob_fp32_head(h, W_split, targets, N, D, V, temperature, out_logp, out_lse, stream) -> int:
    return load().tim_token_logprob_fp32_head(h, W_split, targets, N, D, V, float(temperature), out_logp,
                                              out_lse, stream)


def tim_mismatch_monitor(logp_train, logp_rollout, mask, N, tau_tok, token_reject, out, stream) -> int:
    return load().tim_mismatch_monitor(logp_train, logp_rollout, mask, N, float(tau_tok), token_reject, out,
                                       stream)


def tim_process_logits(logits, dtype, N, V, stride, rules, out, out_dtype, out_stride, stream) -> int:
    """C ABI; rules is a tim_logits_rules or None."""
    return load().tim_process_logits(logits, dtype, N, V, stride, rules, out, out_dtype, out_stride, stream)


def tim_processed_logprob(logits, dtype, N, V, stride, rules, targets, out_logp, out_lse, stream) -> int:
    return load().tim_processed_logprob(logits, dtype, N, V, stride, rules, targets, out_logp, out_lse, stream)


def tim_processed_logprob_backward(logits, dtype, N, V, stride, rules, targets, grad_logp, lse, dlogits,
                                   dlogits_stride, stream) -> int:
    return load().tim_processed_logprob_backward(logits, dtype, N, V, stride, rules, targets, grad_logp, lse, dlogits,
                                                 dlogits_stride, stream)


def tim_distill_topk(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K, temperature, loss, lse,
                     lse_tail, stream) -> int:
    return load().tim_distill_topk(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                                   temperature, loss, lse, lse_tail, stream)


def tim_distill_topk_backward(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K, temperature,
                              grad_loss, lse, lse_tail, dlogits, dlogits_stride, stream) -> int:
    return load().tim_distill_topk_backward(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                                            temperature, grad_loss, lse, lse_tail, dlogits, dlogits_stride, stream)


def tim_distill_topk_step(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K, temperature,
                          grad_loss, loss, lse, lse_tail, dlogits, dlogits_stride, stream) -> int:
    return load().tim_distill_topk_step(logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                                        temperature, grad_loss, loss, lse, lse_tail, dlogits, dlogits_stride, stream)


def tim_selftest_wait_timeout(budget_us, stream) -> int:
    """C ABI: a kernel waits on a barrier nothing arrives on, for budget_us
    microseconds, and records TIM_ERR_TIMEOUT (no fault; see include/tim.h)."""
    return load().tim_selftest_wait_timeout(budget_us, stream)


def tim_check(stream) -> int:
    return load().tim_check(stream)


def tim_last_error() -> str:
    return load().tim_last_error().decode(errors="replace")


def tim_version() -> int:
    return load().tim_version()


def tim_debug_build() -> int:
    """1 when calls go to the checked build (libtim_debug.so), else 0."""
    return load().tim_debug_build()


def tim_debug_violation(stream=None):
    """The first violation the checked build's kernels recorded since the last
    call, as (check name, index, value bits), cleared on read; ("none", 0, 0)
    if none (always so in libtim.so).  Synchronises the stream."""
    import torch
    out = (ctypes.c_int64 * 4)()
    s = 0 if stream is None and not torch.cuda.is_available() else _stream_handle(stream, None)
    _raise_if(load().tim_debug_violation(out, s))
    return CHECKS.get(int(out[0]), str(int(out[0]))), int(out[1]), int(out[2])


def _raise_if(rc: int):
    if rc != TIM_OK:
        raise TimError(rc, tim_last_error())


# ----------------------------------------------------------------------------- torch wrappers
def _stream_handle(stream, device):
    import torch
    s = torch.cuda.current_stream(device) if stream is None else stream
    return s.cuda_stream


def _need(t, name, dtype, ndim, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s must be %d-D" % (name, ndim))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _need_out(t, name, dtype, shape, device):
    """An output buffer the kernels write in full: exact dtype, shape, device,
    contiguous (a shorter buffer would be written past its end)."""
    _need(t, name, dtype, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


_modules = None


def _torch():
    """(torch, torch.Tensor, the raw handle of a device's current stream): looked up
    once; a decoding step pays for every look-up of its calls."""
    global _modules
    if _modules is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            def raw(index):
                return torch.cuda.current_stream(index).cuda_stream
        _modules = (torch, torch.Tensor, raw)
    return _modules


def _need_array(t, name, dtype, shape, device):
    """_need_out with its whole check in one condition where it holds."""
    if not (t.__class__ is _torch()[1] and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _need_out(t, name, dtype, shape, device)
    return t.data_ptr()


def _new(shape, dtype, device, stream):
    """An output buffer in the memory of the stream that will write it (given back
    while that stream still works on it, it is not handed to another)."""
    torch = _torch()[0]
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_output(t, name, N, device, stream):
    """An fp32 [N] output and its address: the caller's, checked, or a new one."""
    f32 = _torch()[0].float32
    if t is not None:
        return t, _need_array(t, name, f32, (N,), device)
    t = _new(N, f32, device, stream)
    return t, t.data_ptr()


def _launch(function, device, stream, *args):
    """Calls a C entry point on `device` and `stream` (None: the current one)."""
    torch, _, raw = _torch()
    if torch.cuda.current_device() == device.index:
        rc = function(*args, raw(device.index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = function(*args, raw(device.index) if stream is None else stream.cuda_stream)
    if rc != TIM_OK:
        _raise_if(rc)


def token_logprob(h, W, targets, out_logp=None, out_lse=None, stream=None, temperature: float = 1.0):
    """(logp [N] fp32, lse [N] fp32) for bf16 h [N, D], bf16 W [V, D], int32 targets [N]:
    log softmax(h W^T / temperature) at the targets (temperature 1: raw logits)."""
    import torch
    _need(h, "h", torch.bfloat16, 2)
    dev = h.device
    _need(W, "W", torch.bfloat16, 2, dev)
    _need(targets, "targets", torch.int32, 1, dev)
    N, D = h.shape
    V = W.shape[0]
    if W.shape[1] != D or targets.shape[0] != N:
        raise ValueError("shape mismatch: h %s, W %s, targets %s" % (tuple(h.shape), tuple(W.shape),
                                                                       tuple(targets.shape)))
    if out_logp is None:
        out_logp = torch.empty(N, dtype=torch.float32, device=dev)
    if out_lse is None:
        out_lse = torch.empty(N, dtype=torch.float32, device=dev)
    _need_out(out_logp, "out_logp", torch.float32, (N,), dev)
    _need_out(out_lse, "out_lse", torch.float32, (N,), dev)
    with torch.cuda.device(dev):
        if temperature == 1.0:
            rc = tim_token_logprob(h.data_ptr(), W.data_ptr(), targets.data_ptr(), N, D, V,
                                   out_logp.data_ptr(), out_lse.data_ptr(), _stream_handle(stream, dev))
        else:
            rc = tim_token_logprob_temperature(h.data_ptr(), W.data_ptr(), targets.data_ptr(), N, D, V,
                                               temperature, out_logp.data_ptr(), out_lse.data_ptr(),
                                               _stream_handle(stream, dev))
    _raise_if(rc)
    return out_logp, out_lse


def token_logprob_backward(h, W, targets, grad_logp, lse, temperature: float = 1.0, dh=None, dW=None,
                           accumulate_dW: bool = False, stream=None):
    """(dh fp32 [N, D], dW fp32 [V, D]): gradients of sum_t grad_logp_t l_t
    for bf16 h [N, D], bf16 W [V, D], int32 targets, the forward's lse [N]
    at the same temperature.  With accumulate_dW the gradient is added to dW."""
    import torch
    _need(h, "h", torch.bfloat16, 2)
    dev = h.device
    _need(W, "W", torch.bfloat16, 2, dev)
    _need(targets, "targets", torch.int32, 1, dev)
    _need(grad_logp, "grad_logp", torch.float32, 1, dev)
    _need(lse, "lse", torch.float32, 1, dev)
    N, D = h.shape
    V = W.shape[0]
    if W.shape[1] != D or any(t.shape[0] != N for t in (targets, grad_logp, lse)):
        raise ValueError("shape mismatch")
    if dh is None:
        dh = torch.empty((N, D), dtype=torch.float32, device=dev)
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs dW")
        dW = torch.empty((V, D), dtype=torch.float32, device=dev)
    _need_out(dh, "dh", torch.float32, (N, D), dev)
    _need_out(dW, "dW", torch.float32, (V, D), dev)
    with torch.cuda.device(dev):
        rc = tim_token_logprob_backward(h.data_ptr(), W.data_ptr(), targets.data_ptr(), grad_logp.data_ptr(),
                                        lse.data_ptr(), N, D, V, temperature, dh.data_ptr(), dW.data_ptr(),
                                        accumulate_dW, _stream_handle(stream, dev))
    _raise_if(rc)
    return dh, dW


def split_weight_fp32(W, out=None, stream=None):
    """fp32 W [V, D] -> its three bf16 parts, a bf16 tensor [V, 3 * Dp]
    (Dp = D rounded up to 64): the operand of token_logprob_fp32_head."""
    import torch
    _need(W, "W", torch.float32, 2)
    dev = W.device
    V, D = W.shape
    nbytes = tim_split_weight_bytes(V, D)
    if nbytes < 0:
        raise ValueError("W shape %s out of range" % (tuple(W.shape),))
    cols = nbytes // (2 * V)
    if out is None:
        out = torch.empty((V, cols), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, 2, dev)
    if tuple(out.shape) != (V, cols):
        raise ValueError("out must be [%d, %d]" % (V, cols))
    with torch.cuda.device(dev):
        rc = tim_split_weight_fp32(W.data_ptr(), V, D, out.data_ptr(), _stream_handle(stream, dev))
    _raise_if(rc)
    return out


def token_logprob_fp32_head(h, W_split, targets, out_logp=None, out_lse=None, stream=None,
                            temperature: float = 1.0):
    """(logp, lse) fp32 [N] of log softmax(h W^T / temperature) at the targets
    with fp32 weights W, given as split_weight_fp32(W); h bf16 [N, D]."""
    import torch
    _need(h, "h", torch.bfloat16, 2)
    dev = h.device
    _need(W_split, "W_split", torch.bfloat16, 2, dev)
    _need(targets, "targets", torch.int32, 1, dev)
    N, D = h.shape
    V = W_split.shape[0]
    if tim_split_weight_bytes(V, D) != W_split.numel() * 2 or targets.shape[0] != N:
        raise ValueError("shape mismatch: h %s, W_split %s, targets %s"
                         % (tuple(h.shape), tuple(W_split.shape), tuple(targets.shape)))
    if out_logp is None:
        out_logp = torch.empty(N, dtype=torch.float32, device=dev)
    if out_lse is None:
        out_lse = torch.empty(N, dtype=torch.float32, device=dev)
    _need_out(out_logp, "out_logp", torch.float32, (N,), dev)
    _need_out(out_lse, "out_lse", torch.float32, (N,), dev)
    with torch.cuda.device(dev):
        rc = tim_token_logprob_fp32_head(h.data_ptr(), W_split.data_ptr(), targets.data_ptr(), N, D, V,
                                         temperature, out_logp.data_ptr(), out_lse.data_ptr(),
                                         _stream_handle(stream, dev))
    _raise_if(rc)
    return out_logp, out_lse


def mismatch_stats(logp_train, logp_rollout, mask, seq_offsets, C: float = 2.0,
                   tau_seq: float = math.nan, seq_estimator: int = 3, token_weight: bool = False,
                   stream=None, out=None, seq_records: bool = False):
    """Mismatch statistics of packed sequences.

    logp_train, logp_rollout fp32 [N]; mask bool/uint8 [N]; seq_offsets int32 [S + 1].
    Returns a dict: seq_stats fp32 [S, 12] (SEQ_FIELDS), seq_flags int32 [S],
    batch fp64 [20] (BATCH_FIELDS), token_weight fp32 [N] or None, and with
    seq_records=True seq_records int32 [S, SEQ_RECORD_WORDS] (the records the
    batch record is folded from; see mismatch_fold).
    """
    import torch
    _need(logp_train, "logp_train", torch.float32, 1)
    dev = logp_train.device
    _need(logp_rollout, "logp_rollout", torch.float32, 1, dev)
    _need(mask, "mask", (torch.uint8, torch.bool), 1, dev)
    _need(seq_offsets, "seq_offsets", torch.int32, 1, dev)
    N = logp_train.shape[0]
    S = seq_offsets.shape[0] - 1
    if logp_rollout.shape[0] != N or mask.shape[0] != N or S < 0:
        raise ValueError("shape mismatch")
    if out is None:
        out = {
            "seq_stats": torch.empty((S, len(SEQ_FIELDS)), dtype=torch.float32, device=dev),
            "seq_flags": torch.empty(S, dtype=torch.int32, device=dev),
            "batch": torch.empty(len(BATCH_FIELDS), dtype=torch.float64, device=dev),
            "token_weight": torch.empty(N, dtype=torch.float32, device=dev) if token_weight else None,
            "seq_records": torch.empty((S, SEQ_RECORD_WORDS), dtype=torch.int32, device=dev)
            if seq_records else None,
        }
    _need_out(out["seq_stats"], "seq_stats", torch.float32, (S, len(SEQ_FIELDS)), dev)
    _need_out(out["seq_flags"], "seq_flags", torch.int32, (S,), dev)
    _need_out(out["batch"], "batch", torch.float64, (len(BATCH_FIELDS),), dev)
    if out.get("token_weight") is not None:
        _need_out(out["token_weight"], "token_weight", torch.float32, (N,), dev)
    if out.get("seq_records") is not None:
        _need_out(out["seq_records"], "seq_records", torch.int32, (S, SEQ_RECORD_WORDS), dev)
        if out["seq_records"].data_ptr() % 16:
            raise ValueError("seq_records must be 16-byte aligned")
    d = tim_mismatch_out()
    d.num_seqs = S
    d.num_tokens = N
    d.tau_seq = float(tau_seq)
    d.seq_estimator = int(seq_estimator)
    d.token_weight = out["token_weight"].data_ptr() if out.get("token_weight") is not None else None
    d.seq_stats = out["seq_stats"].data_ptr()
    d.seq_flags = out["seq_flags"].data_ptr()
    d.batch_stats = out["batch"].data_ptr()
    d.seq_records = out["seq_records"].data_ptr() if out.get("seq_records") is not None else None
    with torch.cuda.device(dev):
        rc = tim_mismatch_stats(logp_train.data_ptr(), logp_rollout.data_ptr(), mask.data_ptr(),
                                seq_offsets.data_ptr(), C, d, _stream_handle(stream, dev))
    _raise_if(rc)
    return out


def mismatch_fold(seq_records, out=None, stream=None):
    """The batch record (fp64 [20], BATCH_FIELDS) of a batch scored in parts:
    the parts' seq_records (int32 [S_part, SEQ_RECORD_WORDS] each, from
    mismatch_stats(..., seq_records=True)) concatenated in the batch's sequence
    order.  Bit-identical to mismatch_stats over the whole batch."""
    import torch
    _need(seq_records, "seq_records", torch.int32, 2)
    dev = seq_records.device
    if seq_records.shape[1] != SEQ_RECORD_WORDS:
        raise ValueError("seq_records must have %d columns" % SEQ_RECORD_WORDS)
    if seq_records.data_ptr() % 16:
        raise ValueError("seq_records must be 16-byte aligned")
    if out is None:
        out = torch.empty(len(BATCH_FIELDS), dtype=torch.float64, device=dev)
    _need_out(out, "out", torch.float64, (len(BATCH_FIELDS),), dev)
    with torch.cuda.device(dev):
        rc = tim_mismatch_fold(seq_records.data_ptr(), seq_records.shape[0], out.data_ptr(),
                               _stream_handle(stream, dev))
    _raise_if(rc)
    return out


def mismatch_monitor(logp_train, logp_rollout, mask, tau_tok: float, token_reject: bool = True, stream=None,
                     out=None):
    """Mismatch monitor over the used tokens: batch fp64 [7] (MONITOR_FIELDS:
    n_used, p95 |delta|, ratio quantiles 0.01 / 0.5 / 0.99, n_extreme,
    frac_extreme) and token_reject uint8 [N] (None unless requested)."""
    import torch
    _need(logp_train, "logp_train", torch.float32, 1)
    dev = logp_train.device
    _need(logp_rollout, "logp_rollout", torch.float32, 1, dev)
    _need(mask, "mask", (torch.uint8, torch.bool), 1, dev)
    N = logp_train.shape[0]
    if logp_rollout.shape[0] != N or mask.shape[0] != N:
        raise ValueError("shape mismatch")
    if out is None:
        out = {"batch": torch.empty(len(MONITOR_FIELDS), dtype=torch.float64, device=dev),
               "token_reject": torch.empty(N, dtype=torch.uint8, device=dev) if token_reject else None}
    _need_out(out["batch"], "batch", torch.float64, (len(MONITOR_FIELDS),), dev)
    rej = out.get("token_reject")
    if rej is not None:
        _need_out(rej, "token_reject", torch.uint8, (N,), dev)
    with torch.cuda.device(dev):
        rc = tim_mismatch_monitor(logp_train.data_ptr(), logp_rollout.data_ptr(), mask.data_ptr(), N, tau_tok,
                                  None if rej is None else rej.data_ptr(), out["batch"].data_ptr(),
                                  _stream_handle(stream, dev))
    _raise_if(rc)
    return out


def tis_ppo(logp_theta, logp_old, logp_rollout, advantages, mask, seq_offsets, eps_low: float = 0.2,
            eps_high: float = 0.2, C: float = 2.0, token_outputs: bool = True, stream=None, out=None):
    """TIS-weighted PPO clipped surrogate of packed sequences.

    logp_theta, logp_old, logp_rollout, advantages fp32 [N]; mask bool/uint8 [N];
    seq_offsets int32 [S + 1].  Returns a dict: token_loss, token_grad fp32 [N]
    (None unless token_outputs), seq_loss fp32 [S], batch fp64 [9] (PPO_FIELDS).
    """
    import torch
    _need(logp_theta, "logp_theta", torch.float32, 1)
    dev = logp_theta.device
    for name, t in (("logp_old", logp_old), ("logp_rollout", logp_rollout), ("advantages", advantages)):
        _need(t, name, torch.float32, 1, dev)
    _need(mask, "mask", (torch.uint8, torch.bool), 1, dev)
    _need(seq_offsets, "seq_offsets", torch.int32, 1, dev)
    N = logp_theta.shape[0]
    S = seq_offsets.shape[0] - 1
    if any(t.shape[0] != N for t in (logp_old, logp_rollout, advantages, mask)) or S < 0:
        raise ValueError("shape mismatch")
    if out is None:
        out = {
            "token_loss": torch.empty(N, dtype=torch.float32, device=dev) if token_outputs else None,
            "token_grad": torch.empty(N, dtype=torch.float32, device=dev) if token_outputs else None,
            "seq_loss": torch.empty(S, dtype=torch.float32, device=dev),
            "batch": torch.empty(len(PPO_FIELDS), dtype=torch.float64, device=dev),
        }
    for name in ("token_loss", "token_grad"):
        if out.get(name) is not None:
            _need_out(out[name], name, torch.float32, (N,), dev)
    _need_out(out["seq_loss"], "seq_loss", torch.float32, (S,), dev)
    _need_out(out["batch"], "batch", torch.float64, (len(PPO_FIELDS),), dev)
    d = tim_ppo_out()
    d.num_seqs = S
    d.num_tokens = N
    d.token_loss = out["token_loss"].data_ptr() if out.get("token_loss") is not None else None
    d.token_grad = out["token_grad"].data_ptr() if out.get("token_grad") is not None else None
    d.seq_loss = out["seq_loss"].data_ptr()
    d.batch_stats = out["batch"].data_ptr()
    with torch.cuda.device(dev):
        rc = tim_tis_ppo(logp_theta.data_ptr(), logp_old.data_ptr(), logp_rollout.data_ptr(),
                         advantages.data_ptr(), mask.data_ptr(), seq_offsets.data_ptr(), eps_low, eps_high, C,
                         d, _stream_handle(stream, dev))
    _raise_if(rc)
    return out


# ----------------------------------------------------------------------------- a head's logits
@dataclasses.dataclass
class LogitsRules:
    """The sampler's rules, row by row (tim_logits_rules in include/tim.h); None
    leaves a rule out.  All on the logits' device and contiguous: temperature,
    repetition, presence, frequency fp32 [N]; history int32 [H] with history_spans
    int32 [N, 3] (begin, first generated token, end); bias_offsets int32 [N + 1]
    with bias_ids int32 and bias_values fp32 [B] (a row's ids ascending); allowed
    int32 or uint32 [R, ceil(V / 32) or more] bits, with allowed_rows int32 [N]
    (a row of `allowed`, negative = none) or R >= N."""
    temperature: object = None
    repetition: object = None
    presence: object = None
    frequency: object = None
    history: object = None
    history_spans: object = None
    bias_offsets: object = None
    bias_ids: object = None
    bias_values: object = None
    allowed: object = None
    allowed_rows: object = None

    def struct(self, N: int, V: int, device):
        """The C struct, after checking every tensor against N rows of V logits."""
        torch = _torch()[0]
        f32, i32, rows = torch.float32, torch.int32, (N,)
        r = tim_logits_rules()
        if self.temperature is not None:
            r.temperature = _need_array(self.temperature, "temperature", f32, rows, device)
        if self.repetition is not None:
            r.repetition = _need_array(self.repetition, "repetition", f32, rows, device)
        if self.presence is not None:
            r.presence = _need_array(self.presence, "presence", f32, rows, device)
        if self.frequency is not None:
            r.frequency = _need_array(self.frequency, "frequency", f32, rows, device)
        if (self.history is None) != (self.history_spans is None):
            raise ValueError("history and history_spans go together")
        if self.history is not None:
            r.num_history = _list_size(self.history, "history")
            r.history = _need_array(self.history, "history", i32, (r.num_history,), device)
            r.history_spans = _need_array(self.history_spans, "history_spans", i32, (N, 3), device)
        if self.bias_offsets is not None or self.bias_ids is not None or self.bias_values is not None:
            if self.bias_offsets is None or self.bias_ids is None or self.bias_values is None:
                raise ValueError("bias_offsets, bias_ids and bias_values go together")
            r.num_bias = _list_size(self.bias_ids, "bias_ids")
            r.bias_offsets = _need_array(self.bias_offsets, "bias_offsets", i32, (N + 1,), device)
            r.bias_ids = _need_array(self.bias_ids, "bias_ids", i32, (r.num_bias,), device)
            r.bias_values = _need_array(self.bias_values, "bias_values", f32, (r.num_bias,), device)
        if self.allowed is not None:
            _need(self.allowed, "allowed", (i32, torch.uint32), 2, device)
            R, words = self.allowed.shape
            if words < (V + 31) // 32:
                raise ValueError("allowed must have at least %d words a row" % ((V + 31) // 32))
            r.allowed, r.allowed_stride, r.num_allowed = self.allowed.data_ptr(), words, min(R, 2 ** 31 - 1)
            if self.allowed_rows is not None:
                r.allowed_rows = _need_array(self.allowed_rows, "allowed_rows", i32, rows, device)
            elif R < N:
                raise ValueError("allowed has fewer rows than the logits: give allowed_rows")
        elif self.allowed_rows is not None:
            raise ValueError("allowed_rows without allowed")
        return r


def _list_size(t, name):
    if not isinstance(t, _torch()[1]):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != 1:
        raise ValueError("%s must be 1-D" % name)
    if t.shape[0] >= 2 ** 30:
        raise ValueError("%s must have fewer than 2^30 entries" % name)
    return t.shape[0]


_dtype_codes = {}


def _dtype_code(dtype):
    if not _dtype_codes:
        torch = _torch()[0]
        _dtype_codes.update({torch.float32: TIM_F32, torch.bfloat16: TIM_BF16, torch.float16: TIM_F16})
    return _dtype_codes.get(dtype)


def _need_logits(t, name, dtype=None, device=None, shape=None):
    """Rows of logits: 2-D, a row's elements adjacent, rows any stride >= V apart.
    Returns (address, type code, N, V, stride)."""
    if not isinstance(t, _torch()[1]):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    code = _dtype_code(t.dtype)
    if code is None or (dtype is not None and t.dtype is not dtype):
        raise TypeError("%s must have dtype %s, got %s"
                        % (name, "float32, bfloat16 or float16" if dtype is None else dtype, t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    N, V = t.shape
    if shape is not None and (N, V) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, (N, V)))
    if V < 1:
        raise ValueError("%s must have at least one column" % name)
    stride, step = t.stride()
    if V > 1 and step != 1:
        raise ValueError("a row of %s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if N <= 1:
        stride = V
    elif stride < V:
        raise ValueError("the rows of %s must not overlap" % name)
    return t.data_ptr(), code, N, V, stride


def _rules_struct(rules, N, V, dev):
    return None if rules is None else ctypes.byref(rules.struct(N, V, dev))


def packed_spans(seq_offsets, prompt_lens, num_tokens: int):
    """history_spans (int32 [T, 3], T = num_tokens = seq_offsets[S]) of packed
    sequences for LogitsRules, with the packed input tokens as the history:
    position t of sequence s has read the tokens from seq_offsets[s] up to its
    own, the first prompt_lens[s] of them the prompt.  seq_offsets int32 [S + 1],
    prompt_lens int32 [S], on one device."""
    import torch
    off = seq_offsets.long()
    t = torch.arange(num_tokens, device=off.device)
    s = torch.bucketize(t, off[1:], right=True).clamp_(max=max(0, off.shape[0] - 2))
    begin, end = off[s], t + 1
    return torch.stack([begin, torch.minimum(begin + prompt_lens.long()[s], end), end], 1).to(torch.int32)


def process_logits(logits, rules, out=None, out_dtype=None, stream=None):
    """The processed logits [N, V] (y in include/tim.h) of fp32, bf16 or fp16
    logits under `rules` (a LogitsRules or None), in the logits' type or fp32.
    out may be the logits themselves."""
    head = _need_logits(logits, "logits")
    dev, N, V = logits.device, head[2], head[3]
    if out is None:
        out = _new((N, V), out_dtype or logits.dtype, dev, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out must have dtype %s, got %s" % (out_dtype, out.dtype))
    address, code, _, _, stride = _need_logits(out, "out", None, dev, (N, V))
    if code != head[1] and code != TIM_F32:
        raise TypeError("out must have the logits' dtype or float32, got %s" % out.dtype)
    _launch(tim_process_logits, dev, stream, *head, _rules_struct(rules, N, V, dev), address, code, stride)
    return out


def processed_logprob(logits, rules, targets, out_logp=None, out_lse=None, stream=None):
    """(logp [N] fp32, lse [N] fp32) of the int32 targets [N] under the processed
    logits, which are not written."""
    head = _need_logits(logits, "logits")
    dev, N, V = logits.device, head[2], head[3]
    torch = _torch()[0]
    t = _need_array(targets, "targets", torch.int32, (N,), dev)
    out_logp, logp_ptr = _row_output(out_logp, "out_logp", N, dev, stream)
    out_lse, lse_ptr = _row_output(out_lse, "out_lse", N, dev, stream)
    _launch(tim_processed_logprob, dev, stream, *head, _rules_struct(rules, N, V, dev), t, logp_ptr, lse_ptr)
    return out_logp, out_lse


def processed_logprob_backward(logits, rules, targets, grad_logp, lse, dlogits=None, stream=None):
    """The gradient [N, V], in the logits' type, of sum_i grad_logp_i logp_i with
    respect to the raw logits, from the forward's lse.  dlogits may be the
    logits themselves."""
    head = _need_logits(logits, "logits")
    dev, N, V = logits.device, head[2], head[3]
    torch = _torch()[0]
    f32 = torch.float32
    t = _need_array(targets, "targets", torch.int32, (N,), dev)
    g = _need_array(grad_logp, "grad_logp", f32, (N,), dev)
    lse_ptr = _need_array(lse, "lse", f32, (N,), dev)
    if dlogits is None:
        dlogits = _new((N, V), logits.dtype, dev, stream)
    out = _need_logits(dlogits, "dlogits", logits.dtype, dev, (N, V))
    _launch(tim_processed_logprob_backward, dev, stream, *head, _rules_struct(rules, N, V, dev), t, g, lse_ptr,
            out[0], out[4])
    return dlogits


def _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse, temperature):
    """(C arguments up to the temperature, N, V, device)."""
    torch = _torch()[0]
    head = _need_logits(logits, "logits")
    dev, N, V = logits.device, head[2], head[3]
    _need(teacher_ids, "teacher_ids", torch.int32, 2, dev)
    K = teacher_ids.shape[1]
    if teacher_ids.shape[0] != N or not 1 <= K <= DISTILL_MAX_K:
        raise ValueError("teacher_ids must be [%d, 1 .. %d], got %s" % (N, DISTILL_MAX_K, tuple(teacher_ids.shape)))
    t = _need_array(teacher_logits, "teacher_logits", torch.float32, (N, K), dev)
    lse = None if teacher_lse is None else _need_array(teacher_lse, "teacher_lse", torch.float32, (N,), dev)
    return (*head, teacher_ids.data_ptr(), t, lse, K, float(temperature)), N, V, dev


def _distill_rows(out, N, tail, dev, stream):
    """(dict of the row outputs, their addresses)."""
    given = {} if out is None else out
    loss, loss_ptr = _row_output(given.get("loss"), "loss", N, dev, stream)
    lse, lse_ptr = _row_output(given.get("lse"), "lse", N, dev, stream)
    rest, rest_ptr = _row_output(given.get("lse_tail"), "lse_tail", N, dev, stream) if tail else (None, None)
    return {**given, "loss": loss, "lse": lse, "lse_tail": rest}, (loss_ptr, lse_ptr, rest_ptr)


def distill_topk(logits, teacher_ids, teacher_logits, teacher_lse=None, temperature: float = 1.0, out=None,
                 stream=None):
    """Distillation loss of fp32, bf16 or fp16 logits [N, V] from a teacher's top
    logits: teacher_ids int32 [N, K] (an id outside [0, V) is an empty entry),
    teacher_logits fp32 [N, K], and teacher_lse fp32 [N] where the teacher's mass
    outside its list is one more outcome.  Returns a dict: loss, lse fp32 [N] and
    lse_tail (fp32 [N] with teacher_lse, else None)."""
    args, N, _, dev = _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    out, rows = _distill_rows(out, N, teacher_lse is not None, dev, stream)
    _launch(tim_distill_topk, dev, stream, *args, *rows)
    return out


def distill_topk_backward(logits, teacher_ids, teacher_logits, grad_loss, lse, lse_tail=None, teacher_lse=None,
                          temperature: float = 1.0, dlogits=None, stream=None):
    """The gradient [N, V], in the logits' type, of sum_i grad_loss_i loss_i, from
    the forward's lse and (with teacher_lse) lse_tail.  dlogits may be the logits
    themselves."""
    torch = _torch()[0]
    f32 = torch.float32
    args, N, V, dev = _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    g = _need_array(grad_loss, "grad_loss", f32, (N,), dev)
    lse_ptr = _need_array(lse, "lse", f32, (N,), dev)
    if (lse_tail is None) != (teacher_lse is None):
        raise ValueError("lse_tail and teacher_lse go together")
    tail = None if lse_tail is None else _need_array(lse_tail, "lse_tail", f32, (N,), dev)
    if dlogits is None:
        dlogits = _new((N, V), logits.dtype, dev, stream)
    out = _need_logits(dlogits, "dlogits", logits.dtype, dev, (N, V))
    _launch(tim_distill_topk_backward, dev, stream, *args, g, lse_ptr, tail, out[0], out[4])
    return dlogits


def distill_topk_step(logits, teacher_ids, teacher_logits, grad_loss, teacher_lse=None, temperature: float = 1.0,
                      out=None, dlogits=None, stream=None):
    """distill_topk and its gradient in one call, for weights grad_loss fp32 [N]
    known beforehand: the dict of distill_topk with dlogits [N, V] added (which
    may be the logits themselves)."""
    torch = _torch()[0]
    args, N, V, dev = _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    g = _need_array(grad_loss, "grad_loss", torch.float32, (N,), dev)
    out, rows = _distill_rows(out, N, teacher_lse is not None, dev, stream)
    if dlogits is None:
        dlogits = _new((N, V), logits.dtype, dev, stream)
    d = _need_logits(dlogits, "dlogits", logits.dtype, dev, (N, V))
    out["dlogits"] = dlogits
    _launch(tim_distill_topk_step, dev, stream, *args, g, *rows, d[0], d[4])
    return out


def check(stream=None, device=None):
    """Synchronises the stream and raises TimError if a kernel recorded a status."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _raise_if(tim_check(_stream_handle(stream, dev)))
