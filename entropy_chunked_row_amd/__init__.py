"""Python binding of liblp.so: per-token log-probs, entropy and exact KL over a
large vocabulary on MI355X.

Functions carry the C names (include/lp.h).  This layer only marshals
arguments: it checks dtypes, layouts, the length of every per-row array
(T, or T x K for the K-target calls) and that every tensor sits on the main
operand's device, all before anything is launched; it allocates outputs and
workspace with torch (device memory is all torch is used for) and passes raw
pointers plus the current HIP stream.  Every number is computed by the HIP
kernels; if liblp.so is missing, every call raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

from . import _lib
from ._lib import LP_BF16, LP_FP16, LP_FP32, LPError, check, load

__all__ = [
    "lp_logprobs_entropy", "lp_lm_head_logprobs_entropy", "lp_lm_head_logprobs_entropy_backward",
    "lp_lm_head_workspace_bytes", "lp_kl_full_vocab", "lp_prob_diff", "lp_version", "lp_timing_enable",
    "lp_timing_read", "lp_timing_clock", "lp_logprobs_entropy_k", "lp_lm_head_logprobs_entropy_k",
    "lp_lm_head_logprobs_entropy_backward_k", "lp_prob_diff_stats", "lp_lm_head_kl_workspace_bytes",
    "lp_lm_head_kl", "lp_lm_head_kl_backward", "LogitRules", "lp_process_logits", "lp_processed_logprobs_entropy",
    "lp_processed_logprobs_entropy_backward", "lp_processed_workspace_bytes", "lp_embedding", "lp_embedding_backward",
    "lp_embedding_workspace_bytes", "lp_lm_head_w4_quantize", "lp_lm_head_w4_logits", "lp_top_logits",
    "lp_top_workspace_bytes", "lp_distill_top", "lp_distill_top_backward", "lp_distill_top_workspace_bytes",
    "lp_beam_select", "lp_beam_workspace_bytes", "lp_beam_reorder", "lp_lm_head_fp8_quantize", "lp_lm_head_fp8_logits",
    "lp_lm_head_fp8_workspace_bytes", "LPError", "load",
]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_dtype_codes = {}


def _dtype_code(t) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.bfloat16: LP_BF16, torch.float16: LP_FP16, torch.float32: LP_FP32})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported logits dtype {t.dtype}")
    return code


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(t, name):
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must be a device (GPU) tensor")


def _on(device, **tensors):
    """Every given tensor lives on `device` (checked after all shapes, so a
    wrong length is reported as such even for host tensors)."""
    for name, t in tensors.items():
        if t is None:
            continue
        _dev(t, name)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, name):
    """2-D tensor with unit stride along columns; returns its leading dimension."""
    stride, shape = t.stride(), t.shape
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return stride[0] if shape[0] > 1 else max(stride[0], shape[1])


def _vec(t, name, dtype=None, n=None):
    """Contiguous tensor of `dtype` (bool accepted for uint8) holding exactly
    `n` elements when n is given: a short per-row array would be read past
    its end by the kernels, so it is refused here."""
    if t is None:
        return None
    torch = _torch()
    if dtype is not None and t.dtype != dtype:
        if dtype == torch.uint8 and t.dtype == torch.bool:
            t = t.view(torch.uint8)
        else:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t


def _bf16_2d(t, name):
    torch = _torch()
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def lp_version() -> int:
    return load().lp_version()


def lp_timing_enable(on) -> None:
    """Start (clearing old records) or stop per-kernel HIP-event timing; 2 also
    samples the fused forward GEMM's shader clock (lp_timing_clock)."""
    load().lp_timing_enable(2 if on == 2 else (1 if on else 0))


def lp_timing_clock(kernel: str = "k_fwd_tile"):
    """(mean shader clock in MHz, workgroups sampled) of the last sampled launch."""
    import ctypes
    mhz = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    check("lp_timing_clock", load().lp_timing_clock(kernel.encode(), ctypes.byref(mhz), ctypes.byref(n)))
    return float(mhz.value), int(n.value)


def lp_timing_read(kernel: str):
    """(launches, total_ms) recorded for `kernel` since timing was enabled."""
    import ctypes
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    check("lp_timing_read", load().lp_timing_read(kernel.encode(), ctypes.byref(n), ctypes.byref(ms)))
    return int(n.value), float(ms.value)


def lp_logprobs_entropy(logits, targets, mask=None, temperature: float = 1.0, chunk_rows: int = -1, *,
                        want_entropy: bool = True, logprob=None, entropy=None, stream=None):
    """(logprob[T], entropy[T] or None) of model-precision logits [T, V]."""
    torch = _torch()
    lib = load()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [T, V]")
    T, V = logits.shape
    ld = _rows(logits, "logits")
    targets = _vec(targets, "targets", torch.int64, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    logprob = _vec(logprob, "logprob", torch.float32, T)
    entropy = _vec(entropy, "entropy", torch.float32, T)
    _on(logits.device, logits=logits, targets=targets, mask=mask, logprob=logprob, entropy=entropy)
    if logprob is None:
        logprob = torch.empty(T, dtype=torch.float32, device=logits.device)
    if want_entropy and entropy is None:
        entropy = torch.empty(T, dtype=torch.float32, device=logits.device)
    st = lib.lp_logprobs_entropy(_ptr(logits), _dtype_code(logits), T, V, ld, _ptr(targets), _ptr(mask),
                                 float(temperature), int(chunk_rows), _ptr(logprob), _ptr(entropy), _stream(stream))
    check("lp_logprobs_entropy", st)
    return logprob, entropy


def lp_lm_head_workspace_bytes(T: int, h: int, V: int, tile_rows: int, backward: bool) -> int:
    return int(load().lp_lm_head_workspace_bytes(T, h, V, tile_rows, 1 if backward else 0))


def _workspace(nbytes: int, device, workspace):
    """(tensor, size in bytes): the caller's workspace after checks, or a new one."""
    torch = _torch()
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        _on(device, workspace=workspace)
        size = workspace.numel() * workspace.element_size()
        if size < nbytes:
            raise ValueError(f"workspace too small: {size} bytes, {nbytes} needed")
        return workspace, size
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    return ws, ws.numel()


def _lm_head_operands(hidden, weight):
    """(T, h, V) of bf16 hidden [T, h] and weight [V, h]."""
    _bf16_2d(hidden, "hidden")
    _bf16_2d(weight, "weight")
    T, h = hidden.shape
    V, h2 = weight.shape
    if h2 != h:
        raise ValueError("hidden and weight disagree on h")
    return T, h, V


def lp_lm_head_logprobs_entropy(hidden, weight, targets, mask=None, temperature: float = 1.0,
                                tile_rows: int = 4096, *, want_entropy: bool = True, want_lse: bool = True,
                                workspace=None, stream=None):
    """(logprob, entropy, lse) of softmax(hidden @ weight^T / temperature); bf16 hidden [T, h], weight [V, h]."""
    torch = _torch()
    lib = load()
    T, h, V = _lm_head_operands(hidden, weight)
    ld_h, ld_w = _rows(hidden, "hidden"), _rows(weight, "weight")
    targets = _vec(targets, "targets", torch.int64, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    dev = hidden.device
    _on(dev, hidden=hidden, weight=weight, targets=targets, mask=mask)
    lp = torch.empty(T, dtype=torch.float32, device=dev)
    H = torch.empty(T, dtype=torch.float32, device=dev) if want_entropy else None
    lse = torch.empty(T, dtype=torch.float32, device=dev) if want_lse else None
    ws, ws_bytes = _workspace(lp_lm_head_workspace_bytes(T, h, V, tile_rows, False), dev, workspace)
    st = lib.lp_lm_head_logprobs_entropy(_ptr(hidden), ld_h, _ptr(weight), ld_w, T, h, V, _ptr(targets), _ptr(mask),
                                         float(temperature), int(tile_rows), _ptr(lp), _ptr(H), _ptr(lse), _ptr(ws),
                                         ws_bytes, _stream(stream))
    check("lp_lm_head_logprobs_entropy", st)
    return lp, H, lse


def lp_lm_head_logprobs_entropy_backward(hidden, weight, targets, mask, temperature: float, tile_rows: int,
                                         lse, entropy, grad_logprob, grad_entropy=None, *,
                                         need_grad_hidden: bool = True, need_grad_weight: bool = True,
                                         workspace=None, stream=None) -> Tuple:
    """(grad_hidden fp32 [T, h] or None, grad_weight fp32 [V, h] or None)."""
    torch = _torch()
    lib = load()
    T, h, V = _lm_head_operands(hidden, weight)
    ld_h, ld_w = _rows(hidden, "hidden"), _rows(weight, "weight")
    targets = _vec(targets, "targets", torch.int64, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    lse = _vec(lse, "lse", torch.float32, T)
    entropy = _vec(entropy, "entropy", torch.float32, T)
    grad_logprob = _vec(grad_logprob, "grad_logprob", torch.float32, T)
    grad_entropy = _vec(grad_entropy, "grad_entropy", torch.float32, T)
    dev = hidden.device
    _on(dev, hidden=hidden, weight=weight, targets=targets, mask=mask, lse=lse, entropy=entropy,
        grad_logprob=grad_logprob, grad_entropy=grad_entropy)
    dH = torch.empty((T, h), dtype=torch.float32, device=dev) if need_grad_hidden else None
    dW = torch.empty((V, h), dtype=torch.float32, device=dev) if need_grad_weight else None
    ws, ws_bytes = _workspace(lp_lm_head_workspace_bytes(T, h, V, tile_rows, True), dev, workspace)
    st = lib.lp_lm_head_logprobs_entropy_backward(
        _ptr(hidden), ld_h, _ptr(weight), ld_w, T, h, V, _ptr(targets), _ptr(mask), float(temperature),
        int(tile_rows), _ptr(lse), _ptr(entropy), _ptr(grad_logprob), _ptr(grad_entropy), _ptr(dH), _ptr(dW),
        _ptr(ws), ws_bytes, _stream(stream))
    check("lp_lm_head_logprobs_entropy_backward", st)
    return dH, dW


def lp_kl_full_vocab(student, teacher, targets=None, diff_mask=None, *, want_target_logprobs: bool = True,
                     stream=None):
    """(kl, lp_student, lp_teacher, prob_diff); the last three are None without targets."""
    torch = _torch()
    lib = load()
    if student.dtype != teacher.dtype or student.shape != teacher.shape or student.dim() != 2:
        raise ValueError("student and teacher must be 2-D with the same dtype and shape")
    T, V = student.shape
    ld_s, ld_t = _rows(student, "student"), _rows(teacher, "teacher")
    targets = _vec(targets, "targets", torch.int64, T)
    diff_mask = _vec(diff_mask, "diff_mask", torch.uint8, T)
    dev = student.device
    _on(dev, student=student, teacher=teacher, targets=targets, diff_mask=diff_mask)
    kl = torch.empty(T, dtype=torch.float32, device=dev)
    lps = lpt = diff = None
    if targets is not None and want_target_logprobs:
        lps = torch.empty(T, dtype=torch.float32, device=dev)
        lpt = torch.empty(T, dtype=torch.float32, device=dev)
        diff = torch.empty(T, dtype=torch.float32, device=dev)
    st = lib.lp_kl_full_vocab(_ptr(student), _ptr(teacher), _dtype_code(student), T, V, ld_s, ld_t, _ptr(kl),
                              _ptr(targets), _ptr(diff_mask), _ptr(lps), _ptr(lpt), _ptr(diff), _stream(stream))
    check("lp_kl_full_vocab", st)
    return kl, lps, lpt, diff


def lp_prob_diff(lp_a, lp_b, mask=None, *, out=None, stream=None):
    """mask * |exp(lp_a) - exp(lp_b)| elementwise (fp32 vectors)."""
    torch = _torch()
    lib = load()
    lp_a = _vec(lp_a, "lp_a", torch.float32)
    n = lp_a.numel()
    lp_b = _vec(lp_b, "lp_b", torch.float32, n)
    mask = _vec(mask, "mask", torch.uint8, n)
    out = _vec(out, "out", torch.float32, n)
    _on(lp_a.device, lp_a=lp_a, lp_b=lp_b, mask=mask, out=out)
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=lp_a.device)
    st = lib.lp_prob_diff(_ptr(lp_a), _ptr(lp_b), _ptr(mask), n, _ptr(out), _stream(stream))
    check("lp_prob_diff", st)
    return out


def _targets_k(targets, T):
    torch = _torch()
    t = _vec(targets, "targets", torch.int64)
    if t is None or t.dim() != 2 or t.size(0) != T:
        raise ValueError("targets must be [T, K]")
    return t, t.size(1)


def lp_logprobs_entropy_k(logits, targets, mask=None, temperature: float = 1.0, chunk_rows: int = -1, *,
                          want_entropy: bool = True, stream=None):
    """(logprob [T, K], entropy [T] or None) with K targets per row (targets [T, K] int64)."""
    torch = _torch()
    lib = load()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [T, V]")
    T, V = logits.shape
    ld = _rows(logits, "logits")
    targets, K = _targets_k(targets, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    _on(logits.device, logits=logits, targets=targets, mask=mask)
    lp = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    H = torch.empty(T, dtype=torch.float32, device=logits.device) if want_entropy else None
    st = lib.lp_logprobs_entropy_k(_ptr(logits), _dtype_code(logits), T, V, ld, _ptr(targets), K, _ptr(mask),
                                   float(temperature), int(chunk_rows), _ptr(lp), _ptr(H), _stream(stream))
    check("lp_logprobs_entropy_k", st)
    return lp, H


def lp_lm_head_logprobs_entropy_k(hidden, weight, targets, mask=None, temperature: float = 1.0,
                                  tile_rows: int = 4096, *, workspace=None, stream=None):
    """(logprob [T, K], entropy [T], lse [T]) of the fused LM head with K targets per row."""
    torch = _torch()
    lib = load()
    T, h, V = _lm_head_operands(hidden, weight)
    ld_h, ld_w = _rows(hidden, "hidden"), _rows(weight, "weight")
    targets, K = _targets_k(targets, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    dev = hidden.device
    _on(dev, hidden=hidden, weight=weight, targets=targets, mask=mask)
    lp = torch.empty((T, K), dtype=torch.float32, device=dev)
    H = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(lp_lm_head_workspace_bytes(T, h, V, tile_rows, False), dev, workspace)
    st = lib.lp_lm_head_logprobs_entropy_k(_ptr(hidden), ld_h, _ptr(weight), ld_w, T, h, V, _ptr(targets), K,
                                           _ptr(mask), float(temperature), int(tile_rows), _ptr(lp), _ptr(H),
                                           _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    check("lp_lm_head_logprobs_entropy_k", st)
    return lp, H, lse


def lp_lm_head_logprobs_entropy_backward_k(hidden, weight, targets, mask, temperature: float, tile_rows: int,
                                           lse, entropy, grad_logprob, grad_entropy=None, *,
                                           need_grad_hidden: bool = True, need_grad_weight: bool = True,
                                           workspace=None, stream=None):
    """Backward of the K-target fused LM head; grad_logprob is [T, K]."""
    torch = _torch()
    lib = load()
    T, h, V = _lm_head_operands(hidden, weight)
    ld_h, ld_w = _rows(hidden, "hidden"), _rows(weight, "weight")
    targets, K = _targets_k(targets, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    lse = _vec(lse, "lse", torch.float32, T)
    entropy = _vec(entropy, "entropy", torch.float32, T)
    grad_logprob = _vec(grad_logprob, "grad_logprob", torch.float32, T * K)
    if grad_logprob is None or grad_logprob.shape != (T, K):
        raise ValueError("grad_logprob must be [T, K]")
    grad_entropy = _vec(grad_entropy, "grad_entropy", torch.float32, T)
    dev = hidden.device
    _on(dev, hidden=hidden, weight=weight, targets=targets, mask=mask, lse=lse, entropy=entropy,
        grad_logprob=grad_logprob, grad_entropy=grad_entropy)
    dH = torch.empty((T, h), dtype=torch.float32, device=dev) if need_grad_hidden else None
    dW = torch.empty((V, h), dtype=torch.float32, device=dev) if need_grad_weight else None
    ws, ws_bytes = _workspace(lp_lm_head_workspace_bytes(T, h, V, tile_rows, True), dev, workspace)
    st = lib.lp_lm_head_logprobs_entropy_backward_k(
        _ptr(hidden), ld_h, _ptr(weight), ld_w, T, h, V, _ptr(targets), K, _ptr(mask), float(temperature),
        int(tile_rows), _ptr(lse), _ptr(entropy), _ptr(grad_logprob), _ptr(grad_entropy), _ptr(dH), _ptr(dW),
        _ptr(ws), ws_bytes, _stream(stream))
    check("lp_lm_head_logprobs_entropy_backward_k", st)
    return dH, dW


def lp_prob_diff_stats(lp_a, lp_b, mask=None, *, stream=None):
    """Device float64 [5]: count, max, mean, std of mask * |exp(a) - exp(b)| and Pearson(exp(a), exp(b))."""
    torch = _torch()
    lib = load()
    lp_a = _vec(lp_a, "lp_a", torch.float32)
    n = lp_a.numel()
    lp_b = _vec(lp_b, "lp_b", torch.float32, n)
    mask = _vec(mask, "mask", torch.uint8, n)
    _on(lp_a.device, lp_a=lp_a, lp_b=lp_b, mask=mask)
    out = torch.empty(5, dtype=torch.float64, device=lp_a.device)
    ws = torch.empty(max(int(lib.lp_prob_diff_stats_workspace_bytes()), 256), dtype=torch.uint8, device=lp_a.device)
    st = lib.lp_prob_diff_stats(_ptr(lp_a), _ptr(lp_b), _ptr(mask), n, _ptr(out), _ptr(ws), ws.numel(),
                                _stream(stream))
    check("lp_prob_diff_stats", st)
    return out


def lp_lm_head_kl_workspace_bytes(T: int, h_student: int, V: int, tile_rows: int, backward: bool) -> int:
    return int(load().lp_lm_head_kl_workspace_bytes(T, h_student, V, tile_rows, 1 if backward else 0))


def _heads(student_hidden, student_weight, teacher_hidden, teacher_weight):
    for t, n in ((student_hidden, "student_hidden"), (student_weight, "student_weight"),
                 (teacher_hidden, "teacher_hidden"), (teacher_weight, "teacher_weight")):
        _bf16_2d(t, n)
    T, hs = student_hidden.shape
    V, hs2 = student_weight.shape
    T2, ht = teacher_hidden.shape
    V2, ht2 = teacher_weight.shape
    if hs2 != hs or ht2 != ht or T2 != T or V2 != V:
        raise ValueError("student / teacher hidden and weight shapes disagree")
    args = [_ptr(student_hidden), _rows(student_hidden, "student_hidden"), _ptr(student_weight),
            _rows(student_weight, "student_weight"), hs, _ptr(teacher_hidden), _rows(teacher_hidden, "teacher_hidden"),
            _ptr(teacher_weight), _rows(teacher_weight, "teacher_weight"), ht]
    tensors = dict(student_hidden=student_hidden, student_weight=student_weight, teacher_hidden=teacher_hidden,
                   teacher_weight=teacher_weight)
    return T, V, hs, ht, args, tensors


def lp_lm_head_kl(student_hidden, student_weight, teacher_hidden, teacher_weight, mask=None, targets=None,
                  diff_mask=None, tile_rows: int = 4096, *, want_lse: bool = True, workspace=None, stream=None):
    """(kl, lp_student, lp_teacher, prob_diff, lse_student, lse_teacher) of the logits hidden @ W^T of each
    model (bf16 hiddens [T, h_*], weights [V, h_*]); the target outputs are None without targets."""
    torch = _torch()
    lib = load()
    T, V, hs, ht, head_args, heads = _heads(student_hidden, student_weight, teacher_hidden, teacher_weight)
    mask = _vec(mask, "mask", torch.uint8, T)
    targets = _vec(targets, "targets", torch.int64, T)
    diff_mask = _vec(diff_mask, "diff_mask", torch.uint8, T)
    dev = student_hidden.device
    _on(dev, **heads, mask=mask, targets=targets, diff_mask=diff_mask)
    f32 = dict(dtype=torch.float32, device=dev)
    kl = torch.empty(T, **f32)
    lps = lpt = diff = None
    if targets is not None:
        lps, lpt, diff = torch.empty(T, **f32), torch.empty(T, **f32), torch.empty(T, **f32)
    lseu = torch.empty(T, **f32) if want_lse else None
    lsev = torch.empty(T, **f32) if want_lse else None
    ws, ws_bytes = _workspace(lp_lm_head_kl_workspace_bytes(T, hs, V, tile_rows, False), dev, workspace)
    st = lib.lp_lm_head_kl(*head_args, T, V, _ptr(mask), _ptr(targets), _ptr(diff_mask), int(tile_rows), _ptr(kl),
                           _ptr(lps), _ptr(lpt), _ptr(diff), _ptr(lseu), _ptr(lsev), _ptr(ws), ws_bytes,
                           _stream(stream))
    check("lp_lm_head_kl", st)
    return kl, lps, lpt, diff, lseu, lsev


def lp_lm_head_kl_backward(student_hidden, student_weight, teacher_hidden, teacher_weight, mask, tile_rows: int,
                           lse_student, lse_teacher, grad_kl, *, need_grad_hidden: bool = True,
                           need_grad_weight: bool = True, workspace=None, stream=None) -> Tuple:
    """(grad_hidden fp32 [T, h_student] or None, grad_weight fp32 [V, h_student] or None) of sum_t g_t KL_t."""
    torch = _torch()
    lib = load()
    T, V, hs, ht, head_args, heads = _heads(student_hidden, student_weight, teacher_hidden, teacher_weight)
    mask = _vec(mask, "mask", torch.uint8, T)
    lse_student = _vec(lse_student, "lse_student", torch.float32, T)
    lse_teacher = _vec(lse_teacher, "lse_teacher", torch.float32, T)
    grad_kl = _vec(grad_kl, "grad_kl", torch.float32, T)
    dev = student_hidden.device
    _on(dev, **heads, mask=mask, lse_student=lse_student, lse_teacher=lse_teacher, grad_kl=grad_kl)
    dH = torch.empty((T, hs), dtype=torch.float32, device=dev) if need_grad_hidden else None
    dW = torch.empty((V, hs), dtype=torch.float32, device=dev) if need_grad_weight else None
    ws, ws_bytes = _workspace(lp_lm_head_kl_workspace_bytes(T, hs, V, tile_rows, True), dev, workspace)
    st = lib.lp_lm_head_kl_backward(*head_args, T, V, _ptr(mask), int(tile_rows), _ptr(lse_student),
                                    _ptr(lse_teacher), _ptr(grad_kl), _ptr(dH), _ptr(dW), _ptr(ws), ws_bytes,
                                    _stream(stream))
    check("lp_lm_head_kl_backward", st)
    return dH, dW


# ---------------------------------------------------------------------------
# logit rules
# ---------------------------------------------------------------------------

class _NoScope:
    """No context: `device` is current already."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_SCOPE = _NoScope()


def _scope(device, stream):
    """Context in which a call on `device` allocates and launches: outputs and
    workspaces come from the memory of the stream that the kernels run on, and
    `device` is current while they are launched."""
    torch = _torch()
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, expected {device}")
        return torch.cuda.stream(stream)
    if device.index != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return _NO_SCOPE


def _raw_stream(device, stream):
    """hipStream_t of `stream`, or of `device`'s current stream (looked up without making a Stream object, which
    costs a small call more than its launch)."""
    return stream.cuda_stream if stream is not None else _torch()._C._cuda_getCurrentRawStream(device.index)


def _same_device(device, named):
    """Every (name, tensor) lives on `device`."""
    index = device.index  # None for the host, which no tensor's device number equals
    for name, t in named:
        if t is not None and t.get_device() != index:
            _on(device, **{name: t})


class LogitRules:
    """Penalties for repeated tokens, biases and a grammar mask on T rows of
    logits (struct lp_logit_rules; a rule left None is off).

    tokens [B, L] int32 with contiguous rows, hist_len [T] int32: row t's
    history is the first hist_len[t] tokens of buffer row_seq[t] (int32 [T];
    None: buffer t), its first prompt_len[t] the prompt (int32 [T]; None: no
    prompt).  repetition, frequency, presence: fp32 [T].  bias_offsets int64
    [T + 1] into bias_tokens (int32) and bias_values (fp32).  allowed [T, W]
    int32 or uint32 with contiguous rows, W >= ceil(V / 32).

    Types and layouts are checked here and again by each call that takes the
    rules, as are the lengths that depend on T and V and the device.  The
    tensors are kept, not copied: a call reads them as they are when it is made
    (resized or pointed elsewhere included), and what they hold when it runs
    on the stream."""

    __slots__ = ("_tokens", "_vectors", "_biases", "_allowed")

    def __init__(self, tokens=None, hist_len=None, prompt_len=None, row_seq=None, repetition=None, frequency=None,
                 presence=None, bias_offsets=None, bias_tokens=None, bias_values=None, allowed=None):
        torch = _torch()
        i32, f32 = torch.int32, torch.float32
        self._tokens = tokens
        # (name, field of lp_logit_rules, tensor, dtype) of the per-row arrays
        self._vectors = vectors = []
        if hist_len is not None:
            vectors.append(("hist_len", "hist_len", hist_len, i32))
        elif tokens is not None:
            raise ValueError("tokens need hist_len")
        if prompt_len is not None:
            vectors.append(("prompt_len", "prompt_len", prompt_len, i32))
        if row_seq is not None:
            vectors.append(("row_seq", "row_buffer", row_seq, i32))
        if repetition is not None:
            vectors.append(("repetition", "repetition", repetition, f32))
        if frequency is not None:
            vectors.append(("frequency", "frequency", frequency, f32))
        if presence is not None:
            vectors.append(("presence", "presence", presence, f32))
        if tokens is None and vectors:
            raise ValueError("penalties need tokens and hist_len")
        self._biases = None
        if bias_offsets is not None:
            if bias_tokens is None or bias_values is None:
                raise ValueError("biases need bias_tokens and bias_values")
            self._biases = bias_offsets, bias_tokens, bias_values
        elif bias_tokens is not None or bias_values is not None:
            raise ValueError("biases need bias_offsets")
        self._allowed = allowed
        self._layouts()

    @property
    def _per_row(self):
        return [(name, t) for name, _, t, _ in self._vectors]

    @property
    def _whole(self):
        named = [("tokens", self._tokens), *zip(("bias_offsets", "bias_tokens", "bias_values"), self._biases or ()),
                 ("allowed", self._allowed)]
        return [(name, t) for name, t in named if t is not None]

    def _layouts(self):
        """Types and layouts as they are now; (pitch of tokens, entries of the biases, pitch of allowed)."""
        torch = _torch()
        ld_tokens = bias_count = ld_allowed = 0
        tokens = self._tokens
        if tokens is not None:
            if tokens.dtype is not torch.int32:
                raise TypeError(f"tokens must be torch.int32, got {tokens.dtype}")
            ld_tokens = _rows(tokens, "tokens")
            for name, _, t, dt in self._vectors:
                if t.dtype is not dt or not t.is_contiguous():
                    _vec(t, name, dt)
        if self._biases is not None:
            offsets, ids, values = self._biases
            bias_count = ids.numel()
            if offsets.dtype is not torch.int64 or not offsets.is_contiguous():
                _vec(offsets, "bias_offsets", torch.int64)
            if ids.dtype is not torch.int32 or not ids.is_contiguous():
                _vec(ids, "bias_tokens", torch.int32)
            if values.dtype is not torch.float32 or not values.is_contiguous() or values.numel() != bias_count:
                _vec(values, "bias_values", torch.float32, bias_count)
        allowed = self._allowed
        if allowed is not None:
            if allowed.dtype is not torch.int32 and allowed.dtype is not torch.uint32:
                raise TypeError(f"allowed must be int32 or uint32, got {allowed.dtype}")
            ld_allowed = _rows(allowed, "allowed")
        return ld_tokens, bias_count, ld_allowed

    def _check(self, T, V, device):
        """The ctypes argument for a call on T rows of V columns on `device`."""
        c = _lib.LogitRulesC()
        c.ld_tokens, c.bias_count, c.ld_allowed = self._layouts()
        index = device.index
        elsewhere = False  # a tensor on another device, reported after every length
        tokens = self._tokens
        if tokens is not None:
            buffers, length = tokens.shape
            elsewhere = tokens.get_device() != index
            # no buffers, or buffers of no tokens: nobody has a history
            some = buffers and length
            if some:
                c.tokens, c.buffers, c.max_len = tokens.data_ptr(), buffers, length
            for name, field, t, _ in self._vectors:
                if t.numel() != T:
                    raise ValueError(f"{name} must have {T} elements, got {t.numel()}")
                if t.get_device() != index:
                    elsewhere = True
                if some:
                    setattr(c, field, t.data_ptr())
            if some and buffers < T and not c.row_buffer:
                raise ValueError(f"tokens must have a buffer for each of {T} rows, got {buffers}")
        if self._biases is not None:
            offsets, ids, values = self._biases
            if offsets.numel() != T + 1:
                raise ValueError(f"bias_offsets must have {T + 1} elements, got {offsets.numel()}")
            c.bias_offsets, c.bias_tokens, c.bias_values = offsets.data_ptr(), ids.data_ptr(), values.data_ptr()
            if offsets.get_device() != index or ids.get_device() != index or values.get_device() != index:
                elsewhere = True
        allowed = self._allowed
        if allowed is not None:
            rows, words = allowed.shape
            if rows != T or words < (V + 31) // 32:
                raise ValueError(f"allowed must be [{T}, >= {(V + 31) // 32}], got {list(allowed.shape)}")
            c.allowed = allowed.data_ptr()
            if allowed.get_device() != index:
                elsewhere = True
        if elsewhere:
            _same_device(device, self._per_row + self._whole)
        return ctypes.byref(c)


def _processed_operands(logits, rules):
    """(T, V, ld, rules argument) of logits [T, V] under `rules` (None: no rules)."""
    ld = _rows(logits, "logits")
    T, V = logits.shape
    return T, V, ld, None if rules is None else rules._check(T, V, logits.device)


def lp_process_logits(logits, rules, mask=None, *, out=None, stream=None):
    """logits [T, V] under `rules` (LogitRules or None), rounded once to their dtype.  Rows with mask 0 keep what `out`
    held, and are 0 where no out is given; out may be the logits themselves (in place)."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    T, V, ld, c_rules = _processed_operands(logits, rules)
    mask = _vec(mask, "mask", torch.uint8, T)
    if out is not None and (out.shape != logits.shape or out.dtype != logits.dtype):
        raise ValueError("out must have the logits' shape and dtype")
    ld_out = V if out is None else _rows(out, "out")
    dev = logits.device
    _same_device(dev, (("logits", logits), ("mask", mask), ("out", out)))
    with _scope(dev, stream):
        if out is None:
            # the kernel leaves unscored rows alone: they are cleared first
            out = (torch.empty if mask is None else torch.zeros)((T, V), dtype=logits.dtype, device=dev)
        st = lib.lp_process_logits(_ptr(logits), dtype, T, V, ld, c_rules, _ptr(mask), _ptr(out), ld_out,
                                   _raw_stream(dev, stream))
    check("lp_process_logits", st)
    return out


def lp_processed_workspace_bytes(T: int, V: int) -> int:
    return int(load().lp_processed_workspace_bytes(T, V))


def lp_processed_logprobs_entropy(logits, rules, targets, mask=None, temperature: float = 1.0, *,
                                  want_entropy: bool = True, want_lse: bool = True, workspace=None, stream=None):
    """(logprob, entropy, lse) of softmax(rules(logits) / temperature); logits [T, V], rules LogitRules or None."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    T, V, ld, c_rules = _processed_operands(logits, rules)
    targets = _vec(targets, "targets", torch.int64, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    dev = logits.device
    _same_device(dev, (("logits", logits), ("targets", targets), ("mask", mask)))
    f32 = dict(dtype=torch.float32, device=dev)
    with _scope(dev, stream):
        lp = torch.empty(T, **f32)
        H = torch.empty(T, **f32) if want_entropy else None
        lse = torch.empty(T, **f32) if want_lse else None
        ws, ws_bytes = _workspace(lp_processed_workspace_bytes(T, V), dev, workspace)
        st = lib.lp_processed_logprobs_entropy(_ptr(logits), dtype, T, V, ld, c_rules, _ptr(targets), _ptr(mask),
                                               float(temperature), _ptr(lp), _ptr(H), _ptr(lse), _ptr(ws), ws_bytes,
                                               _raw_stream(dev, stream))
    check("lp_processed_logprobs_entropy", st)
    return lp, H, lse


def lp_processed_logprobs_entropy_backward(logits, rules, targets, mask, temperature: float, lse, entropy,
                                           grad_logprob, grad_entropy=None, *, grad_logits=None, stream=None):
    """Gradient [T, V] of sum g_lp * logprob + g_H * entropy with respect to the raw logits, in their dtype."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    T, V, ld, c_rules = _processed_operands(logits, rules)
    targets = _vec(targets, "targets", torch.int64, T)
    mask = _vec(mask, "mask", torch.uint8, T)
    lse = _vec(lse, "lse", torch.float32, T)
    entropy = _vec(entropy, "entropy", torch.float32, T)
    grad_logprob = _vec(grad_logprob, "grad_logprob", torch.float32, T)
    grad_entropy = _vec(grad_entropy, "grad_entropy", torch.float32, T)
    if grad_logits is not None and (grad_logits.shape != logits.shape or grad_logits.dtype != logits.dtype):
        raise ValueError("grad_logits must have the logits' shape and dtype")
    ld_grad = V if grad_logits is None else _rows(grad_logits, "grad_logits")
    dev = logits.device
    _same_device(dev, (("logits", logits), ("targets", targets), ("mask", mask), ("lse", lse), ("entropy", entropy),
                       ("grad_logprob", grad_logprob), ("grad_entropy", grad_entropy), ("grad_logits", grad_logits)))
    with _scope(dev, stream):
        if grad_logits is None:
            grad_logits = torch.empty((T, V), dtype=logits.dtype, device=dev)
        st = lib.lp_processed_logprobs_entropy_backward(
            _ptr(logits), dtype, T, V, ld, c_rules, _ptr(targets), _ptr(mask), float(temperature), _ptr(lse),
            _ptr(entropy), _ptr(grad_logprob), _ptr(grad_entropy), _ptr(grad_logits), ld_grad, _raw_stream(dev, stream))
    check("lp_processed_logprobs_entropy_backward", st)
    return grad_logits


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def lp_embedding(weight, tokens, scale: float = 1.0, *, out=None, stream=None):
    """scale * weight[tokens] (weight [V, h] bf16/fp16/fp32; tokens int64 of any shape) in the weight's dtype,
    [*tokens.shape, h]; ids outside [0, V) give zeros.  out: [N, h] with contiguous rows."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(weight)
    ld_w = _rows(weight, "weight")
    V, h = weight.shape
    tokens = _vec(tokens, "tokens", torch.int64)
    N = tokens.numel()
    if out is not None and (out.dtype != weight.dtype or out.dim() != 2 or out.shape != (N, h)):
        raise ValueError(f"out must be [{N}, {h}] of the weight's dtype")
    ld_out = h if out is None else _rows(out, "out")
    dev = weight.device
    _same_device(dev, (("weight", weight), ("tokens", tokens), ("out", out)))
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((*tokens.shape, h), dtype=weight.dtype, device=dev)
        st = lib.lp_embedding(_ptr(weight), dtype, V, h, ld_w, _ptr(tokens), N, float(scale), _ptr(out), ld_out,
                              _raw_stream(dev, stream))
    check("lp_embedding", st)
    return out


def lp_embedding_workspace_bytes(N: int, h: int, V: int) -> int:
    return int(load().lp_embedding_workspace_bytes(N, h, V))


def lp_embedding_backward(grad_out, tokens, V: int, scale: float = 1.0, *, grad_weight=None, accumulate: bool = False,
                          workspace=None, stream=None):
    """fp32 [V, h] gradient of lp_embedding's weight.  grad_out [N, h] with contiguous rows (or contiguous of any
    shape [..., h]), tokens int64 with N elements.  With accumulate the sums are added to grad_weight (a tied head's)
    and rows that no token names stay as they are."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(grad_out)
    if grad_out.dim() != 2:
        if grad_out.dim() < 1 or not grad_out.is_contiguous():
            raise ValueError("grad_out must be 2-D with contiguous rows, or contiguous")
        grad_out = grad_out.view(-1, grad_out.size(-1)) if grad_out.size(-1) else grad_out
    ld_g = _rows(grad_out, "grad_out")
    N, h = grad_out.shape
    tokens = _vec(tokens, "tokens", torch.int64, N)
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate needs grad_weight")
    else:
        _vec(grad_weight, "grad_weight", torch.float32, V * h)
        if grad_weight.shape != (V, h):
            raise ValueError(f"grad_weight must be [{V}, {h}]")
    dev = grad_out.device
    _same_device(dev, (("grad_out", grad_out), ("tokens", tokens), ("grad_weight", grad_weight)))
    with _scope(dev, stream):
        if grad_weight is None:
            grad_weight = torch.empty((V, h), dtype=torch.float32, device=dev)
        ws, ws_bytes = _workspace(lp_embedding_workspace_bytes(N, h, V), dev, workspace)
        st = lib.lp_embedding_backward(_ptr(grad_out), dtype, N, h, ld_g, _ptr(tokens), V, float(scale),
                                       1 if accumulate else 0, _ptr(grad_weight), _ptr(ws), ws_bytes,
                                       _raw_stream(dev, stream))
    check("lp_embedding_backward", st)
    return grad_weight


# ---------------------------------------------------------------------------
# 4-bit head
# ---------------------------------------------------------------------------

def lp_lm_head_w4_quantize(weight, group: int = 128, *, packed=None, scales=None, stream=None) -> Tuple:
    """(packed uint8 [V, h / 2], scales bf16 [V, ceil(h / group)]) of a dense head weight [V, h] (bf16/fp16/fp32)."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(weight)
    ld_w = _rows(weight, "weight")
    V, h = weight.shape
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    groups = (h + group - 1) // group
    for name, t, dt, n in (("packed", packed, torch.uint8, h // 2), ("scales", scales, torch.bfloat16, groups)):
        if t is not None and (t.dtype != dt or t.dim() != 2 or t.shape != (V, n)):
            raise ValueError(f"{name} must be [{V}, {n}] {dt}")
    dev = weight.device
    _same_device(dev, (("weight", weight), ("packed", packed), ("scales", scales)))
    with _scope(dev, stream):
        if packed is None:
            packed = torch.empty((V, h // 2), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty((V, groups), dtype=torch.bfloat16, device=dev)
        st = lib.lp_lm_head_w4_quantize(_ptr(weight), dtype, V, h, ld_w, group, _ptr(packed), _rows(packed, "packed"),
                                        _ptr(scales), _rows(scales, "scales"), _raw_stream(dev, stream))
    check("lp_lm_head_w4_quantize", st)
    return packed, scales


def lp_lm_head_w4_logits(hidden, packed, scales, group: int = 128, *, out_dtype=None, out=None, stream=None):
    """Logits [T, V] of hidden [T, h] (bf16/fp16) through a head of lp_lm_head_w4_quantize; out_dtype defaults to
    hidden's."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(hidden)
    ld_h = _rows(hidden, "hidden")
    T, h = hidden.shape
    if packed.dtype != torch.uint8:
        raise TypeError(f"packed must be uint8, got {packed.dtype}")
    if scales.dtype != torch.bfloat16:
        raise TypeError(f"scales must be bfloat16, got {scales.dtype}")
    ld_p, ld_s = _rows(packed, "packed"), _rows(scales, "scales")
    V = packed.size(0)
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if packed.size(1) * 2 != h or scales.shape != (V, (h + group - 1) // group):
        raise ValueError(f"hidden [{T}, {h}], packed {list(packed.shape)} and scales {list(scales.shape)} disagree "
                         f"(group {group})")
    if out is not None:
        if out.dim() != 2 or out.shape != (T, V) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be [{T}, {V}] of out_dtype")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = hidden.dtype
    dev = hidden.device
    _same_device(dev, (("hidden", hidden), ("packed", packed), ("scales", scales), ("out", out)))
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((T, V), dtype=out_dtype, device=dev)
        st = lib.lp_lm_head_w4_logits(_ptr(hidden), dtype, T, h, ld_h, _ptr(packed), ld_p, _ptr(scales), ld_s, V, group,
                                      _ptr(out), _dtype_code(out), _rows(out, "out"), _raw_stream(dev, stream))
    check("lp_lm_head_w4_logits", st)
    return out


# ---------------------------------------------------------------------------
# the largest logits, distillation from them, beams
# ---------------------------------------------------------------------------

def lp_top_workspace_bytes(dtype: int, T: int, V: int, K: int) -> int:
    return int(load().lp_top_workspace_bytes(dtype, T, V, K))


def lp_top_logits(logits, K: int, mask=None, temperature: float = 1.0, *, want_rest: bool = True, want_lse: bool = True,
                  workspace=None, stream=None) -> Tuple:
    """(ids int64 [T, K], logprob fp32 [T, K], rest [T], lse [T]) of the K largest entries of each row of logits [T, V],
    K <= min(V, 256): columns from the largest down (equal ones from the lowest column up), their log-probs under softmax(logits /
    temperature), the log of the mass of all others, and the log-sum-exp.  Unscored rows: ids -1, else 0."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    ld = _rows(logits, "logits")
    T, V = logits.shape
    mask = _vec(mask, "mask", torch.uint8, T)
    dev = logits.device
    _same_device(dev, (("logits", logits), ("mask", mask)))
    K = int(K)
    with _scope(dev, stream):
        ids = torch.empty((T, max(K, 0)), dtype=torch.int64, device=dev)
        logprob = torch.empty((T, max(K, 0)), dtype=torch.float32, device=dev)
        rest = torch.empty(T, dtype=torch.float32, device=dev) if want_rest else None
        lse = torch.empty(T, dtype=torch.float32, device=dev) if want_lse else None
        ws, ws_bytes = _workspace(lp_top_workspace_bytes(dtype, T, V, K), dev, workspace)
        st = lib.lp_top_logits(_ptr(logits), dtype, T, V, ld, K, _ptr(mask), float(temperature), _ptr(ids), _ptr(logprob),
                               _ptr(rest), _ptr(lse), _ptr(ws), ws_bytes, _raw_stream(dev, stream))
    check("lp_top_logits", st)
    return ids, logprob, rest, lse


def lp_distill_top_workspace_bytes(dtype: int, T: int, V: int) -> int:
    return int(load().lp_distill_top_workspace_bytes(dtype, T, V))


def _teacher_lists(logits, teacher_ids, teacher_logprob, teacher_rest, mask):
    """(T, V, ld, K, lists and mask after checks) of logits [T, V] and a teacher's lists [T, K]."""
    torch = _torch()
    ld = _rows(logits, "logits")
    T, V = logits.shape
    if teacher_ids.dim() != 2 or teacher_ids.size(0) != T:
        raise ValueError(f"teacher_ids must be [{T}, K], got {list(teacher_ids.shape)}")
    K = teacher_ids.size(1)
    teacher_ids = _vec(teacher_ids, "teacher_ids", torch.int64)
    teacher_logprob = _vec(teacher_logprob, "teacher_logprob", torch.float32, T * K)
    if teacher_logprob.shape != (T, K):
        raise ValueError(f"teacher_logprob must be [{T}, {K}], got {list(teacher_logprob.shape)}")
    teacher_rest = _vec(teacher_rest, "teacher_rest", torch.float32, T)
    return T, V, ld, K, teacher_ids, teacher_logprob, teacher_rest, _vec(mask, "mask", torch.uint8, T)


def lp_distill_top(logits, teacher_ids, teacher_logprob, teacher_rest=None, mask=None, temperature: float = 1.0, *,
                   want_lse: bool = True, workspace=None, stream=None) -> Tuple:
    """(loss, lse, lse_rest), fp32 [T]: KL from a teacher's lists (ids int64 [T, K], log-probs fp32 [T, K], and the log of the
    mass outside them, fp32 [T] or None), as lp_top_logits gives them, to softmax(logits / temperature) of the
    student's logits [T, V].  Ids outside [0, V) are padding.  lse and lse_rest (the log-sum-exp over columns that no entry names)
    are for the backward."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    T, V, ld, K, ids, logprob, rest, mask = _teacher_lists(logits, teacher_ids, teacher_logprob, teacher_rest, mask)
    dev = logits.device
    _same_device(dev, (("logits", logits), ("teacher_ids", ids), ("teacher_logprob", logprob), ("teacher_rest", rest),
                       ("mask", mask)))
    f32 = dict(dtype=torch.float32, device=dev)
    with _scope(dev, stream):
        loss = torch.empty(T, **f32)
        lse = torch.empty(T, **f32) if want_lse else None
        lse_rest = torch.empty(T, **f32) if want_lse else None
        ws, ws_bytes = _workspace(lp_distill_top_workspace_bytes(dtype, T, V), dev, workspace)
        st = lib.lp_distill_top(_ptr(logits), dtype, T, V, ld, K, _ptr(ids), _ptr(logprob), _ptr(rest), _ptr(mask),
                                float(temperature), _ptr(loss), _ptr(lse), _ptr(lse_rest), _ptr(ws), ws_bytes,
                                _raw_stream(dev, stream))
    check("lp_distill_top", st)
    return loss, lse, lse_rest


def lp_distill_top_backward(logits, teacher_ids, teacher_logprob, teacher_rest, mask, temperature: float, lse, lse_rest,
                            grad_loss, *, grad_logits=None, stream=None):
    """Gradient [T, V] of sum grad_loss * loss (lp_distill_top) with respect to the student's raw logits, in their dtype."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    T, V, ld, K, ids, logprob, rest, mask = _teacher_lists(logits, teacher_ids, teacher_logprob, teacher_rest, mask)
    lse = _vec(lse, "lse", torch.float32, T)
    lse_rest = _vec(lse_rest, "lse_rest", torch.float32, T)
    grad_loss = _vec(grad_loss, "grad_loss", torch.float32, T)
    if grad_logits is not None and (grad_logits.shape != logits.shape or grad_logits.dtype != logits.dtype):
        raise ValueError("grad_logits must have the logits' shape and dtype")
    ld_grad = V if grad_logits is None else _rows(grad_logits, "grad_logits")
    dev = logits.device
    _same_device(dev, (("logits", logits), ("teacher_ids", ids), ("teacher_logprob", logprob), ("teacher_rest", rest),
                       ("mask", mask), ("lse", lse), ("lse_rest", lse_rest), ("grad_loss", grad_loss),
                       ("grad_logits", grad_logits)))
    with _scope(dev, stream):
        if grad_logits is None:
            grad_logits = torch.empty((T, V), dtype=logits.dtype, device=dev)
        st = lib.lp_distill_top_backward(_ptr(logits), dtype, T, V, ld, K, _ptr(ids), _ptr(logprob), _ptr(rest), _ptr(mask),
                                         float(temperature), _ptr(lse), _ptr(lse_rest), _ptr(grad_loss),
                                         _ptr(grad_logits), ld_grad, _raw_stream(dev, stream))
    check("lp_distill_top_backward", st)
    return grad_logits


def lp_beam_workspace_bytes(dtype: int, B: int, W: int, V: int, N: int) -> int:
    return int(load().lp_beam_workspace_bytes(dtype, B, W, V, N))


def lp_beam_select(logits, beam_scores, N: Optional[int] = None, finished=None, end_token: int = 0, temperature: float = 1.0,
                   *, workspace=None, stream=None) -> Tuple:
    """(scores fp32 [B, N], parents int32 [B, N], tokens int64 [B, N]): the N (default W) best continuations of each
    request over its W beams, by beam_scores [B, W] + log softmax(logits / temperature), logits [B * W, V].  A beam that
    is finished (uint8 or bool [B, W]) is one candidate, its score and end_token; one whose score is not finite is none.
    Places that nothing fills: -inf, -1, -1."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(logits)
    ld = _rows(logits, "logits")
    rows, V = logits.shape
    if beam_scores.dim() != 2 or beam_scores.numel() != rows:
        raise ValueError(f"beam_scores must be [B, W] for the {rows} rows of logits, got {list(beam_scores.shape)}")
    B, W = beam_scores.shape
    N = W if N is None else int(N)
    beam_scores = _vec(beam_scores, "beam_scores", torch.float32)
    finished = _vec(finished, "finished", torch.uint8, rows)
    dev = logits.device
    _same_device(dev, (("logits", logits), ("beam_scores", beam_scores), ("finished", finished)))
    with _scope(dev, stream):
        scores = torch.empty((B, max(N, 0)), dtype=torch.float32, device=dev)
        parents = torch.empty((B, max(N, 0)), dtype=torch.int32, device=dev)
        tokens = torch.empty((B, max(N, 0)), dtype=torch.int64, device=dev)
        ws, ws_bytes = _workspace(lp_beam_workspace_bytes(dtype, B, W, V, N), dev, workspace)
        st = lib.lp_beam_select(_ptr(logits), dtype, B, W, V, ld, _ptr(beam_scores), _ptr(finished), N, int(end_token),
                                float(temperature), _ptr(scores), _ptr(parents), _ptr(tokens), _ptr(ws), ws_bytes,
                                _raw_stream(dev, stream))
    check("lp_beam_select", st)
    return scores, parents, tokens


def _levels(sizes, strides, name):
    """(size, stride) of dimensions that one step leads through, sizes of 1 left out."""
    size, stride = 1, 0
    for n, st in zip(reversed(sizes), reversed(strides)):
        if n == 1:
            continue
        if size == 1:
            size, stride = n, st
        elif st == stride * size:
            size *= n
        else:
            raise ValueError(f"{name}: the dimensions before and behind the beams must each be walked in one step")
    return size, stride


def _state_layout(t, dim, name):
    """(outer size, its stride, row stride, mid size, its stride, width), strides and width in bytes, of a state whose
    dimension `dim` is the beams."""
    e, shape, strides = t.element_size(), t.shape, t.stride()
    if 0 in shape:  # strides say nothing
        return 0, 0, 0, 0, 0, 0
    width, k = 1, len(shape)
    while k > dim + 1 and (shape[k - 1] == 1 or strides[k - 1] == width):
        width *= shape[k - 1]
        k -= 1
    mid, mid_stride = _levels(shape[dim + 1:k], strides[dim + 1:k], name) if k > dim + 1 else (1, 0)
    outer, outer_stride = _levels(shape[:dim], strides[:dim], name) if dim else (1, 0)
    return outer, outer_stride * e, strides[dim] * e, mid, mid_stride * e, width * e


def lp_beam_reorder(state, parents, *, dim: int = 0, out=None, stream=None):
    """States follow their beams: along dimension `dim`, row b * N + n of the result is row b * W + parents[b, n] of
    state (W = its size / B), zeros where that parent lies outside [0, W).  state of any dtype, the dimensions before
    `dim` walked in one step, those behind it in at most two (a prefix of each row of a cache); out likewise, in the
    state's parts where neither is dense behind `dim`; parents int32 [B, N], as lp_beam_select gives them."""
    torch = _torch()
    lib = load()
    if parents.dim() != 2:
        raise ValueError(f"parents must be [B, N], got {list(parents.shape)}")
    parents = _vec(parents, "parents", torch.int32)
    B, N = parents.shape
    if not -state.dim() <= dim < state.dim():
        raise ValueError(f"dim {dim} is outside a state of {state.dim()} dimensions")
    dim %= state.dim()
    rows = state.size(dim)
    if N == 0 or (rows == 0 or rows % B if B else rows):
        raise ValueError(f"{rows} rows are no beams of {B} requests that {N} slots go on from")
    shape = list(state.shape)
    shape[dim] = B * N
    if out is not None and (list(out.shape) != shape or out.dtype != state.dtype):
        raise ValueError(f"out must be {shape} of the state's dtype")
    outer, s_outer, s_row, mid, s_mid, width = _state_layout(state, dim, "state")
    dev = state.device
    _same_device(dev, (("state", state), ("parents", parents), ("out", out)))
    with _scope(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=state.dtype, device=dev)
            dm = width
            dr = mid * width
            do = B * N * dr
        else:
            d_outer, do, dr, d_mid, dm, d_width = _state_layout(out, dim, "out")
            if d_outer != outer or d_mid * d_width != mid * width:
                raise ValueError("out cannot be walked as the state is")
            if d_width != width:
                if mid == 1:  # out's parts lie behind each other in the state
                    mid, width, s_mid = d_mid, d_width, d_width
                elif d_mid == 1:
                    dm = width  # the state's parts lie behind each other in out
                else:
                    raise ValueError("out cannot be walked as the state is")
        st = lib.lp_beam_reorder(_ptr(state), s_outer, s_row, s_mid, outer, mid, width, _ptr(parents), B, rows // B if B else 1, N,
                                 _ptr(out), do, dr, dm, _raw_stream(dev, stream))
    check("lp_beam_reorder", st)
    return out


# ---------------------------------------------------------------------------
# 8-bit head
# ---------------------------------------------------------------------------

def lp_lm_head_fp8_quantize(weight, *, q=None, scales=None, stream=None) -> Tuple:
    """(q float8_e4m3fn [V, h], scales fp32 [ceil(V / 128), ceil(h / 128)]) of a dense head weight [V, h]
    (bf16/fp16/fp32)."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(weight)
    ld_w = _rows(weight, "weight")
    V, h = weight.shape
    blocks = ((V + 127) // 128, (h + 127) // 128)
    for name, t, dt, shape in (("q", q, torch.float8_e4m3fn, (V, h)), ("scales", scales, torch.float32, blocks)):
        if t is not None and (t.dtype != dt or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be {list(shape)} {dt}")
    dev = weight.device
    _same_device(dev, (("weight", weight), ("q", q), ("scales", scales)))
    with _scope(dev, stream):
        if q is None:
            q = torch.empty((V, h), dtype=torch.float8_e4m3fn, device=dev)
        if scales is None:
            scales = torch.empty(blocks, dtype=torch.float32, device=dev)
        st = lib.lp_lm_head_fp8_quantize(_ptr(weight), dtype, V, h, ld_w, _ptr(q), _rows(q, "q"), _ptr(scales),
                                         _rows(scales, "scales"), _raw_stream(dev, stream))
    check("lp_lm_head_fp8_quantize", st)
    return q, scales


def lp_lm_head_fp8_workspace_bytes(T: int, h: int, V: int) -> int:
    return int(load().lp_lm_head_fp8_workspace_bytes(T, h, V))


def lp_lm_head_fp8_logits(hidden, q, scales, *, out_dtype=None, out=None, workspace=None, stream=None):
    """Logits [T, V] of hidden [T, h] (bf16/fp16, brought to e4m3 with a scale for each 128 columns of a row) through a head of
    lp_lm_head_fp8_quantize; out_dtype defaults to hidden's."""
    torch = _torch()
    lib = load()
    dtype = _dtype_code(hidden)
    ld_h = _rows(hidden, "hidden")
    T, h = hidden.shape
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"q must be float8_e4m3fn, got {q.dtype}")
    if scales.dtype != torch.float32:
        raise TypeError(f"scales must be float32, got {scales.dtype}")
    ld_q, ld_s = _rows(q, "q"), _rows(scales, "scales")
    V = q.size(0)
    if q.size(1) != h or scales.shape != ((V + 127) // 128, (h + 127) // 128):
        raise ValueError(f"hidden [{T}, {h}], q {list(q.shape)} and scales {list(scales.shape)} disagree")
    if out is not None:
        if out.dim() != 2 or out.shape != (T, V) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be [{T}, {V}] of out_dtype")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = hidden.dtype
    dev = hidden.device
    _same_device(dev, (("hidden", hidden), ("q", q), ("scales", scales), ("out", out)))
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((T, V), dtype=out_dtype, device=dev)
        ws, ws_bytes = _workspace(lp_lm_head_fp8_workspace_bytes(T, h, V), dev, workspace)
        st = lib.lp_lm_head_fp8_logits(_ptr(hidden), dtype, T, h, ld_h, _ptr(q), ld_q, _ptr(scales), ld_s, V, _ptr(out),
                                       _dtype_code(out), _rows(out, "out"), _ptr(ws), ws_bytes, _raw_stream(dev, stream))
    check("lp_lm_head_fp8_logits", st)
    return out
