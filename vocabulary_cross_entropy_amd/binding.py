"""Thin Python binding of libvce (include/vce.h) over ctypes.

Argument marshalling only: torch tensors supply device memory and the HIP
stream, every step of the computation runs in the library's HIP kernels.
There is no fallback: if ``libvce.so`` is missing or the device is not a GPU,
the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvce.so")

DTYPE_FP32 = 0
DTYPE_BF16 = 1

STATUS = {0: "VCE_OK", 1: "VCE_EINVAL", 2: "VCE_EDTYPE", 3: "VCE_EALIGN", 4: "VCE_EALIAS",
          5: "VCE_EWORKSPACE", 6: "VCE_EHIP", 7: "VCE_EUNSUPPORTED", 8: "VCE_ESCRATCH"}

# (name, restype, argtypes) for every symbol include/vce.h declares.
_I64, _I32, _F32, _VP, _SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_F64, _U64 = ctypes.c_double, ctypes.c_uint64
SIGNATURES = {
    "vce_strerror": (ctypes.c_char_p, [_I32]),
    "ce_forward": (_I32, [_VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _I64, _F32, _I32, _I64,
                          _VP, _VP, _VP, _VP, _VP, _VP]),
    "ce_backward": (_I32, [_VP, _VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _VP,
                           _VP, _VP, _VP, _F32, _I32, _I64, _I32, _VP]),
    "ce_forward_backward": (_I32, [_VP, _VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _I64,
                                   _VP, _F32, _I32, _I64, _I32, _VP, _VP, _VP, _VP, _VP]),
    "ce_forward_shard": (_I32, [_VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _I64, _I64,
                                _I64, _VP, _VP, _VP]),
    "ce_merge_shards": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _I64, _I64, _I64, _F32, _I32,
                               _I64, _VP, _VP, _VP, _VP, _VP, _VP]),
    "ce_backward_shard": (_I32, [_VP, _VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _I64,
                                 _I64, _I64, _VP, _VP, _VP, _VP, _VP, _F32, _I32, _I64, _I32,
                                 _VP]),
    "vce_shift_targets": (_I32, [_VP, _I64, _I64, _I64, _I64, _I32, _I64, _VP, _VP]),
    "lce_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "lce_forward": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _F32, _I32, _I64, _VP, _VP, _VP, _VP,
                           _VP, _VP, _SZ, _VP]),
    "lce_forward_noalloc": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _F32, _I32, _I64, _VP, _VP,
                                   _VP, _VP, _VP, _VP]),
    "lce_backward": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _F32, _I32,
                            _I64, _VP, _VP, _VP, _SZ, _VP]),
    "lce_forward_scaled": (_I32, [_VP, _VP, _I64, _I64, _I64, _F32, _VP, _F32, _I32, _I64, _VP,
                                  _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lce_backward_scaled": (_I32, [_VP, _VP, _I64, _I64, _I64, _F32, _VP, _VP, _VP, _VP, _VP,
                                   _VP, _F32, _I32, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "lce_workspace_size_f32": (_SZ, [_I64, _I64, _I64]),
    "lce_forward_f32": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _F32, _I32, _I64, _VP, _VP, _VP,
                               _VP, _VP, _VP, _SZ, _VP]),
    "lce_backward_f32": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _F32,
                                _I32, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "lce_forward_shard": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _VP, _VP,
                                 _SZ, _VP]),
    "lce_backward_shard": (_I32, [_VP, _VP, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _VP, _VP,
                                  _VP, _VP, _F32, _I32, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "lce_forward_shard_scaled": (_I32, [_VP, _VP, _I64, _I64, _I64, _F32, _VP, _I64, _I64, _VP,
                                        _VP, _VP, _SZ, _VP]),
    "lce_backward_shard_scaled": (_I32, [_VP, _VP, _I64, _I64, _I64, _F32, _VP, _I64, _I64, _VP,
                                         _VP, _VP, _VP, _VP, _F32, _I32, _I64, _VP, _VP, _VP,
                                         _SZ, _VP]),
    "vce_gemm_bf16": (_I32, [_VP, _I64, _I32, _VP, _I64, _I32, _I64, _I64, _I64, _VP, _I64, _VP]),
    "rms_forward": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _I64, _VP, _I32, _F32, _F32, _VP,
                           _VP, _VP, _VP]),
    "rms_forward_mx8": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _I64, _VP, _I32, _F32, _F32,
                               _VP, _VP, _VP, _VP, _VP]),
    "rms_backward_workspace_size": (_SZ, [_I64, _I64]),
    "rms_backward": (_I32, [_VP, _VP, _I32, _I64, _I64, _VP, _I32, _F32, _VP, _VP, _VP, _VP, _VP,
                            _SZ, _VP]),
    "mx_quantize": (_I32, [_VP, _I32, _I64, _I64, _I64, _I32, _VP, _VP, _VP]),
    "mx_dequantize": (_I32, [_VP, _VP, _I32, _I64, _I64, _VP, _I32, _VP]),
    "mx_logits": (_I32, [_VP, _VP, _I32, _VP, _VP, _I32, _I64, _I64, _I64, _F32, _VP, _I32, _I64,
                         _VP]),
    "ce_sample_workspace_size": (_SZ, [_I64, _I64]),
    "ce_sample": (_I32, [_VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP,
                         _VP, _VP, _SZ, _VP]),
    "adamw_step": (_I32, [_VP, _I64, _I32, _VP, _VP, _VP, _VP, _VP, _I64, _F64, _F64, _F64, _F64,
                          _F64, _I64, _VP, _VP, _VP, _U64, _VP]),
    "grad_norm_workspace_size": (_SZ, [_I64, _I64]),
    "grad_norm": (_I32, [_VP, _I64, _F64, _VP, _VP, _VP, _SZ, _VP]),
    "beam_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "beam_step": (_I32, [_VP, _I32, _I64, _I64, _I64, _I64, _I64, _VP, _VP, _I64, _I64, _VP, _VP,
                         _VP, _VP, _SZ, _VP]),
    "beam_reorder": (_I32, [_VP, _I64, _I64, _I64, _VP, _I64, _VP]),
    "lora_forward_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "lora_forward": (_I32, [_VP, _I64, _I64, _I64, _I64, _VP, _VP, _I64, _I64, _VP, _VP, _VP, _VP,
                            _I64, _VP, _I32, _I64, _VP, _SZ, _VP]),
    "lora_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I32]),
    "lora_backward": (_I32, [_VP, _I32, _I64, _VP, _I64, _I64, _I64, _I64, _VP, _VP, _I64, _I64,
                             _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
}

_lib = None


class VceError(RuntimeError):
    def __init__(self, name: str, code: int, text: str):
        super().__init__(f"{name} failed: {STATUS.get(code, code)} ({text})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libvce.so (built in-tree by ``python -m vocabulary_cross_entropy_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m vocabulary_cross_entropy_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().vce_strerror(code).decode()


def _check(name: str, code: int):
    if code != 0:
        raise VceError(name, code, strerror(code))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_FP32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise RuntimeError("libvce runs on the GPU only: tensors must be on a HIP device")


def _check_buf(t, name: str, numel: int, dtype=torch.float32, *, one_ok: bool = False,
               like: torch.Tensor | None = None):
    """A tensor handed to the library as a flat buffer: its dtype, element
    count (``numel``, or 1 with ``one_ok``), contiguity (the library reads it
    in flattened row order) and device (that of ``like``).  None passes."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel and not (one_ok and t.numel() == 1):
        want = f"{numel}" + (" or 1" if one_ok else "")
        raise ValueError(f"{name} must hold {want} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")


def _check_rows(N: int, like: torch.Tensor, *, stats=None, n_valid=None, grad_output=None,
                reduce_loss=False, loss_tok=None, loss_mean=None, entropy=None,
                grad_entropy=None):
    """The per-row buffers of a logits or linear call with N rows."""
    _check_buf(stats, "stats", 4 * N, like=like)
    _check_buf(n_valid, "n_valid", 1, torch.int32, like=like)
    if grad_output is not None:
        _check_buf(grad_output, "grad_output", 1 if reduce_loss else N, like=like)
    _check_buf(loss_tok, "loss_tok", N, like=like)
    _check_buf(loss_mean, "loss_mean", 1, like=like)
    _check_buf(entropy, "entropy", N, like=like)
    _check_buf(grad_entropy, "grad_entropy", N, like=like)


def _logits3d(logits: torch.Tensor, targets: torch.Tensor):
    if logits.dim() == 2:
        logits = logits.unsqueeze(0)
        targets = targets.unsqueeze(0)
    if logits.dim() != 3 or tuple(targets.shape) != tuple(logits.shape[:2]):
        raise ValueError("logits must be (d0, d1, V) with targets (d0, d1)")
    if logits.stride(2) != 1:
        raise ValueError("the vocabulary dimension of logits must be contiguous")
    if targets.dtype != torch.int64:
        raise TypeError("targets must be int64")
    return logits, targets


def _check_grad(grad: torch.Tensor, logits: torch.Tensor):
    if tuple(grad.shape) != tuple(logits.shape) or tuple(grad.stride()) != tuple(logits.stride()) \
            or grad.dtype != logits.dtype:
        raise ValueError("grad must have the shape, dtype and strides of logits")
    if grad.device != logits.device:
        raise ValueError(f"grad must be on {logits.device}, got {grad.device}")


def _grad_like(logits: torch.Tensor) -> torch.Tensor:
    """An uninitialised tensor with the dtype and strides of ``logits`` whose
    rows start at the same offset within 16 bytes (the backward splits the
    logits row and the gradient row at the same element)."""
    es = logits.element_size()
    pad = (logits.data_ptr() % 16) // es
    span = 1 + sum((n - 1) * st for n, st in zip(logits.shape, logits.stride()))
    buf = torch.empty(pad + span, dtype=logits.dtype, device=logits.device)
    return buf.as_strided(logits.shape, logits.stride(), pad)


def ce_forward(logits: torch.Tensor, targets: torch.Tensor, label_smoothing: float = 0.0,
               reduce_loss: bool = False, ignore_idx: int = -100, *, stream=None, out=None,
               with_entropy: bool = False):
    """Forward of logits cross-entropy.  Returns (loss_tok, loss_mean, stats, n_valid),
    plus the per-row entropy with ``with_entropy``; loss_mean and n_valid are None
    unless reduce_loss.  ``out`` gives the output tensors in the same order."""
    logits, targets = _logits3d(logits, targets)
    d0, d1, V = logits.shape
    dev = logits.device
    if out is None:
        loss_tok = torch.empty((d0, d1), dtype=torch.float32, device=dev)
        stats = torch.empty((d0, d1, 4), dtype=torch.float32, device=dev)
        loss_mean = torch.empty((), dtype=torch.float32, device=dev) if reduce_loss else None
        n_valid = torch.empty((), dtype=torch.int32, device=dev) if reduce_loss else None
        ent = torch.empty((d0, d1), dtype=torch.float32, device=dev) if with_entropy else None
    else:
        loss_tok, loss_mean, stats, n_valid = out[:4]
        ent = out[4] if with_entropy else None
    _check_rows(d0 * d1, logits, stats=stats, n_valid=n_valid, loss_tok=loss_tok,
                loss_mean=loss_mean, entropy=ent)
    _need_cuda(logits, targets)
    rc = lib().ce_forward(_ptr(logits), _dtype_code(logits), d0, d1, V, logits.stride(0),
                          logits.stride(1), _ptr(targets), targets.stride(0), targets.stride(1),
                          float(label_smoothing), int(bool(reduce_loss)), int(ignore_idx),
                          _ptr(loss_tok), _ptr(loss_mean), _ptr(stats), _ptr(n_valid), _ptr(ent),
                          _stream(stream))
    _check("ce_forward", rc)
    if with_entropy:
        return loss_tok, loss_mean, stats, n_valid, ent
    return loss_tok, loss_mean, stats, n_valid


def ce_backward(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                n_valid: torch.Tensor | None, grad_output: torch.Tensor,
                label_smoothing: float = 0.0, reduce_loss: bool = False, ignore_idx: int = -100,
                overwrite_input: bool = False, *, grad: torch.Tensor | None = None, stream=None,
                entropy: torch.Tensor | None = None, grad_entropy: torch.Tensor | None = None):
    """Gradient of logits cross-entropy rebuilt from ``stats``.  With
    ``overwrite_input`` the logits tensor itself receives the gradient.  With
    ``grad_entropy`` (per row) the entropy's gradient is added; ``entropy`` is
    then the forward's entropy output."""
    logits, targets = _logits3d(logits, targets)
    d0, d1, V = logits.shape
    _check_rows(d0 * d1, logits, stats=stats, n_valid=n_valid if reduce_loss else None,
                grad_output=grad_output, reduce_loss=reduce_loss, entropy=entropy,
                grad_entropy=grad_entropy)
    if overwrite_input:
        grad = logits
    elif grad is None:
        grad = _grad_like(logits)
    elif grad.dim() == 2:
        grad = grad.unsqueeze(0)
    _check_grad(grad, logits)
    _need_cuda(logits, targets, stats, grad_output)
    rc = lib().ce_backward(_ptr(logits), _ptr(grad), _dtype_code(logits), d0, d1, V,
                           logits.stride(0), logits.stride(1), _ptr(targets), targets.stride(0),
                           targets.stride(1), _ptr(stats), _ptr(n_valid), _ptr(grad_output),
                           _ptr(entropy), _ptr(grad_entropy), float(label_smoothing),
                           int(bool(reduce_loss)), int(ignore_idx), int(bool(overwrite_input)),
                           _stream(stream))
    _check("ce_backward", rc)
    return grad


def ce_forward_backward(logits: torch.Tensor, targets: torch.Tensor, grad_output: torch.Tensor,
                        label_smoothing: float = 0.0, reduce_loss: bool = False,
                        ignore_idx: int = -100, overwrite_input: bool = False, *,
                        grad: torch.Tensor | None = None, stream=None, out=None):
    """``ce_forward`` then ``ce_backward`` with the same arguments, in one pass
    over the logits.  Returns (loss_tok, loss_mean, stats, n_valid, grad)."""
    logits, targets = _logits3d(logits, targets)
    d0, d1, V = logits.shape
    dev = logits.device
    if out is None:
        loss_tok = torch.empty((d0, d1), dtype=torch.float32, device=dev)
        stats = torch.empty((d0, d1, 4), dtype=torch.float32, device=dev)
        loss_mean = torch.empty((), dtype=torch.float32, device=dev) if reduce_loss else None
        n_valid = torch.empty((), dtype=torch.int32, device=dev) if reduce_loss else None
    else:
        loss_tok, loss_mean, stats, n_valid = out
    _check_rows(d0 * d1, logits, stats=stats, n_valid=n_valid, grad_output=grad_output,
                reduce_loss=reduce_loss, loss_tok=loss_tok, loss_mean=loss_mean)
    if overwrite_input:
        grad = logits
    elif grad is None:
        grad = _grad_like(logits)
    elif grad.dim() == 2:
        grad = grad.unsqueeze(0)
    _check_grad(grad, logits)
    _need_cuda(logits, targets, grad_output)
    rc = lib().ce_forward_backward(_ptr(logits), _ptr(grad), _dtype_code(logits), d0, d1, V,
                                   logits.stride(0), logits.stride(1), _ptr(targets),
                                   targets.stride(0), targets.stride(1), _ptr(grad_output),
                                   float(label_smoothing), int(bool(reduce_loss)),
                                   int(ignore_idx), int(bool(overwrite_input)), _ptr(loss_tok),
                                   _ptr(loss_mean), _ptr(stats), _ptr(n_valid), _stream(stream))
    _check("ce_forward_backward", rc)
    return loss_tok, loss_mean, stats, n_valid, grad


def ce_forward_shard(logits: torch.Tensor, targets: torch.Tensor, vocab_start: int,
                     ignore_idx: int = -100, *, stream=None, out=None, with_entropy: bool = False,
                     out_w=None):
    """Partial statistics (d0, d1, 4) of one vocabulary shard: ``logits`` holds
    columns vocab_start .. vocab_start + V_local - 1 of the full vocabulary.
    With ``with_entropy`` also the shard's entropy statistic (d0, d1), returned
    second."""
    logits, targets = _logits3d(logits, targets)
    d0, d1, V = logits.shape
    part = torch.empty((d0, d1, 4), dtype=torch.float32, device=logits.device) if out is None \
        else out
    pw = None
    if with_entropy:
        pw = torch.empty((d0, d1), dtype=torch.float32, device=logits.device) if out_w is None \
            else out_w
    _check_buf(part, "partial", 4 * d0 * d1, like=logits)
    _check_buf(pw, "partial_w", d0 * d1, like=logits)
    _need_cuda(logits, targets)
    rc = lib().ce_forward_shard(_ptr(logits), _dtype_code(logits), d0, d1, V, logits.stride(0),
                                logits.stride(1), _ptr(targets), targets.stride(0),
                                targets.stride(1), int(vocab_start), int(ignore_idx), _ptr(part),
                                _ptr(pw), _stream(stream))
    _check("ce_forward_shard", rc)
    return (part, pw) if with_entropy else part


def ce_merge_shards(partials: torch.Tensor, targets: torch.Tensor, V: int,
                    label_smoothing: float = 0.0, reduce_loss: bool = False,
                    ignore_idx: int = -100, *, stream=None, out=None,
                    partials_w: torch.Tensor | None = None, out_entropy=None):
    """Merge stacked shard partials (n_shards, d0, d1, 4) (or (n_shards, N, 4)
    with targets (N)) into (loss_tok, loss_mean, stats, n_valid) over the full
    vocabulary of V columns, as ce_forward returns them.  With ``partials_w``
    (the shards' entropy statistics stacked the same way) the per-row entropy
    is appended."""
    if targets.dim() == 1:
        targets = targets.unsqueeze(0)
    if targets.dtype != torch.int64:
        raise TypeError("targets must be int64")
    d0, d1 = targets.shape
    if not partials.is_contiguous() or partials.dtype != torch.float32 or \
            partials.numel() != partials.shape[0] * d0 * d1 * 4:
        raise ValueError("partials must be contiguous float32 (n_shards, d0, d1, 4)")
    dev = partials.device
    if out is None:
        loss_tok = torch.empty((d0, d1), dtype=torch.float32, device=dev)
        stats = torch.empty((d0, d1, 4), dtype=torch.float32, device=dev)
        loss_mean = torch.empty((), dtype=torch.float32, device=dev) if reduce_loss else None
        n_valid = torch.empty((), dtype=torch.int32, device=dev) if reduce_loss else None
    else:
        loss_tok, loss_mean, stats, n_valid = out
    _check_rows(d0 * d1, partials, stats=stats, n_valid=n_valid, loss_tok=loss_tok,
                loss_mean=loss_mean, entropy=out_entropy)
    _need_cuda(partials, targets)
    ent = None
    if partials_w is not None:
        if not partials_w.is_contiguous() or partials_w.dtype != torch.float32 or \
                partials_w.numel() != partials.shape[0] * d0 * d1:
            raise ValueError("partials_w must be contiguous float32 (n_shards, d0, d1)")
        ent = torch.empty((d0, d1), dtype=torch.float32, device=dev) if out_entropy is None \
            else out_entropy
    rc = lib().ce_merge_shards(_ptr(partials), _ptr(partials_w), partials.shape[0], d0, d1,
                               _ptr(targets), targets.stride(0), targets.stride(1), int(V),
                               float(label_smoothing), int(bool(reduce_loss)), int(ignore_idx),
                               _ptr(loss_tok), _ptr(loss_mean), _ptr(stats), _ptr(n_valid),
                               _ptr(ent), _stream(stream))
    _check("ce_merge_shards", rc)
    if ent is not None:
        return loss_tok, loss_mean, stats, n_valid, ent
    return loss_tok, loss_mean, stats, n_valid


def ce_backward_shard(logits: torch.Tensor, targets: torch.Tensor, vocab_start: int, V: int,
                      stats: torch.Tensor, n_valid: torch.Tensor | None,
                      grad_output: torch.Tensor, label_smoothing: float = 0.0,
                      reduce_loss: bool = False, ignore_idx: int = -100,
                      overwrite_input: bool = False, *, grad: torch.Tensor | None = None,
                      stream=None, entropy: torch.Tensor | None = None,
                      grad_entropy: torch.Tensor | None = None):
    """Gradient of one vocabulary shard's logits from the merged ``stats``
    (with ``grad_entropy``, plus the entropy's, ``entropy`` the merged one)."""
    logits, targets = _logits3d(logits, targets)
    d0, d1, VL = logits.shape
    _check_rows(d0 * d1, logits, stats=stats, n_valid=n_valid if reduce_loss else None,
                grad_output=grad_output, reduce_loss=reduce_loss, entropy=entropy,
                grad_entropy=grad_entropy)
    if overwrite_input:
        grad = logits
    elif grad is None:
        grad = _grad_like(logits)
    elif grad.dim() == 2:
        grad = grad.unsqueeze(0)
    _check_grad(grad, logits)
    _need_cuda(logits, targets, stats, grad_output)
    rc = lib().ce_backward_shard(_ptr(logits), _ptr(grad), _dtype_code(logits), d0, d1, VL,
                                 logits.stride(0), logits.stride(1), _ptr(targets),
                                 targets.stride(0), targets.stride(1), int(vocab_start), int(V),
                                 _ptr(stats), _ptr(n_valid), _ptr(grad_output), _ptr(entropy),
                                 _ptr(grad_entropy), float(label_smoothing),
                                 int(bool(reduce_loss)), int(ignore_idx),
                                 int(bool(overwrite_input)), _stream(stream))
    _check("ce_backward_shard", rc)
    return grad


def shift_targets(targets: torch.Tensor, seq_axis: int, ignore_idx: int = -100, *,
                  stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Causal label shift of (d0, d1) (or (M,) as one sequence) int64 targets
    along ``seq_axis``: each position takes the next position's label, the
    last one ``ignore_idx``.  Returns a contiguous tensor of the same shape."""
    _need_cuda(targets)
    if targets.dtype != torch.int64:
        raise TypeError("targets must be int64")
    t2 = targets.unsqueeze(0) if targets.dim() == 1 else targets
    if t2.dim() != 2:
        raise ValueError("targets must be (d0, d1) or (M,)")
    if targets.dim() == 1 and seq_axis == 0:
        raise ValueError("a 1-D target vector is one sequence: use seq_axis 1 (or -1)")
    seq_axis = 1 if seq_axis == -1 else seq_axis
    d0, d1 = t2.shape
    res = torch.empty(targets.shape, dtype=torch.int64, device=targets.device) if out is None \
        else out
    rc = lib().vce_shift_targets(_ptr(t2), d0, d1, t2.stride(0), t2.stride(1), int(seq_axis),
                                 int(ignore_idx), _ptr(res), _stream(stream))
    _check("vce_shift_targets", rc)
    return res


def lce_workspace_size(M: int, H: int, V: int) -> int:
    return int(lib().lce_workspace_size(M, H, V))


def lce_workspace_size_f32(M: int, H: int, V: int) -> int:
    return int(lib().lce_workspace_size_f32(M, H, V))


def lce_workspace(M: int, H: int, V: int, device="cuda", f32: bool = False) -> torch.Tensor:
    """Workspace for the BF16 linear form, or with ``f32`` for the FP32 one."""
    n = lce_workspace_size_f32(M, H, V) if f32 else lce_workspace_size(M, H, V)
    if n == 0:
        raise ValueError(f"no workspace plan for M={M}, H={H}, V={V}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _check_linear(X, W, targets, dtype=torch.bfloat16):
    if X.dtype != dtype or W.dtype != dtype:
        raise TypeError(f"X and W must be {dtype}")
    if not (X.is_contiguous() and W.is_contiguous() and targets.is_contiguous()):
        raise ValueError("X, W and targets must be contiguous")
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1] or targets.numel() != X.shape[0]:
        raise ValueError("X (M,H), W (V,H), targets (M)")
    if targets.dtype != torch.int64:
        raise TypeError("targets must be int64")
    if W.device != X.device or targets.device != X.device:
        raise ValueError("X, W and targets must be on one device")


def _check_like(t, name: str, ref: torch.Tensor):
    """An output with the shape and dtype of ``ref`` (dX like X, dW like W)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(ref.shape) or t.dtype != ref.dtype:
        raise ValueError(f"{name} must be {ref.dtype} of shape {tuple(ref.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")


def lce_forward(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                label_smoothing: float = 0.0, reduce_loss: bool = True, ignore_idx: int = -100,
                *, workspace: torch.Tensor | None = None, stream=None, out=None,
                with_entropy: bool = False, logit_scale: float = 1.0):
    """Fused linear cross-entropy forward, BF16 X and W.  Returns (loss_tok,
    loss_mean, stats, n_valid), plus the per-token entropy with ``with_entropy``.
    ``logit_scale`` (finite, > 0): the loss of logit_scale * X W^T
    (``lce_forward_scaled``); the backward must get the same value."""
    return _lce_forward(False, X, W, targets, label_smoothing, reduce_loss, ignore_idx,
                        workspace, stream, out, with_entropy, logit_scale)


def lce_forward_noalloc(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                        label_smoothing: float = 0.0, reduce_loss: bool = True,
                        ignore_idx: int = -100, *, stream=None, out=None,
                        with_entropy: bool = False):
    """``lce_forward`` with the library's static scratch instead of a workspace
    (no device allocation by the library; ``out`` lets the caller supply the
    outputs too).  Problems beyond the scratch raise (VCE_ESCRATCH)."""
    _check_linear(X, W, targets)
    M, H = X.shape
    V = W.shape[0]
    dev = X.device
    if out is None:
        loss_tok = torch.empty(M, dtype=torch.float32, device=dev)
        stats = torch.empty((M, 4), dtype=torch.float32, device=dev)
        loss_mean = torch.empty((), dtype=torch.float32, device=dev) if reduce_loss else None
        n_valid = torch.empty((), dtype=torch.int32, device=dev) if reduce_loss else None
        ent = torch.empty(M, dtype=torch.float32, device=dev) if with_entropy else None
    else:
        loss_tok, loss_mean, stats, n_valid = out[:4]
        ent = out[4] if with_entropy else None
    _check_rows(M, X, stats=stats, n_valid=n_valid, loss_tok=loss_tok, loss_mean=loss_mean,
                entropy=ent)
    _need_cuda(X, W, targets)
    rc = lib().lce_forward_noalloc(_ptr(X), _ptr(W), M, H, V, _ptr(targets),
                                   float(label_smoothing), int(bool(reduce_loss)),
                                   int(ignore_idx), _ptr(loss_tok), _ptr(loss_mean), _ptr(stats),
                                   _ptr(n_valid), _ptr(ent), _stream(stream))
    _check("lce_forward_noalloc", rc)
    if with_entropy:
        return loss_tok, loss_mean, stats, n_valid, ent
    return loss_tok, loss_mean, stats, n_valid


def lce_forward_f32(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                    label_smoothing: float = 0.0, reduce_loss: bool = True,
                    ignore_idx: int = -100, *, workspace: torch.Tensor | None = None,
                    stream=None, out=None, with_entropy: bool = False):
    """As ``lce_forward`` for FP32 X and W (workspace from ``lce_workspace(..., f32=True)``)."""
    return _lce_forward(True, X, W, targets, label_smoothing, reduce_loss, ignore_idx,
                        workspace, stream, out, with_entropy)


def _lce_forward(f32, X, W, targets, label_smoothing, reduce_loss, ignore_idx, workspace,
                 stream, out, with_entropy, logit_scale=1.0):
    _check_linear(X, W, targets, torch.float32 if f32 else torch.bfloat16)
    M, H = X.shape
    V = W.shape[0]
    dev = X.device
    if workspace is None:
        workspace = lce_workspace(M, H, V, dev, f32)
    if out is None:
        loss_tok = torch.empty(M, dtype=torch.float32, device=dev)
        stats = torch.empty((M, 4), dtype=torch.float32, device=dev)
        loss_mean = torch.empty((), dtype=torch.float32, device=dev) if reduce_loss else None
        n_valid = torch.empty((), dtype=torch.int32, device=dev) if reduce_loss else None
        ent = torch.empty(M, dtype=torch.float32, device=dev) if with_entropy else None
    else:
        loss_tok, loss_mean, stats, n_valid = out[:4]
        ent = out[4] if with_entropy else None
    _check_rows(M, X, stats=stats, n_valid=n_valid, loss_tok=loss_tok, loss_mean=loss_mean,
                entropy=ent)
    _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=X)
    _need_cuda(X, W, targets)
    if logit_scale != 1.0:
        name = "lce_forward_scaled"
        rc = lib().lce_forward_scaled(_ptr(X), _ptr(W), M, H, V, float(logit_scale),
                                      _ptr(targets), float(label_smoothing),
                                      int(bool(reduce_loss)), int(ignore_idx), _ptr(loss_tok),
                                      _ptr(loss_mean), _ptr(stats), _ptr(n_valid), _ptr(ent),
                                      _ptr(workspace), workspace.numel(), _stream(stream))
    else:
        name = "lce_forward_f32" if f32 else "lce_forward"
        rc = getattr(lib(), name)(_ptr(X), _ptr(W), M, H, V, _ptr(targets),
                                  float(label_smoothing), int(bool(reduce_loss)),
                                  int(ignore_idx), _ptr(loss_tok), _ptr(loss_mean), _ptr(stats),
                                  _ptr(n_valid), _ptr(ent), _ptr(workspace), workspace.numel(),
                                  _stream(stream))
    _check(name, rc)
    if with_entropy:
        return loss_tok, loss_mean, stats, n_valid, ent
    return loss_tok, loss_mean, stats, n_valid


def lce_backward(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                 n_valid: torch.Tensor | None, grad_output: torch.Tensor,
                 label_smoothing: float = 0.0, reduce_loss: bool = True, ignore_idx: int = -100,
                 *, workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                 dW: torch.Tensor | None = None, stream=None, entropy: torch.Tensor | None = None,
                 grad_entropy: torch.Tensor | None = None, logit_scale: float = 1.0):
    """Fused linear cross-entropy backward.  Returns (dX, dW), BF16.  With
    ``grad_entropy`` the entropy's gradient is added (``entropy``: the
    forward's entropy output).  ``logit_scale``: as given to the forward."""
    return _lce_backward(False, X, W, targets, stats, n_valid, grad_output, label_smoothing,
                         reduce_loss, ignore_idx, workspace, dX, dW, stream, entropy,
                         grad_entropy, logit_scale)


def lce_backward_f32(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                     stats: torch.Tensor, n_valid: torch.Tensor | None,
                     grad_output: torch.Tensor, label_smoothing: float = 0.0,
                     reduce_loss: bool = True, ignore_idx: int = -100, *,
                     workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                     dW: torch.Tensor | None = None, stream=None,
                     entropy: torch.Tensor | None = None,
                     grad_entropy: torch.Tensor | None = None):
    """As ``lce_backward`` for FP32 X and W; (dX, dW) FP32."""
    return _lce_backward(True, X, W, targets, stats, n_valid, grad_output, label_smoothing,
                         reduce_loss, ignore_idx, workspace, dX, dW, stream, entropy,
                         grad_entropy)


def _lce_backward(f32, X, W, targets, stats, n_valid, grad_output, label_smoothing,
                  reduce_loss, ignore_idx, workspace, dX, dW, stream, entropy, grad_entropy,
                  logit_scale=1.0):
    _check_linear(X, W, targets, torch.float32 if f32 else torch.bfloat16)
    M, H = X.shape
    V = W.shape[0]
    if workspace is None:
        workspace = lce_workspace(M, H, V, X.device, f32)
    dX = torch.empty_like(X) if dX is None else dX
    dW = torch.empty_like(W) if dW is None else dW
    _check_rows(M, X, stats=stats, n_valid=n_valid if reduce_loss else None,
                grad_output=grad_output, reduce_loss=reduce_loss, entropy=entropy,
                grad_entropy=grad_entropy)
    _check_like(dX, "dX", X)
    _check_like(dW, "dW", W)
    _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=X)
    _need_cuda(X, W, targets, stats, grad_output)
    if logit_scale != 1.0:
        name = "lce_backward_scaled"
        rc = lib().lce_backward_scaled(_ptr(X), _ptr(W), M, H, V, float(logit_scale),
                                       _ptr(targets), _ptr(stats), _ptr(n_valid),
                                       _ptr(grad_output), _ptr(entropy), _ptr(grad_entropy),
                                       float(label_smoothing), int(bool(reduce_loss)),
                                       int(ignore_idx), _ptr(dX), _ptr(dW), _ptr(workspace),
                                       workspace.numel(), _stream(stream))
    else:
        name = "lce_backward_f32" if f32 else "lce_backward"
        rc = getattr(lib(), name)(_ptr(X), _ptr(W), M, H, V, _ptr(targets), _ptr(stats),
                                  _ptr(n_valid), _ptr(grad_output), _ptr(entropy),
                                  _ptr(grad_entropy), float(label_smoothing),
                                  int(bool(reduce_loss)), int(ignore_idx), _ptr(dX), _ptr(dW),
                                  _ptr(workspace), workspace.numel(), _stream(stream))
    _check(name, rc)
    return dX, dW


def lce_forward_shard(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, vocab_start: int,
                      ignore_idx: int = -100, *, workspace: torch.Tensor | None = None,
                      stream=None, out=None, with_entropy: bool = False, out_w=None,
                      logit_scale: float = 1.0):
    """Partial statistics (M, 4) of the vocabulary shard W (V_local, H) holding
    rows vocab_start .. vocab_start + V_local - 1 of the full classifier; with
    ``with_entropy`` also its entropy statistic (M), returned second.  With
    ``logit_scale`` s the shard's logits are s X W^T
    (``lce_forward_shard_scaled``); every shard and the backward take the
    same s."""
    _check_linear(X, W, targets)
    M, H = X.shape
    V = W.shape[0]
    if workspace is None:
        workspace = lce_workspace(M, H, V, X.device)
    part = torch.empty((M, 4), dtype=torch.float32, device=X.device) if out is None else out
    pw = None
    if with_entropy:
        pw = torch.empty(M, dtype=torch.float32, device=X.device) if out_w is None else out_w
    _check_buf(part, "partial", 4 * M, like=X)
    _check_buf(pw, "partial_w", M, like=X)
    _need_cuda(X, W, targets)
    if logit_scale != 1.0:
        name = "lce_forward_shard_scaled"
        rc = lib().lce_forward_shard_scaled(_ptr(X), _ptr(W), M, H, V, float(logit_scale),
                                            _ptr(targets), int(vocab_start), int(ignore_idx),
                                            _ptr(part), _ptr(pw), _ptr(workspace),
                                            workspace.numel(), _stream(stream))
    else:
        name = "lce_forward_shard"
        rc = lib().lce_forward_shard(_ptr(X), _ptr(W), M, H, V, _ptr(targets), int(vocab_start),
                                     int(ignore_idx), _ptr(part), _ptr(pw), _ptr(workspace),
                                     workspace.numel(), _stream(stream))
    _check(name, rc)
    return (part, pw) if with_entropy else part


def lce_backward_shard(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, vocab_start: int,
                       V: int, stats: torch.Tensor, n_valid: torch.Tensor | None,
                       grad_output: torch.Tensor, label_smoothing: float = 0.0,
                       reduce_loss: bool = True, ignore_idx: int = -100, *,
                       workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                       dW: torch.Tensor | None = None, stream=None,
                       entropy: torch.Tensor | None = None,
                       grad_entropy: torch.Tensor | None = None,
                       logit_scale: float = 1.0):
    """(dX share, dW) of one vocabulary shard from the merged ``stats``; the
    shards' dX shares sum to the full dX.  ``entropy``, ``grad_entropy`` as in
    ``ce_backward_shard``; ``logit_scale`` as given to ``lce_forward_shard``
    (``lce_backward_shard_scaled``)."""
    _check_linear(X, W, targets)
    M, H = X.shape
    VL = W.shape[0]
    if workspace is None:
        workspace = lce_workspace(M, H, VL, X.device)
    dX = torch.empty_like(X) if dX is None else dX
    dW = torch.empty_like(W) if dW is None else dW
    _check_rows(M, X, stats=stats, n_valid=n_valid if reduce_loss else None,
                grad_output=grad_output, reduce_loss=reduce_loss, entropy=entropy,
                grad_entropy=grad_entropy)
    _check_like(dX, "dX", X)
    _check_like(dW, "dW", W)
    _need_cuda(X, W, targets, stats, grad_output)
    if logit_scale != 1.0:
        name = "lce_backward_shard_scaled"
        rc = lib().lce_backward_shard_scaled(_ptr(X), _ptr(W), M, H, VL, float(logit_scale),
                                             _ptr(targets), int(vocab_start), int(V),
                                             _ptr(stats), _ptr(n_valid), _ptr(grad_output),
                                             _ptr(entropy), _ptr(grad_entropy),
                                             float(label_smoothing), int(bool(reduce_loss)),
                                             int(ignore_idx), _ptr(dX), _ptr(dW),
                                             _ptr(workspace), workspace.numel(), _stream(stream))
    else:
        name = "lce_backward_shard"
        rc = lib().lce_backward_shard(_ptr(X), _ptr(W), M, H, VL, _ptr(targets),
                                      int(vocab_start), int(V), _ptr(stats), _ptr(n_valid),
                                      _ptr(grad_output), _ptr(entropy), _ptr(grad_entropy),
                                      float(label_smoothing), int(bool(reduce_loss)),
                                      int(ignore_idx), _ptr(dX), _ptr(dW), _ptr(workspace),
                                      workspace.numel(), _stream(stream))
    _check(name, rc)
    return dX, dW


def gemm_bf16(P: torch.Tensor, Q: torch.Tensor, K: int | None = None, *, p_dim: bool = False,
              q_dim: bool = False, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """C[i, j] = sum_k P(i, k) Q(j, k) with the library's matrix-core GEMM.

    P is (rows, K) K-contiguous, or with ``p_dim`` (K, rows) holding P(i, k) at
    [k, i]; likewise Q with ``q_dim``.  BF16, row-major, unit inner stride."""
    _need_cuda(P, Q)
    rows = P.shape[1] if p_dim else P.shape[0]
    cols = Q.shape[1] if q_dim else Q.shape[0]
    if K is None:
        K = P.shape[0] if p_dim else P.shape[1]
    C = torch.empty((rows, cols), dtype=torch.float32, device=P.device) if out is None else out
    rc = lib().vce_gemm_bf16(_ptr(P), P.stride(0), int(p_dim), _ptr(Q), Q.stride(0), int(q_dim),
                             rows, cols, K, _ptr(C), C.stride(0), _stream(stream))
    _check("vce_gemm_bf16", rc)
    return C


# ---- around the head: norm, microscaled formats -----------------------------------------
# These calls run on their tensors' device whatever the current one is, and
# allocate outputs and scratch under the stream they run on, so that freed
# scratch is not handed to another stream while a kernel still uses it.

MX_FORMATS = {"e4m3": 0, "e2m1": 1}


def _at(t):
    return None if t is None else t.data_ptr()


def _elem_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_FP32
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _mx_format(fmt: str) -> int:
    if fmt not in MX_FORMATS:
        raise ValueError(f"format must be one of {sorted(MX_FORMATS)}, got {fmt!r}")
    return MX_FORMATS[fmt]


def _on_stream(ref: torch.Tensor, stream, fn):
    """fn(stream handle) with ref's device current and, given ``stream``, allocations under it."""
    if not ref.is_cuda:
        _need_cuda(ref)
    if stream is None:
        index = ref.get_device()
        if index == torch.cuda.current_device():
            # the handle alone: a Stream object costs more than the launch
            return fn(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(ref.device):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device != ref.device:
            raise ValueError(f"stream must be on {ref.device}, got {s.device}")
        with torch.cuda.stream(s):
            return fn(s.cuda_stream)


def _check_out(t, name: str, shape, dtype, ref: torch.Tensor):
    """A given output: its shape, dtype, contiguity and device.  None passes."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of "
                         f"{tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")


def _rows2d(t: torch.Tensor, name: str):
    """(rows, cols, row stride) of a 2-D tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(shape)}")
    rows, cols = shape
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return rows, cols, ld


def _check_weight(weight: torch.Tensor, H: int, ref: torch.Tensor):
    if weight.dim() != 1 or weight.numel() != H or not weight.is_contiguous():
        raise ValueError(f"weight must be contiguous with {H} elements")
    if weight.device != ref.device:
        raise ValueError(f"weight must be on {ref.device}, got {weight.device}")
    return _elem_dtype(weight, "weight")


def _rms_forward(mx, x, weight, residual, eps, weight_offset, stream, out):
    dt = _elem_dtype(x, "x")
    M, H, ldx = _rows2d(x, "x")
    ldr = 0
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError("residual must have the shape and dtype of x")
        if residual.device != x.device:
            raise ValueError(f"residual must be on {x.device}, got {residual.device}")
        ldr = _rows2d(residual, "residual")[2]
    wdt = _check_weight(weight, H, x)
    if mx and H % 32:
        raise ValueError(f"rows of a multiple of 32 elements are needed, got {H}")
    n = 4 if mx else 3
    if out is None:
        out = (None,) * n
    else:
        if len(out) != n:
            raise ValueError(f"out must hold {n} tensors (None to allocate)")
        if mx:
            _check_out(out[0], "q", (M, H), torch.uint8, x)
            _check_out(out[1], "scales", (M, H // 32), torch.uint8, x)
        else:
            _check_out(out[0], "y", (M, H), x.dtype, x)
        _check_out(out[-2], "rstd", (M,), torch.float32, x)
        _check_out(out[-1], "h", (M, H), x.dtype, x)

    def call(s):
        r, h = out[-2:]
        if r is None:
            r = x.new_empty(M, dtype=torch.float32)
        if h is None and residual is not None:
            h = x.new_empty((M, H))
        if mx:
            q, sc = out[:2]
            if q is None:
                q = x.new_empty((M, H), dtype=torch.uint8)
            if sc is None:
                sc = x.new_empty((M, H // 32), dtype=torch.uint8)
            _check("rms_forward_mx8", lib().rms_forward_mx8(
                x.data_ptr(), dt, M, H, ldx, _at(residual), ldr, weight.data_ptr(), wdt,
                weight_offset, eps, q.data_ptr(), sc.data_ptr(), _at(h), r.data_ptr(), s))
            return q, sc, r, h
        y = x.new_empty((M, H)) if out[0] is None else out[0]
        _check("rms_forward", lib().rms_forward(
            x.data_ptr(), dt, M, H, ldx, _at(residual), ldr, weight.data_ptr(), wdt,
            weight_offset, eps, y.data_ptr(), _at(h), r.data_ptr(), s))
        return y, r, h
    return _on_stream(x, stream, call)


def rms_forward(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                eps: float = 1e-6, *, weight_offset: float = 0.0, stream=None, out=None):
    """Residual + RMS norm: h = x + residual, y = h / sqrt(mean h^2 + eps) * (weight +
    weight_offset) over the rows of x (M, H), BF16 or FP32; weight (H) of either.  Rows may be
    strided.  Returns (y, rstd, h), h None without a residual.  ``out`` gives the outputs in
    that order (None entries are allocated); y or h may be x or residual themselves."""
    return _rms_forward(False, x, weight, residual, eps, weight_offset, stream, out)


def rms_forward_mx8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                    eps: float = 1e-6, *, weight_offset: float = 0.0, stream=None, out=None):
    """``rms_forward`` with y as microscaled 8 bits (E4M3, one scale per 32), the operand of
    ``mx_logits``.  Returns (q, scales, rstd, h)."""
    return _rms_forward(True, x, weight, residual, eps, weight_offset, stream, out)


def rms_backward_workspace_size(M: int, H: int) -> int:
    return int(lib().rms_backward_workspace_size(M, H))


def rms_backward_workspace(M: int, H: int, device="cuda") -> torch.Tensor:
    n = rms_backward_workspace_size(M, H)
    if n == 0:
        raise ValueError(f"no workspace plan for M={M}, H={H}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def rms_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                 dh: torch.Tensor | None = None, *, weight_offset: float = 0.0,
                 workspace: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                 dweight: torch.Tensor | None = None, need_dweight: bool = True, stream=None):
    """Gradient of ``rms_forward``: dy of y, dh (optional) of h by the residual stream; h is the
    forward's h (x without a residual), rstd its rstd.  Returns (dx, dweight): dx (M, H), the
    gradient of x and of the residual alike, in their dtype (may be given as dy, dh or h), and
    dweight (H) FP32, None without ``need_dweight``."""
    dt = _elem_dtype(h, "h")
    M, H, _ = _rows2d(h, "h")
    wdt = _check_weight(weight, H, h)
    shape, hdt = (M, H), h.dtype
    _check_out(dy, "dy", shape, hdt, h)
    _check_out(h, "h", shape, hdt, h)
    _check_out(dh, "dh", shape, hdt, h)
    _check_out(dx, "dx", shape, hdt, h)
    _check_buf(rstd, "rstd", M, like=h)
    _check_out(dweight, "dweight", (H,), torch.float32, h)
    if workspace is not None:
        _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=h)

    def call(s):
        o = torch.empty_like(h) if dx is None else dx
        dw, ws = dweight, workspace
        if need_dweight or dw is not None:
            if dw is None:
                dw = h.new_empty(H, dtype=torch.float32)
            if ws is None:
                ws = rms_backward_workspace(M, H, h.device)
        _check("rms_backward", lib().rms_backward(
            _at(dy), _at(h), dt, M, H, _at(weight), wdt, weight_offset, _at(rstd), _at(dh),
            _at(o), _at(dw), _at(ws), 0 if ws is None else ws.numel(), s))
        return o, dw
    return _on_stream(h, stream, call)


def mx_quantize(x: torch.Tensor, fmt: str = "e2m1", *, stream=None, out=None):
    """x (rows, K), BF16 or FP32, K a multiple of 32, to a microscaled format ("e4m3" or
    "e2m1").  Returns uint8 (q, scales): q (rows, K) or (rows, K / 2), scales (rows, K / 32)."""
    f = _mx_format(fmt)
    dt = _elem_dtype(x, "x")
    rows, K, ldx = _rows2d(x, "x")
    if K == 0 or K % 32:
        raise ValueError(f"rows of a multiple of 32 elements are needed, got {K}")
    q, sc = (None, None) if out is None else out
    qk = K if fmt == "e4m3" else K // 2
    _check_out(q, "q", (rows, qk), torch.uint8, x)
    _check_out(sc, "scales", (rows, K // 32), torch.uint8, x)

    def call(s):
        qo = x.new_empty((rows, qk), dtype=torch.uint8) if q is None else q
        so = x.new_empty((rows, K // 32), dtype=torch.uint8) if sc is None else sc
        _check("mx_quantize", lib().mx_quantize(_at(x), dt, rows, K, ldx, f, _at(qo), _at(so), s))
        return qo, so
    return _on_stream(x, stream, call)


def _check_mx(q: torch.Tensor, scales: torch.Tensor, fmt: str, name: str):
    """(rows, K, format code) of a microscaled matrix."""
    f = _mx_format(fmt)
    if q.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name} and its scales must be uint8")
    shape = q.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(shape)}")
    rows, K = shape
    if fmt == "e2m1":
        K *= 2
    if K == 0 or K % 32 or scales.shape != (rows, K // 32):
        raise ValueError(f"{name} {tuple(shape)} in {fmt} needs scales of "
                         f"({rows}, {K} / 32), got {tuple(scales.shape)}")
    if not (q.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name} and its scales must be contiguous")
    if scales.device != q.device:
        raise ValueError(f"{name} and its scales must be on one device")
    return rows, K, f


def mx_dequantize(q: torch.Tensor, scales: torch.Tensor, fmt: str = "e2m1",
                  dtype: torch.dtype = torch.bfloat16, *, stream=None, out=None):
    """The values (rows, K) that q and scales stand for, as BF16 or FP32."""
    rows, K, f = _check_mx(q, scales, fmt, "q")
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    _check_out(out, "out", (rows, K), dtype, q)

    def call(s):
        o = q.new_empty((rows, K), dtype=dtype) if out is None else out
        _check("mx_dequantize", lib().mx_dequantize(_at(q), _at(scales), f, rows, K, _at(o),
                                                    _elem_dtype(o, "out"), s))
        return o
    return _on_stream(q, stream, call)


def mx_logits(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
              *, x_fmt: str = "e4m3", w_fmt: str = "e2m1", logit_scale: float = 1.0,
              dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """logit_scale * X W^T (M, V) from microscaled X (M, K) and W (V, K), as BF16 or FP32.
    ``out`` may have padded rows (a row stride above V)."""
    M, K, xf = _check_mx(x, x_scales, x_fmt, "x")
    V, Kw, wf = _check_mx(w, w_scales, w_fmt, "w")
    if K != Kw:
        raise ValueError(f"x has rows of {K} values, w of {Kw}")
    if w.device != x.device:
        raise ValueError(f"w must be on {x.device}, got {w.device}")
    if out is not None:
        dtype = out.dtype
        if tuple(out.shape) != (M, V) or (V > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be ({M}, {V}) with contiguous rows")
        if out.device != x.device:
            raise ValueError(f"out must be on {x.device}, got {out.device}")
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")

    def call(s):
        o = x.new_empty((M, V), dtype=dtype) if out is None else out
        _check("mx_logits", lib().mx_logits(
            _at(x), _at(x_scales), xf, _at(w), _at(w_scales), wf, M, K, V, logit_scale, _at(o),
            _elem_dtype(o, "out"), o.stride(0), s))
        return o
    return _on_stream(x, stream, call)


def ce_sample_workspace_size(N: int, V: int) -> int:
    return int(lib().ce_sample_workspace_size(N, V))


def ce_sample_workspace(N: int, V: int, device="cuda") -> torch.Tensor:
    n = ce_sample_workspace_size(N, V)
    if n == 0:
        raise ValueError(f"no workspace plan for N={N}, V={V}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def ce_sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
              top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
              min_p: torch.Tensor | None = None, *, with_logprob: bool = False,
              workspace: torch.Tensor | None = None, stream=None, out=None):
    """One token per row of logits (N, V) or (d0, d1, V), BF16 or FP32, drawn by the uniform
    numbers u (N or (d0, d1), FP32 in [0, 1)).  temperature, top_p, min_p (FP32) and top_k
    (int32), per row like u, or None for off: include/vce.h defines the filters and their order.
    Returns the tokens (int64, shaped like the rows; -1 where a row has no answer), or with
    ``with_logprob`` (tokens, logprob), the log of the probability each was drawn with.  ``out``
    gives the tokens, or both, in that order."""
    dt = _elem_dtype(logits, "logits")
    if logits.dim() not in (2, 3):
        raise ValueError(f"logits must be (N, V) or (d0, d1, V), got {tuple(logits.shape)}")
    lead = tuple(logits.shape[:-1])
    V = logits.shape[-1]
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("the vocabulary dimension of logits must be contiguous")
    d0, d1 = (1, lead[0]) if len(lead) == 1 else lead
    ls0, ls1 = (0, logits.stride(0)) if len(lead) == 1 else logits.stride()[:2]
    N = d0 * d1
    for t, name, td in ((u, "u", torch.float32), (temperature, "temperature", torch.float32),
                        (top_k, "top_k", torch.int32), (top_p, "top_p", torch.float32),
                        (min_p, "min_p", torch.float32)):
        _check_buf(t, name, N, td, like=logits)
    outs = (None, None) if out is None else (tuple(out) if with_logprob else (out, None))
    _check_out(outs[0], "token", lead, torch.int64, logits)
    _check_out(outs[1], "logprob", lead, torch.float32, logits)
    if workspace is not None:
        _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=logits)

    def call(s):
        tok, lp = outs
        if tok is None:
            tok = logits.new_empty(lead, dtype=torch.int64)
        if lp is None and with_logprob:
            lp = logits.new_empty(lead, dtype=torch.float32)
        ws = ce_sample_workspace(N, V, logits.device) if workspace is None else workspace
        _check("ce_sample", lib().ce_sample(
            _at(logits), dt, d0, d1, V, ls0, ls1, _at(temperature), _at(top_k), _at(top_p),
            _at(min_p), _at(u), _at(tok), _at(lp), _at(ws), ws.numel(), s))
        return (tok, lp) if with_logprob else tok
    return _on_stream(logits, stream, call)


class AdamWState:
    """Moments of a list of parameters in flat arrays: parameter i's begin at ``offsets[i]``, a
    multiple of 128.  ``bits`` 32: ``m`` and ``v`` FP32.  8: ``m`` and the root of v as E4M3
    bytes with a scale byte per 32 in ``m_scales`` and ``v_scales`` (``mx_dequantize`` reads them
    as rows of any multiple of 32).  ``master``: FP32 copies of the parameters in the same places, or None."""

    def __init__(self, params, bits: int = 32, master: bool = False):
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits}")
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        dev = params[0].device
        self.bits, self.sizes, self.offsets, at = bits, [], [], 0
        for i, p in enumerate(params):
            _elem_dtype(p, f"params[{i}]")
            if p.device != dev:
                raise ValueError(f"params[{i}] must be on {dev}, got {p.device}")
            if not p.is_contiguous():
                raise ValueError(f"params[{i}] must be contiguous")
            self.sizes.append(p.numel())
            self.offsets.append(at)
            at += (p.numel() + 127) // 128 * 128
        self.total = at
        td = torch.float32 if bits == 32 else torch.uint8
        self.m = torch.zeros(at, dtype=td, device=dev)
        self.v = torch.zeros(at, dtype=td, device=dev)
        self.m_scales = self.v_scales = self.master = None
        if bits == 8:
            self.m_scales = torch.zeros(at // 32, dtype=torch.uint8, device=dev)
            self.v_scales = torch.zeros(at // 32, dtype=torch.uint8, device=dev)
        if master:
            self.master = torch.zeros(at, dtype=torch.float32, device=dev)
            for p, n, o in zip(params, self.sizes, self.offsets):
                self.master[o:o + n].copy_(p.detach().reshape(-1))


def adamw_state(params, bits: int = 32, master: bool = False) -> AdamWState:
    """Zero moments for ``adamw_step`` over these parameters, in FP32 or 8 bits; ``master``
    keeps FP32 copies of the parameters that are stepped in their place."""
    return AdamWState(params, bits, master)


def _scalar(t, name: str, dtype, like: torch.Tensor):
    if t is not None:
        _check_buf(t, name, 1, dtype, like=like)
    return _at(t)


_DATA_PTR, _NUMEL = torch.Tensor.data_ptr, torch.Tensor.numel
_SAME_SIZE, _CONTIGUOUS = torch.Tensor.is_same_size, torch.Tensor.is_contiguous


def _dtype_codes(ts, name: str):
    """Library codes of a list's types."""
    types = [t.dtype for t in ts]
    if not set(types) <= {torch.float32, torch.bfloat16}:
        raise TypeError(f"{name} must be float32 or bfloat16, got {set(types)}")
    return [DTYPE_BF16 if d is torch.bfloat16 else DTYPE_FP32 for d in types]


def _check_tensors(ts, name: str, ref: torch.Tensor):
    """A list of contiguous tensors on ref's device."""
    if not set(map(torch.Tensor.get_device, ts)) <= {ref.get_device()}:
        raise ValueError(f"{name} must be on {ref.device}, got {set(t.device for t in ts)}")
    if not all(map(_CONTIGUOUS, ts)):
        raise ValueError(f"{name} must be contiguous")


def adamw_step(params, grads, state: AdamWState, lr, step, *, betas=(0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: torch.Tensor | None = None, seed: int = 0, stream=None) -> None:
    """One AdamW step in place over the parameters that ``state`` was made for, in one launch
    per 64 of them.  A gradient may be None: that parameter and its moments stay.  lr and
    step (1 for the first) are numbers, or tensors of one element on the device (FP32, int64), read
    when the kernels run.  grad_scale: ``grad_norm``'s scale; not finite (or such an lr, or a step
    below 1, on the device), nothing changes.
    seed: of the random rounding of 8-bit states (the step and place enter it too)."""
    sizes, offsets = state.sizes, state.offsets
    if len(params) != len(sizes) or len(grads) != len(sizes):
        raise ValueError(f"state holds {len(sizes)} parameters, got {len(params)} and "
                         f"{len(grads)} gradients")
    ref = state.m
    have = [g is not None for g in grads]
    if not all(have):
        params, grads, sizes, offsets = (
            [t for t, h in zip(l, have) if h] for l in (params, grads, sizes, offsets))
    # every check over all tensors at once: a call may bring hundreds of small ones
    pt, gt = _dtype_codes(params, "parameters"), _dtype_codes(grads, "gradients")
    if list(map(_NUMEL, params)) != list(sizes) or not all(map(_SAME_SIZE, params, grads)):
        raise ValueError("a parameter has not the size its state was made for, or its gradient "
                         "another shape than it")
    _check_tensors(params, "parameters", ref)
    _check_tensors(grads, "gradients", ref)
    count = len(params)
    # the C structs' fields in order: two pointers, two int64, two int32
    entries = [0] * (5 * count)
    entries[0::5] = map(_DATA_PTR, params)
    entries[1::5] = map(_DATA_PTR, grads)
    entries[2::5] = sizes
    entries[3::5] = offsets
    entries[4::5] = [p | g << 32 for p, g in zip(pt, gt)]
    lr_t = lr if isinstance(lr, torch.Tensor) else None
    step_t = step if isinstance(step, torch.Tensor) else None
    scalars = (_scalar(lr_t, "lr", torch.float32, ref),
               _scalar(step_t, "step", torch.int64, ref),
               _scalar(grad_scale, "grad_scale", torch.float32, ref))
    host = (0.0 if lr_t is not None else float(lr), float(betas[0]), float(betas[1]), float(eps),
            float(weight_decay), 1 if step_t is not None else int(step))
    table = (ctypes.c_int64 * len(entries))(*entries)

    def call(s):
        _check("adamw_step", lib().adamw_step(
            table, count, state.bits, _at(state.m), _at(state.v), _at(state.m_scales),
            _at(state.v_scales), _at(state.master), state.total, *host, *scalars,
            seed & 0xFFFFFFFFFFFFFFFF, s))
    _on_stream(ref, stream, call)


def grad_norm(grads, max_norm: float = float("inf"), *, workspace: torch.Tensor | None = None,
              stream=None, out=None):
    """(norm, scale) of a list of gradients (FP32 or BF16, None entries left out): the root of
    the sum of all squares, and max_norm / norm where that is below 1, else 1 (NaN where norm is
    not finite), as FP32 scalars on the device.  ``out`` gives both."""
    grads = [g for g in grads if g is not None]
    if not grads:
        raise ValueError("no gradients")
    ref, count = grads[0], len(grads)
    codes = _dtype_codes(grads, "gradients")
    _check_tensors(grads, "gradients", ref)
    sizes = list(map(_NUMEL, grads))
    total = sum(sizes)
    entries = [0] * (3 * count)
    entries[0::3] = map(_DATA_PTR, grads)
    entries[1::3] = sizes
    entries[2::3] = codes
    outs = (None, None) if out is None else out
    _check_out(outs[0], "norm", (), torch.float32, ref)
    _check_out(outs[1], "scale", (), torch.float32, ref)
    if workspace is not None:
        _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=ref)
    table = (ctypes.c_int64 * len(entries))(*entries)

    def call(s):
        nrm, sc = (ref.new_empty((), dtype=torch.float32) if t is None else t for t in outs)
        need = int(lib().grad_norm_workspace_size(total, count))
        ws = ref.new_empty(need, dtype=torch.uint8) if workspace is None else workspace
        _check("grad_norm", lib().grad_norm(table, count, max_norm, _at(nrm), _at(sc), _at(ws),
                                            ws.numel(), s))
        return nrm, sc
    return _on_stream(ref, stream, call)


def beam_workspace_size(B: int, K: int, V: int) -> int:
    return int(lib().beam_workspace_size(B, K, V))


def beam_workspace(B: int, K: int, V: int, device="cuda") -> torch.Tensor:
    n = beam_workspace_size(B, K, V)
    if n == 0:
        raise ValueError(f"no workspace plan for B={B}, K={K}, V={V}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def beam_step(logits: torch.Tensor, scores: torch.Tensor, n_out: int | None = None, *,
              ended: torch.Tensor | None = None, end_token: int = 0,
              workspace: torch.Tensor | None = None, stream=None, out=None):
    """The n_out (K unless given) best continuations of every request: logits (B, K, V), BF16 or
    FP32, scores (B, K) FP32, the beams' log-probabilities so far (-inf: an empty beam).  ``ended``
    (B, K) bool: beams that go on as they are, with end_token.  Returns (score, parent, token),
    (B, n_out) each, FP32, int32 and int64, best first (-inf, -1, -1 where candidates run out).
    ``out`` gives the three."""
    dt = _elem_dtype(logits, "logits")
    if logits.dim() != 3:
        raise ValueError(f"logits must be (B, K, V), got {tuple(logits.shape)}")
    B, K, V = logits.shape
    if V > 1 and logits.stride(2) != 1:
        raise ValueError("the vocabulary dimension of logits must be contiguous")
    n = K if n_out is None else int(n_out)
    _check_out(scores, "scores", (B, K), torch.float32, logits)
    _check_out(ended, "ended", (B, K), torch.bool, logits)
    outs = (None,) * 3 if out is None else out
    if len(outs) != 3:
        raise ValueError("out must hold 3 tensors (None to allocate)")
    for t, name, td in zip(outs, ("score", "parent", "token"),
                           (torch.float32, torch.int32, torch.int64)):
        _check_out(t, name, (B, n), td, logits)
    if workspace is not None:
        _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=logits)

    def call(s):
        sc, pa, tok = outs
        if sc is None:
            sc = logits.new_empty((B, n), dtype=torch.float32)
        if pa is None:
            pa = logits.new_empty((B, n), dtype=torch.int32)
        if tok is None:
            tok = logits.new_empty((B, n), dtype=torch.int64)
        ws = beam_workspace(B, K, V, logits.device) if workspace is None else workspace
        _check("beam_step", lib().beam_step(
            _at(logits), dt, B, K, V, logits.stride(0), logits.stride(1), _at(scores), _at(ended),
            end_token, n, _at(sc), _at(pa), _at(tok), _at(ws), ws.numel(), s))
        return sc, pa, tok
    return _on_stream(logits, stream, call)


def _beam_pieces(t: torch.Tensor, name: str):
    """(inner, outer, stride_outer, stride_beam, stride_batch) in bytes of a state (B, K, ...): its
    rows as equally spaced pieces without gaps."""
    es, shape, st = t.element_size(), t.shape, t.stride()
    inner, outer, stride = es, 1, 0
    for n, s in zip(reversed(shape[2:]), reversed(st[2:])):
        if n == 1:
            continue
        if outer == 1 and s * es == inner:
            inner *= n
        elif outer == 1:
            outer, stride = n, s * es
        elif s * es == outer * stride:
            outer *= n
        else:
            raise ValueError(f"the rows of {name} must be contiguous, or equally spaced pieces, got "
                             f"strides {tuple(st)}")
    if t.numel() == 0:
        inner = 0
    return inner, outer, stride, st[1] * es, st[0] * es


def beam_reorder(states, parent: torch.Tensor, *, stream=None) -> None:
    """Every state (B, K, ...) in place: row (b, k) becomes row (b, parent[b, k]), in one launch.
    parent (B, K) int32 as of ``beam_step`` (rows may be strided); an entry outside 0 .. K - 1
    leaves its row.  A state's rows may be views with gaps (the used part of a longer cache)."""
    states = [states] if isinstance(states, torch.Tensor) else list(states)
    if parent.dim() != 2 or parent.dtype != torch.int32:
        raise TypeError(f"parent must be int32 of shape (B, K), got {parent.dtype} of "
                        f"{tuple(parent.shape)}")
    B, K = parent.shape
    if K > 1 and parent.stride(1) != 1:
        raise ValueError("the rows of parent must be contiguous")
    lead, entries = (B, K), []
    same = set(map(torch.Tensor.get_device, states)) <= {parent.get_device()}
    for i, t in enumerate(states):
        if t.shape[:2] != lead:
            raise ValueError(f"states[{i}] must be ({B}, {K}, ...), got {tuple(t.shape)}")
        if not same and t.device != parent.device:
            raise ValueError(f"states[{i}] must be on {parent.device}, got {t.device}")
        size = t.nbytes
        if size and _CONTIGUOUS(t):  # rows without gaps, one after the other
            row = size // (B * K)
            entries += (t.data_ptr(), row, 1, 0, row, row * K)
        else:
            entries += (t.data_ptr(), *_beam_pieces(t, f"states[{i}]"))
    table = (ctypes.c_int64 * len(entries))(*entries)

    def call(s):
        _check("beam_reorder", lib().beam_reorder(table, len(states), B, K, _at(parent),
                                                  parent.stride(0), s))
    if K > 0:
        _on_stream(parent, stream, call)


def lora_forward_workspace_size(M: int, H: int, V: int, n: int, r: int) -> int:
    return int(lib().lora_forward_workspace_size(M, H, V, n, r))


def lora_forward_workspace(M: int, H: int, V: int, n: int, r: int, device="cuda") -> torch.Tensor:
    size = lora_forward_workspace_size(M, H, V, n, r)
    if size == 0:
        raise ValueError(f"no workspace plan for M={M}, H={H}, V={V}, n={n}, r={r}")
    return torch.empty(size, dtype=torch.uint8, device=device)


def lora_backward_workspace_size(M: int, H: int, V: int, n: int, r: int,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    code = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_FP32
    return int(lib().lora_backward_workspace_size(M, H, V, n, r, code))


def lora_backward_workspace(M: int, H: int, V: int, n: int, r: int,
                            dtype: torch.dtype = torch.bfloat16, device="cuda") -> torch.Tensor:
    size = lora_backward_workspace_size(M, H, V, n, r, dtype)
    if size == 0:
        raise ValueError(f"no workspace plan for M={M}, H={H}, V={V}, n={n}, r={r}")
    return torch.empty(size, dtype=torch.uint8, device=device)


def _check_lora(x, a, b, adapter, w, base, scale, workspace):
    """(M, H, V, n, r, ldx) of an adapter call."""
    for t, name in ((x, "x"), (a, "a"), (b, "b")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    M, H, ldx = _rows2d(x, "x")
    if a.dim() != 3 or b.dim() != 3 or a.shape[2] != H or b.shape[0] != a.shape[0] or \
            b.shape[2] != a.shape[1]:
        raise ValueError(f"a must be (n, r, {H}) and b (n, V, r), got {tuple(a.shape)} and "
                         f"{tuple(b.shape)}")
    n, r, V = a.shape[0], a.shape[1], b.shape[1]
    _check_out(a, "a", a.shape, torch.bfloat16, x)
    _check_out(b, "b", b.shape, torch.bfloat16, x)
    _check_out(adapter, "adapter", (M,), torch.int32, x)
    _check_out(scale, "scale", (n,), torch.float32, x)
    _check_out(w, "w", (V, H), torch.bfloat16, x)
    if w is not None and base is not None:
        raise ValueError("either w or what it has given already, not both")
    if workspace is not None:
        _check_buf(workspace, "workspace", workspace.numel(), torch.uint8, like=x)
    return M, H, V, n, r, ldx


def _check_rows_of(t, name, shape, dtype, ref):
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of "
                         f"{tuple(t.shape)}")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")
    return _rows2d(t, name)[2]


def lora_forward(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter: torch.Tensor,
                 w: torch.Tensor | None = None, *, base: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """x W^T + scale[k] (x A_k^T) B_k^T (M, V) for tokens x (M, H), each with its adapter k =
    adapter[i] (int32; outside 0 .. n - 1: none) of a (n, r, H) and b (n, V, r), all BF16; r a
    multiple of 8 up to 128.  ``base`` (M, V): what the shared projection has given already, in the
    place of w; neither: the adapters' share alone.  Result in ``dtype`` (``base``'s and ``out``'s
    where given), BF16 or FP32; ``out`` may have padded rows and may be ``base``."""
    M, H, V, n, r, ldx = _check_lora(x, a, b, adapter, w, base, scale, workspace)
    dtype = out.dtype if out is not None else base.dtype if base is not None else dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    ldb = _check_rows_of(base, "base", (M, V), dtype, x)
    _check_rows_of(out, "out", (M, V), dtype, x)

    def call(s):
        o = x.new_empty((M, V), dtype=dtype) if out is None else out
        ws = lora_forward_workspace(M, H, V, n, r, x.device) if workspace is None else workspace
        _check("lora_forward", lib().lora_forward(
            _at(x), ldx, M, H, V, _at(a), _at(b), n, r, _at(adapter), _at(scale), _at(w),
            _at(base), ldb, _at(o), _elem_dtype(o, "out"), o.stride(0), _at(ws), ws.numel(), s))
        return o
    return _on_stream(x, stream, call)


def lora_backward(dy: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                  adapter: torch.Tensor, w: torch.Tensor | None = None, *,
                  dx_base: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                  need_dx: bool = True, need_adapters: bool = True, out=None,
                  workspace: torch.Tensor | None = None, stream=None):
    """Gradient of ``lora_forward`` from dy (M, V), BF16 or FP32: (dx, da, db), dx (M, H) BF16 =
    dy W + ds A_k (``dx_base`` in the place of dy W where the shared projection lies elsewhere), da
    (n, r, H) and db (n, V, r) FP32, zeros for adapters without tokens; None for what is not
    needed.  W is frozen.  ``out`` gives the three (None entries are allocated); dx may be
    dx_base."""
    M, H, V, n, r, ldx = _check_lora(x, a, b, adapter, w, dx_base, scale, workspace)
    dt = _elem_dtype(dy, "dy")
    ldy = _check_rows_of(dy, "dy", (M, V), dy.dtype, x)
    _check_out(dx_base, "dx_base", (M, H), torch.bfloat16, x)
    outs = (None,) * 3 if out is None else out
    if len(outs) != 3:
        raise ValueError("out must hold 3 tensors (None to allocate)")
    shapes = (((M, H), torch.bfloat16), ((n, r, H), torch.float32), ((n, V, r), torch.float32))
    for t, name, (shape, td) in zip(outs, ("dx", "da", "db"), shapes):
        _check_out(t, name, shape, td, x)

    def call(s):
        need = (need_dx, need_adapters, need_adapters)
        dx, da, db = (x.new_empty(shape, dtype=td) if t is None and wanted else t
                      for t, wanted, (shape, td) in zip(outs, need, shapes))
        ws = workspace
        if ws is None:
            ws = lora_backward_workspace(M, H, V, n, r, dy.dtype, x.device)
        _check("lora_backward", lib().lora_backward(
            _at(dy), dt, ldy, _at(x), ldx, M, H, V, _at(a), _at(b), n, r, _at(adapter),
            _at(scale), _at(w), _at(dx_base), _at(dx), _at(da), _at(db), _at(ws), ws.numel(), s))
        return dx, da, db
    return _on_stream(x, stream, call)
