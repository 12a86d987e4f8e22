"""PyTorch-facing binding of the FLCE library.

PyTorch supplies device memory and the current stream; every step of the
computation runs in libflce.so.  ``flce_forward`` / ``flce_backward`` take
tensors and mirror the C entry points of the same names; the autograd function
and module wrap them the way fla's FusedLinearCrossEntropyLoss wraps its
kernels (fla/modules/fused_linear_cross_entropy.py: the module flattens
[batch, seq, hidden] to [tokens, hidden]), with reduction "none" added and the
gradients produced in backward rather than in forward (DeepSpeed PR 8792).
"""

from __future__ import annotations

import contextlib
import operator
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib

_DTYPES = {torch.bfloat16: _lib.FLCE_BF16, torch.float16: _lib.FLCE_F16, torch.float32: _lib.FLCE_F32}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16, float16 or float32")
    return _DTYPES[t.dtype]


def _reduction_code(reduction: str) -> int:
    if reduction not in _lib.REDUCTIONS:
        raise ValueError(f"reduction must be one of {tuple(_lib.REDUCTIONS)}")
    return _lib.REDUCTIONS[reduction]


def _prep(x, W, b, targets):
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x must be [N, H] and W must be [V, H]")
    if not x.is_cuda:
        raise ValueError("tensors must live on a GPU")
    if W.shape[1] != x.shape[1]:
        raise ValueError("x and W disagree on the hidden size")
    if W.dtype != x.dtype or (b is not None and b.dtype != x.dtype):
        raise TypeError("x, W and b must share one dtype")
    if W.device != x.device or targets.device != x.device or (b is not None and b.device != x.device):
        raise ValueError("x, W, b and targets must be on one device")
    if b is not None and b.shape != (W.shape[0],):
        raise ValueError("b must be [V]")
    x = _pad_hidden(x.contiguous())
    W = _pad_hidden(W.contiguous())
    b = b.contiguous() if b is not None else None
    targets = targets.reshape(-1).to(torch.int64).contiguous()
    if targets.numel() != x.shape[0]:
        raise ValueError("targets must have one entry per row of x")
    return x, W, b, targets


def _pad_hidden(t: torch.Tensor) -> torch.Tensor:
    """The library moves rows in 16-byte pieces and needs H % 8 == 0: other H
    get zero columns up to the next multiple of 8 (a copy), which changes no
    logit, loss or gradient entry of the original columns."""
    H = t.shape[1]
    if H % 8 == 0:
        return t
    out = torch.zeros(t.shape[0], H + (-H) % 8, dtype=t.dtype, device=t.device)
    out[:, :H] = t
    return out


def _check_out(t: Optional[torch.Tensor], shape, like: torch.Tensor, what: str) -> None:
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {like.dtype} tensor of shape {tuple(shape)} on {like.device}")


def _check_ctx(lse: torch.Tensor, n_valid: torch.Tensor, N: int, dev) -> None:
    if lse.dtype != torch.float32 or tuple(lse.shape) != (N,) or not lse.is_contiguous() or lse.device != dev:
        raise ValueError(f"lse must be a contiguous float32 [{N}] tensor on {dev} (as flce_forward returns it)")
    if n_valid.dtype != torch.int64 or n_valid.numel() != 1 or n_valid.device != dev:
        raise ValueError(f"n_valid must be an int64 [1] tensor on {dev} (as flce_forward returns it)")


def flce_workspace_size(N: int, H: int, V: int, dtype: torch.dtype, has_bias: bool,
                        reduction: str = "mean") -> Tuple[int, int]:
    return _lib.flce_workspace_size(N, H, V, _DTYPES[dtype], has_bias, _reduction_code(reduction))


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def flce_keep_workspace_size(N: int, H: int, V: int, dtype: torch.dtype, has_bias: bool,
                             reduction: str = "mean") -> Tuple[int, int, int]:
    """(forward bytes, keep bytes, backward bytes) of flce_forward_keep + flce_backward_kept."""
    return _lib.flce_keep_workspace_size(N, H, V, _DTYPES[dtype], has_bias, _reduction_code(reduction))


def flce_forward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor], targets: torch.Tensor,
                 label_smoothing: float = 0.0, z_loss_scale: float = 0.0, ignore_index: int = -100,
                 reduction: str = "mean", workspace: Optional[torch.Tensor] = None, logit_scale: float = 1.0,
                 return_z_loss: bool = False):
    """Returns (loss, lse, n_valid): loss float32 [1] (sum/mean) or [N] (none); with
    return_z_loss, (loss, lse, n_valid, z_loss), z_loss the s * lse^2 term alone,
    shaped like loss.  The logits are logit_scale * (x W^T + b)."""
    return _forward(x, W, b, targets, label_smoothing, z_loss_scale, ignore_index, reduction, workspace,
                    logit_scale, return_z_loss, None)


def flce_forward_keep(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor], targets: torch.Tensor,
                      label_smoothing: float = 0.0, z_loss_scale: float = 0.0, ignore_index: int = -100,
                      reduction: str = "mean", workspace: Optional[torch.Tensor] = None, logit_scale: float = 1.0,
                      return_z_loss: bool = False, keep: Optional[torch.Tensor] = None):
    """flce_forward that also keeps the first vocabulary slab's logits for
    flce_backward_kept: returns (loss, lse, n_valid, keep) (with return_z_loss,
    z_loss last).  keep: a uint8 device buffer of at least the keep bytes of
    flce_keep_workspace_size to fill (allocated when None)."""
    return _forward(x, W, b, targets, label_smoothing, z_loss_scale, ignore_index, reduction, workspace,
                    logit_scale, return_z_loss, keep if keep is not None else True)


def _forward(x, W, b, targets, label_smoothing, z_loss_scale, ignore_index, reduction, workspace, logit_scale,
             return_z_loss, keep):
    x, W, b, targets = _prep(x, W, b, targets)
    N, H = x.shape
    V = W.shape[0]
    dt, red = _dtype_code(x), _reduction_code(reduction)
    dev = x.device
    if keep is None:
        fwd_bytes, _ = _lib.flce_workspace_size(N, H, V, dt, b is not None, red)
    else:
        fwd_bytes, keep_bytes, _ = _lib.flce_keep_workspace_size(N, H, V, dt, b is not None, red)
        if keep is True:
            keep = torch.empty(keep_bytes, dtype=torch.uint8, device=dev)
        elif keep.dtype != torch.uint8 or keep.device != dev or not keep.is_contiguous() or keep.numel() < keep_bytes:
            raise ValueError(f"keep must be a contiguous uint8 tensor of at least {keep_bytes} bytes on {dev}")
    if workspace is None or workspace.numel() < fwd_bytes:
        workspace = torch.empty(max(fwd_bytes, 1), dtype=torch.uint8, device=dev)
    loss = torch.empty(N if reduction == "none" else 1, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int64, device=dev)
    z_loss = torch.empty_like(loss) if return_z_loss else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        if keep is not None:
            _lib.flce_forward_keep(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                                   float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                                   _lib.options(logit_scale, False, _ptr(z_loss)), loss.data_ptr(), lse.data_ptr(),
                                   n_valid.data_ptr(), keep.data_ptr(), keep.numel(), workspace.data_ptr(),
                                   workspace.numel(), stream)
        elif logit_scale == 1.0 and not return_z_loss:
            _lib.flce_forward(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                              float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                              loss.data_ptr(), lse.data_ptr(), n_valid.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), stream)
        else:
            _lib.flce_forward_ex(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                                 float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                                 _lib.options(logit_scale, False, _ptr(z_loss)), loss.data_ptr(), lse.data_ptr(),
                                 n_valid.data_ptr(), workspace.data_ptr(), workspace.numel(), stream)
    out = (loss, lse, n_valid) if keep is None else (loss, lse, n_valid, keep)
    return out + (z_loss,) if return_z_loss else out


def flce_backward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor], targets: torch.Tensor,
                  lse: torch.Tensor, n_valid: torch.Tensor, grad_loss: torch.Tensor,
                  label_smoothing: float = 0.0, z_loss_scale: float = 0.0, ignore_index: int = -100,
                  reduction: str = "mean", need_dx: bool = True, need_dW: bool = True,
                  need_db: bool = True, workspace: Optional[torch.Tensor] = None,
                  out: Optional[Tuple] = None, logit_scale: float = 1.0, accumulate: bool = False):
    """Returns (dx, dW, db) in the input dtype (None where not requested).  With
    accumulate, the gradients are added to the ``out`` tensors' contents."""
    return _backward(x, W, b, targets, lse, n_valid, grad_loss, label_smoothing, z_loss_scale, ignore_index,
                     reduction, need_dx, need_dW, need_db, workspace, out, logit_scale, accumulate, None)


def flce_backward_kept(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor], targets: torch.Tensor,
                       lse: torch.Tensor, n_valid: torch.Tensor, grad_loss: torch.Tensor, keep: torch.Tensor,
                       label_smoothing: float = 0.0, z_loss_scale: float = 0.0, ignore_index: int = -100,
                       reduction: str = "mean", need_dx: bool = True, need_dW: bool = True,
                       need_db: bool = True, workspace: Optional[torch.Tensor] = None,
                       out: Optional[Tuple] = None, logit_scale: float = 1.0, accumulate: bool = False):
    """flce_backward given the keep buffer that flce_forward_keep filled with
    the same arguments; consumes it (a second backward needs a new forward)."""
    if keep is None:
        raise ValueError("keep is the buffer flce_forward_keep returned")
    return _backward(x, W, b, targets, lse, n_valid, grad_loss, label_smoothing, z_loss_scale, ignore_index,
                     reduction, need_dx, need_dW, need_db, workspace, out, logit_scale, accumulate, keep)


def _backward(x, W, b, targets, lse, n_valid, grad_loss, label_smoothing, z_loss_scale, ignore_index, reduction,
              need_dx, need_dW, need_db, workspace, out, logit_scale, accumulate, keep):
    H0 = x.shape[1] if x.dim() == 2 else -1
    x, W, b, targets = _prep(x, W, b, targets)
    N, H = x.shape
    V = W.shape[0]
    dt, red = _dtype_code(x), _reduction_code(reduction)
    dev = x.device
    _check_ctx(lse, n_valid, N, dev)
    g = grad_loss.reshape(-1).to(device=dev, dtype=torch.float32).contiguous()
    if g.numel() != (N if reduction == "none" else 1):
        raise ValueError("grad_loss must have N entries for none and one otherwise")
    if keep is None:
        _, bwd_bytes = _lib.flce_workspace_size(N, H, V, dt, b is not None, red)
    else:
        _, keep_bytes, bwd_bytes = _lib.flce_keep_workspace_size(N, H, V, dt, b is not None, red)
        if keep.dtype != torch.uint8 or keep.device != dev or not keep.is_contiguous() or keep.numel() < keep_bytes:
            raise ValueError(f"keep must be the contiguous uint8 buffer flce_forward_keep filled ({keep_bytes} bytes)")
    if workspace is None or workspace.numel() < bwd_bytes:
        workspace = torch.empty(max(bwd_bytes, 1), dtype=torch.uint8, device=dev)
    if out is not None:
        dx, dW, db = out
        _check_out(dx, (N, H0), x, "out dx")
        _check_out(dW, (V, H0), x, "out dW")
        _check_out(db, (V,), x, "out db")
    else:
        if accumulate:
            raise ValueError("accumulate needs the out tensors to add to")
        dx = torch.empty(N, H0, dtype=x.dtype, device=dev) if need_dx else None
        dW = torch.empty(V, H0, dtype=x.dtype, device=dev) if need_dW else None
        db = torch.empty_like(b) if (need_db and b is not None) else None
    # H padded to a multiple of 8: the library writes padded gradients, whose
    # first H0 columns are the result (with accumulate, they start from out's).
    kx, kW = dx, dW
    if H != H0:
        kx = _pad_hidden(dx) if (dx is not None and accumulate) else (
            torch.empty(N, H, dtype=x.dtype, device=dev) if dx is not None else None)
        kW = _pad_hidden(dW) if (dW is not None and accumulate) else (
            torch.empty(V, H, dtype=x.dtype, device=dev) if dW is not None else None)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        if keep is not None:
            _lib.flce_backward_kept(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                                    float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                                    _lib.options(logit_scale, accumulate, None), lse.data_ptr(), n_valid.data_ptr(),
                                    g.data_ptr(), keep.data_ptr(), keep.numel(), _ptr(kx), _ptr(kW), _ptr(db),
                                    workspace.data_ptr(), workspace.numel(), stream)
        elif logit_scale == 1.0 and not accumulate:
            _lib.flce_backward(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                               float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                               lse.data_ptr(), n_valid.data_ptr(), g.data_ptr(), _ptr(kx), _ptr(kW), _ptr(db),
                               workspace.data_ptr(), workspace.numel(), stream)
        else:
            _lib.flce_backward_ex(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                                  float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                                  _lib.options(logit_scale, accumulate, None), lse.data_ptr(), n_valid.data_ptr(),
                                  g.data_ptr(), _ptr(kx), _ptr(kW), _ptr(db), workspace.data_ptr(),
                                  workspace.numel(), stream)
    if H != H0:
        if dx is not None:
            dx.copy_(kx[:, :H0])
        if dW is not None:
            dW.copy_(kW[:, :H0])
    return dx, dW, db


def flce_fused_workspace_size(N: int, H: int, V: int, dtype: torch.dtype, has_bias: bool,
                              chunk_tokens: int = 0) -> Tuple[int, int]:
    """(workspace bytes, tokens per chunk) of the fused schedule."""
    return _lib.flce_fused_workspace_size(N, H, V, _DTYPES[dtype], has_bias, chunk_tokens)


def flce_fused_forward_backward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor], targets: torch.Tensor,
                                grad_loss: torch.Tensor, label_smoothing: float = 0.0, z_loss_scale: float = 0.0,
                                ignore_index: int = -100, reduction: str = "mean", need_dx: bool = True,
                                need_dW: bool = True, need_db: bool = True, chunk_tokens: int = 0,
                                workspace: Optional[torch.Tensor] = None, out: Optional[Tuple] = None,
                                logit_scale: float = 1.0, accumulate: bool = False,
                                return_z_loss: bool = False):
    """The fused schedule: loss and gradients in one pass, the gradients formed
    while the forward runs (grad_loss must be known up front: [1] for sum/mean,
    [N] for none).  Returns (loss, lse, n_valid, dx, dW, db) (and z_loss with
    return_z_loss); gradients are None where not requested."""
    if x.dim() == 2 and x.shape[1] % 8 != 0:
        raise ValueError("the fused schedule needs H % 8 == 0; pad x and W with zero columns")
    x, W, b, targets = _prep(x, W, b, targets)
    N, H = x.shape
    V = W.shape[0]
    dt, red = _dtype_code(x), _reduction_code(reduction)
    dev = x.device
    g = grad_loss.reshape(-1).to(device=dev, dtype=torch.float32).contiguous()
    if g.numel() != (N if reduction == "none" else 1):
        raise ValueError("grad_loss must have N entries for none and one otherwise")
    nbytes, _ = _lib.flce_fused_workspace_size(N, H, V, dt, b is not None, chunk_tokens)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    if out is not None:
        dx, dW, db = out
        _check_out(dx, (N, H), x, "out dx")
        _check_out(dW, (V, H), x, "out dW")
        _check_out(db, (V,), x, "out db")
    else:
        if accumulate:
            raise ValueError("accumulate needs the out tensors to add to")
        dx = torch.empty_like(x) if need_dx else None
        dW = torch.empty_like(W) if need_dW else None
        db = torch.empty_like(b) if (need_db and b is not None) else None
    loss = torch.empty(N if reduction == "none" else 1, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int64, device=dev)
    z_loss = torch.empty_like(loss) if return_z_loss else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _lib.flce_fused_forward_backward(x.data_ptr(), W.data_ptr(), _ptr(b), targets.data_ptr(), N, H, V, dt,
                                         float(label_smoothing), float(z_loss_scale), int(ignore_index), red,
                                         _lib.options(logit_scale, accumulate, _ptr(z_loss)), g.data_ptr(),
                                         int(chunk_tokens), loss.data_ptr(), lse.data_ptr(), n_valid.data_ptr(),
                                         _ptr(dx), _ptr(dW), _ptr(db), workspace.data_ptr(), workspace.numel(),
                                         stream)
    res = (loss, lse, n_valid, dx, dW, db)
    return res + (z_loss,) if return_z_loss else res


def _shard_hidden(x: torch.Tensor) -> None:
    # The shard entry points hand the caller fp32 dx partials of x's width,
    # so they take H as the library does (a multiple of 8) rather than pad.
    if x.dim() == 2 and x.shape[1] % 8 != 0:
        raise ValueError("the vocabulary-shard entry points need H % 8 == 0; pad x and W with zero columns")


def flce_shard_workspace_size(N: int, H: int, V_shard: int, dtype: torch.dtype,
                              has_bias: bool) -> Tuple[int, int, int]:
    """(forward, merge, backward) workspace bytes of one vocabulary shard."""
    return _lib.flce_shard_workspace_size(N, H, V_shard, _DTYPES[dtype], has_bias)


def flce_shard_forward(x: torch.Tensor, W_shard: torch.Tensor, b_shard: Optional[torch.Tensor],
                       targets: torch.Tensor, vocab_start: int, V_total: int, label_smoothing: float = 0.0,
                       ignore_index: int = -100, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-token statistics float32 [N, 4] = (m, d, sum z, z_y) over the shard's rows
    W[vocab_start : vocab_start + V_shard] (W_shard); targets are global indices."""
    _shard_hidden(x)
    x, W_shard, b_shard, targets = _prep(x, W_shard, b_shard, targets)
    N, H = x.shape
    V_shard = W_shard.shape[0]
    dt, dev = _dtype_code(x), x.device
    fwd_bytes, _, _ = _lib.flce_shard_workspace_size(N, H, V_shard, dt, b_shard is not None)
    if workspace is None or workspace.numel() < fwd_bytes:
        workspace = torch.empty(max(fwd_bytes, 1), dtype=torch.uint8, device=dev)
    stats = torch.empty(N, 4, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _lib.flce_shard_forward(x.data_ptr(), W_shard.data_ptr(), _ptr(b_shard), targets.data_ptr(), N, H, V_shard,
                                int(vocab_start), int(V_total), dt, float(label_smoothing), int(ignore_index),
                                stats.data_ptr(), workspace.data_ptr(), workspace.numel(), stream)
    return stats


def flce_shard_merge(stats: torch.Tensor, targets: torch.Tensor, V_total: int, label_smoothing: float = 0.0,
                     z_loss_scale: float = 0.0, ignore_index: int = -100, reduction: str = "mean",
                     workspace: Optional[torch.Tensor] = None):
    """Merge stacked shard statistics [num_shards, N, 4] into (loss, lse, n_valid), as
    flce_forward returns them for the whole head."""
    if stats.dim() != 3 or stats.shape[2] != 4 or stats.dtype != torch.float32:
        raise ValueError("stats must be float32 [num_shards, N, 4]")
    stats = stats.contiguous()
    num_shards, N = stats.shape[0], stats.shape[1]
    dev = stats.device
    targets = targets.reshape(-1).to(torch.int64).contiguous()
    _, merge_bytes, _ = _lib.flce_shard_workspace_size(N, 8, 1, _lib.FLCE_F32, False)
    if workspace is None or workspace.numel() < merge_bytes:
        workspace = torch.empty(max(merge_bytes, 1), dtype=torch.uint8, device=dev)
    loss = torch.empty(N if reduction == "none" else 1, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _lib.flce_shard_merge(stats.data_ptr(), num_shards, targets.data_ptr(), N, int(V_total),
                              float(label_smoothing), float(z_loss_scale), int(ignore_index),
                              _reduction_code(reduction), loss.data_ptr(), lse.data_ptr(), n_valid.data_ptr(),
                              workspace.data_ptr(), workspace.numel(), stream)
    return loss, lse, n_valid


def flce_shard_backward(x: torch.Tensor, W_shard: torch.Tensor, b_shard: Optional[torch.Tensor],
                        targets: torch.Tensor, vocab_start: int, V_total: int, lse: torch.Tensor,
                        n_valid: torch.Tensor, grad_loss: torch.Tensor, label_smoothing: float = 0.0,
                        z_loss_scale: float = 0.0, ignore_index: int = -100, reduction: str = "mean",
                        dx_partial: Optional[torch.Tensor] = None, accumulate_dx: bool = False,
                        need_dx: bool = True, need_dW: bool = True, need_db: bool = True,
                        workspace: Optional[torch.Tensor] = None):
    """Returns (dx_partial float32 [N, H], dW_shard, db_shard) (None where not requested).
    dx_partial: the buffer to write (or, with accumulate_dx, to add to); allocated if None."""
    _shard_hidden(x)
    x, W_shard, b_shard, targets = _prep(x, W_shard, b_shard, targets)
    N, H = x.shape
    V_shard = W_shard.shape[0]
    dt, red, dev = _dtype_code(x), _reduction_code(reduction), x.device
    _check_ctx(lse, n_valid, N, dev)
    g = grad_loss.reshape(-1).to(device=dev, dtype=torch.float32).contiguous()
    if g.numel() != (N if reduction == "none" else 1):
        raise ValueError("grad_loss must have N entries for none and one otherwise")
    if dx_partial is not None:
        if (dx_partial.shape != (N, H) or dx_partial.dtype != torch.float32 or not dx_partial.is_contiguous()
                or dx_partial.device != dev):
            raise ValueError(f"dx_partial must be a contiguous float32 [N, H] tensor on {dev}")
    elif need_dx:
        if accumulate_dx:
            raise ValueError("accumulate_dx needs dx_partial")
        dx_partial = torch.empty(N, H, dtype=torch.float32, device=dev)
    _, _, bwd_bytes = _lib.flce_shard_workspace_size(N, H, V_shard, dt, b_shard is not None)
    if workspace is None or workspace.numel() < bwd_bytes:
        workspace = torch.empty(max(bwd_bytes, 1), dtype=torch.uint8, device=dev)
    dW = torch.empty_like(W_shard) if need_dW else None
    db = torch.empty_like(b_shard) if (need_db and b_shard is not None) else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _lib.flce_shard_backward(x.data_ptr(), W_shard.data_ptr(), _ptr(b_shard), targets.data_ptr(), N, H,
                                 V_shard, int(vocab_start), int(V_total), dt, float(label_smoothing),
                                 float(z_loss_scale), int(ignore_index), red, lse.data_ptr(), n_valid.data_ptr(),
                                 g.data_ptr(), _ptr(dx_partial), bool(accumulate_dx), _ptr(dW), _ptr(db),
                                 workspace.data_ptr(), workspace.numel(), stream)
    return dx_partial, dW, db


def _activation_code(activation: str) -> int:
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(_lib.ACTIVATIONS)}")
    return _lib.ACTIVATIONS[activation]


def _dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t as the library reads it: contiguous from a 16-byte boundary (a copy if it is not)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _prep_layer(x, weights, rows, bias=(), kept=()):
    """The operands of a feed-forward call, checked and dense: x [N, H], weights
    [F, H], rows [N, F] (or None), bias [F] (or None); kept: float32
    pre-activations [N, F] (or None)."""
    if x.dim() != 2 or weights[0].dim() != 2:
        raise ValueError("x must be [N, H] and the weights [F, H]")
    if not x.is_cuda:
        raise ValueError("tensors must live on a GPU")
    dtype, dev, (N, H) = x.dtype, x.device, x.shape
    F = weights[0].shape[0]
    if H < 1 or F < 1:
        raise ValueError("H and F must be at least 1")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16, float16 or float32")

    def dense(t, shape, want):
        if t is None:
            return None
        if t.shape != shape:
            raise ValueError(f"expected a tensor of shape {tuple(shape)}, not {tuple(t.shape)}")
        if t.dtype != want:
            raise TypeError(f"expected a {want} tensor, not {t.dtype}: all tensors share x's dtype, but the kept "
                            "pre-activations are float32")
        if t.device != dev:
            raise ValueError("all tensors must be on one device")
        return _dense(t)

    nf = (N, F)
    return ([_dense(x), *[dense(w, (F, H), dtype) for w in weights]], [dense(t, nf, dtype) for t in rows],
            [dense(b, (F,), dtype) for b in bias], [dense(t, nf, torch.float32) for t in kept])


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream of a device, as its address; torch's own call for it makes no Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_HERE = contextlib.nullcontext()


def _on(dev):
    """The device made current, if it is not."""
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, dev) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    if workspace is None or workspace.numel() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace


# Tells autograd that the library wrote into a caller's tensor (or a list of
# them), so that a graph that saved it refuses to use it.
_wrote = torch.autograd.graph.increment_version


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel()


def flce_linear_workspace_size(N: int, H: int, F: int, dtype: torch.dtype,
                               activation: str = "none") -> Tuple[int, int]:
    """(forward bytes, backward bytes) of flce_linear_forward and flce_linear_backward."""
    return _lib.flce_linear_workspace_size(N, H, F, _DTYPES[dtype], _activation_code(activation))


def flce_linear_forward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, activation: str = "none", keep: bool = False,
                        workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """act(x W^T + b) + residual.  Returns (y, z): z the float32 pre-activations
    that flce_linear_backward takes, with keep and an activation, else None.
    out: the tensor to write y to; it may be residual, and may share memory with no
    other tensor of the call."""
    act = _activation_code(activation)
    N, F = x.shape[0], W.shape[0]
    (x, W), (residual_, out_), (b,), _ = _prep_layer(x, (W,), (residual, out), (b,))
    if out is not None and (out_ is not out or (residual_ is not residual and residual is out)):
        raise ValueError("out must be contiguous from a 16-byte boundary")
    dt, dev, H = _dtype_code(x), x.device, x.shape[1]
    y = out if out is not None else torch.empty(N, F, dtype=x.dtype, device=dev)
    z = torch.empty(N, F, dtype=torch.float32, device=dev) if keep and activation != "none" else None
    fwd_bytes, _ = _lib.flce_linear_workspace_size(N, H, F, dt, act)
    workspace = _workspace(workspace, fwd_bytes, dev)
    with _on(dev):
        stream = _raw_stream(dev.index)
        _lib.flce_linear_forward(x.data_ptr(), W.data_ptr(), _ptr(b), _ptr(residual_), N, H, F, dt, act, y.data_ptr(),
                                 _ptr(z), _ptr(workspace), _nbytes(workspace), stream)
    if out is not None:
        _wrote(out)
    return y, z


def flce_linear_backward(x: torch.Tensor, W: torch.Tensor, dy: torch.Tensor, z: Optional[torch.Tensor] = None,
                         activation: str = "none", need_dx: bool = True, need_dW: bool = True, need_db: bool = False,
                         workspace: Optional[torch.Tensor] = None):
    """Returns (dx, dW, db) in the input dtype (None where not requested); z as
    flce_linear_forward kept it.  The residual's gradient is dy."""
    act = _activation_code(activation)
    if activation == "none":
        z = None
    elif z is None:
        raise ValueError("z is what flce_linear_forward returned with keep=True")
    N, F = x.shape[0], W.shape[0]
    (x, W), (dy,), _, (z,) = _prep_layer(x, (W,), (dy,), kept=(z,))
    dt, dev, H = _dtype_code(x), x.device, x.shape[1]
    dx = torch.empty_like(x) if need_dx else None
    dW = torch.empty_like(W) if need_dW else None
    db = torch.empty(F, dtype=x.dtype, device=dev) if need_db else None
    _, bwd_bytes = _lib.flce_linear_workspace_size(N, H, F, dt, act)
    workspace = _workspace(workspace, bwd_bytes, dev)
    with _on(dev):
        stream = _raw_stream(dev.index)
        _lib.flce_linear_backward(x.data_ptr(), W.data_ptr(), _ptr(z), dy.data_ptr(), N, H, F, dt, act, _ptr(dx),
                                  _ptr(dW), _ptr(db), _ptr(workspace), _nbytes(workspace), stream)
    return dx, dW, db


def flce_glu_workspace_size(N: int, H: int, F: int, dtype: torch.dtype) -> Tuple[int, int]:
    """(forward bytes, backward bytes) of flce_glu_forward and flce_glu_backward."""
    return _lib.flce_glu_workspace_size(N, H, F, _DTYPES[dtype])


def flce_glu_forward(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, bg: Optional[torch.Tensor] = None,
                     bu: Optional[torch.Tensor] = None, activation: str = "silu", keep: bool = False,
                     workspace: Optional[torch.Tensor] = None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu).  Returns (h, g, u): the two
    projections, float32, that flce_glu_backward takes, with keep, else None."""
    act = _activation_code(activation)
    N, F = x.shape[0], Wg.shape[0]
    (x, Wg, Wu), _, (bg, bu), _ = _prep_layer(x, (Wg, Wu), (), (bg, bu))
    dt, dev, H = _dtype_code(x), x.device, x.shape[1]
    h = torch.empty(N, F, dtype=x.dtype, device=dev)
    g, u = (torch.empty(N, F, dtype=torch.float32, device=dev) for _ in range(2)) if keep else (None, None)
    fwd_bytes, _ = _lib.flce_glu_workspace_size(N, H, F, dt)
    workspace = _workspace(workspace, fwd_bytes, dev)
    with _on(dev):
        stream = _raw_stream(dev.index)
        _lib.flce_glu_forward(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), _ptr(bg), _ptr(bu), N, H, F, dt, act,
                              h.data_ptr(), _ptr(g), _ptr(u), _ptr(workspace), _nbytes(workspace), stream)
    return h, g, u


def flce_glu_backward(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, g: torch.Tensor, u: torch.Tensor,
                      dh: torch.Tensor, activation: str = "silu", need_dx: bool = True, need_dWg: bool = True,
                      need_dWu: bool = True, need_db: bool = False, workspace: Optional[torch.Tensor] = None):
    """Returns (dx, dWg, dWu, dbg, dbu) in the input dtype (None where not
    requested); g and u as flce_glu_forward kept them."""
    act = _activation_code(activation)
    if g is None or u is None:
        raise ValueError("g and u are what flce_glu_forward returned with keep=True")
    N, F = x.shape[0], Wg.shape[0]
    (x, Wg, Wu), (dh,), _, (g, u) = _prep_layer(x, (Wg, Wu), (dh,), kept=(g, u))
    dt, dev, H = _dtype_code(x), x.device, x.shape[1]
    dx = torch.empty_like(x) if need_dx else None
    dWg = torch.empty_like(Wg) if need_dWg else None
    dWu = torch.empty_like(Wu) if need_dWu else None
    dbg, dbu = ((torch.empty(F, dtype=x.dtype, device=dev), torch.empty(F, dtype=x.dtype, device=dev)) if need_db
                else (None, None))
    _, bwd_bytes = _lib.flce_glu_workspace_size(N, H, F, dt)
    workspace = _workspace(workspace, bwd_bytes, dev)
    with _on(dev):
        stream = _raw_stream(dev.index)
        _lib.flce_glu_backward(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), g.data_ptr(), u.data_ptr(), dh.data_ptr(),
                               N, H, F, dt, act, _ptr(dx), _ptr(dWg), _ptr(dWu), _ptr(dbg), _ptr(dbu),
                               _ptr(workspace), _nbytes(workspace), stream)
    return dx, dWg, dWu, dbg, dbu


def _is_dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one stretch of memory, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    expected = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != expected:
            return False
        expected *= size
    return True


def _extent(t: torch.Tensor):
    """The addresses of t's first byte and of the one past its last (equal when t is empty)."""
    lo = t.data_ptr()
    if t.numel() == 0:
        return lo, lo
    return lo, lo + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _share_memory(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two strided tensors have a byte in common: whether the difference of their addresses is a sum of
    whole multiples of their strides, each multiple within its dimension's range.  Strides are tried from the
    largest on, where few multiples come near enough; a search past 10000 steps counts as yes."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    span = {1: [1 - b.element_size(), a.element_size() - 1]}   # a byte's place in either element
    for t, end in ((a, 1), (b, 0)):
        for n, s in zip(t.shape, t.stride()):
            r = span.setdefault(s * t.element_size(), [0, 0])
            r[end] += (n - 1) if end else (1 - n)
    span.pop(0, None)
    steps = sorted(span.items(), reverse=True)
    below = [(0, 0)]   # what the strides from here on can add up to
    for s, (lo, hi) in reversed(steps):
        below.append((below[-1][0] + s * lo, below[-1][1] + s * hi))
    below.reverse()
    left = 10000

    def reach(i: int, diff: int) -> bool:
        nonlocal left
        if i == len(steps):
            return diff == 0
        s, (lo, hi) = steps[i]
        rest_lo, rest_hi = below[i + 1]
        for x in range(max(lo, -((rest_hi - diff) // s)), min(hi, (diff - rest_lo) // s) + 1):
            left -= 1
            if left < 0 or reach(i + 1, diff - s * x):
                return True
        return False

    return reach(0, b.data_ptr() - a.data_ptr())


def _check_written(tensors) -> None:
    """Refuses tensors of which two share memory, whatever their strides."""
    spans = sorted(((*_extent(t), i) for i, t in enumerate(tensors)))
    open_ = []   # tensors whose extent reaches past the current one's start
    for lo, hi, i in spans:
        open_ = [(h, j) for h, j in open_ if h > lo]
        for _, j in open_:
            if _share_memory(tensors[i], tensors[j]):
                raise ValueError("tensors to be scaled share memory")
        open_.append((hi, i))


# One attribute of every tensor of a list: a training step passes hundreds, and
# a Python loop over them would take longer than the kernels.
_contiguous, _address, _numel, _shape = (torch.Tensor.is_contiguous, torch.Tensor.data_ptr, torch.Tensor.numel,
                                         torch.Tensor.size)
_dtype, _device, _layout = (operator.attrgetter(a) for a in ("dtype", "device", "layout"))


def _prep_grads(grads, out):
    grads = list(grads)
    if not grads:
        raise ValueError("there are no gradients")
    dev = grads[0].device
    if not grads[0].is_cuda:
        raise ValueError("tensors must live on a GPU")
    if set(map(_device, grads)) != {dev}:
        raise ValueError("all gradients must be on one device")
    if set(map(_layout, grads)) != {torch.strided}:
        raise ValueError("gradients must be dense tensors")
    dtypes = list(map(_dtype, grads))
    for t in set(dtypes):
        if t not in _DTYPES:
            raise TypeError(f"unsupported dtype {t}; use bfloat16, float16 or float32")
    if out is not None:
        out = list(out)
        if (list(map(_shape, grads)) != list(map(_shape, out)) or dtypes != list(map(_dtype, out))
                or set(map(_device, out)) != {dev}):
            raise ValueError("out must have one tensor per gradient, of its shape, dtype and device")
    return grads, out, dev, _lib.dtype_array([_DTYPES[t] for t in dtypes])


def _norm_workspace(count, dev):
    nbytes = _lib.flce_grad_norm_workspace_size(count)
    return torch.empty(nbytes, dtype=torch.uint8, device=dev), torch.empty(1, dtype=torch.float32, device=dev)


def flce_grad_norm(grads, norm_type: float = 2.0) -> torch.Tensor:
    """The norm (2 or inf) over every element of every tensor, float32 [1]."""
    grads, _, dev, dtypes = _prep_grads(grads, None)
    if not all(map(_contiguous, grads)):
        grads = [g if _is_dense(g) else g.contiguous() for g in grads]
    workspace, norm = _norm_workspace(len(grads), dev)
    with _on(dev):
        stream = _raw_stream(dev.index)
        _lib.flce_grad_norm(_lib.pointer_array(map(_address, grads)), _lib.size_array(map(_numel, grads)), dtypes,
                            len(grads), float(norm_type), norm.data_ptr(), workspace.data_ptr(), workspace.numel(),
                            stream)
    return norm


def flce_clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, out=None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into the out tensors; returns the norm before, float32 [1].  No two tensors
    that are written may share memory."""
    return _clip(grads, max_norm, norm_type, None, out)


def flce_clip_grads_with_norm(grads, max_norm: float, norm: torch.Tensor, out=None) -> None:
    """flce_clip_grad_norm by a norm the caller has (float32, one element)."""
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one float32 value")
    _clip(grads, max_norm, 2.0, norm, out)


def _clip(grads, max_norm, norm_type, given, out):
    grads, out, dev, dtypes = _prep_grads(grads, out)
    if given is not None and given.device != dev:
        raise ValueError("norm and the gradients must be on one device")
    dst = grads if out is None else out
    src, tmp = grads, dst
    if not (all(map(_contiguous, grads)) and (out is None or all(map(_contiguous, out)))):
        # A gradient whose elements do not fill one stretch of memory goes through
        # a dense copy, as does one whose out tensor orders its elements otherwise.
        # The library sees the copies' addresses, so overlaps are looked for here.
        _check_written(dst)
        src, tmp = [], []
        for g, d in zip(grads, dst):
            if any(st == 0 and sz > 1 for st, sz in zip(d.stride(), d.shape)):
                raise ValueError("a tensor that repeats its elements cannot be scaled")
            plain = _is_dense(g) and _is_dense(d) and (g.stride() == d.stride()
                                                       or (g.is_contiguous() and d.is_contiguous()))
            src.append(g if plain else g.contiguous())
            tmp.append(d if plain else torch.empty(g.shape, dtype=g.dtype, device=dev))
    count = len(src)
    addresses, sizes = _lib.pointer_array(map(_address, src)), _lib.size_array(map(_numel, src))
    outs = None if tmp is grads else _lib.pointer_array(map(_address, tmp))
    norm = None
    with _on(dev):
        stream = _raw_stream(dev.index)
        if given is not None:
            _lib.flce_clip_grads_with_norm(addresses, outs, sizes, dtypes, count, float(max_norm), given.data_ptr(),
                                           stream)
        else:
            workspace, norm = _norm_workspace(count, dev)
            _lib.flce_clip_grad_norm(addresses, outs, sizes, dtypes, count, float(max_norm), float(norm_type),
                                     norm.data_ptr(), workspace.data_ptr(), workspace.numel(), stream)
    if tmp is not dst:
        for t, d in zip(tmp, dst):
            if t is not d:
                d.copy_(t)
    _wrote(dst)
    return norm


class FusedLinearCrossEntropyFunction(torch.autograd.Function):
    """loss = FLCE(x, target, weight, bias); saves only lse and the count."""

    @staticmethod
    def forward(ctx, x, target, weight, bias=None, ignore_index=-100, label_smoothing=0.0,
                z_loss_scale=0.0, reduction="mean", logit_scale=1.0, keep_first_slab=False):
        # keep_first_slab: the forward keeps the first vocabulary slab's logits
        # (flce_forward_keep) so the backward skips their recompute; the buffer
        # (about N x 16384 x 2 bytes) lives until the backward.
        if keep_first_slab:
            loss, lse, n_valid, keep = flce_forward_keep(x, weight, bias, target, label_smoothing, z_loss_scale,
                                                         ignore_index, reduction, logit_scale=logit_scale)
        else:
            (loss, lse, n_valid), keep = flce_forward(x, weight, bias, target, label_smoothing, z_loss_scale,
                                                      ignore_index, reduction, logit_scale=logit_scale), None
        ctx.save_for_backward(x, target, weight, bias, lse, n_valid)
        ctx.keep = keep
        ctx.opts = (ignore_index, label_smoothing, z_loss_scale, reduction, logit_scale)
        return loss if reduction == "none" else loss.reshape(())

    @staticmethod
    def backward(ctx, grad):
        x, target, weight, bias, lse, n_valid = ctx.saved_tensors
        ignore_index, eps, s, reduction, logit_scale = ctx.opts
        keep, ctx.keep = ctx.keep, None   # consumed: a second backward recomputes every slab
        args = (x, weight, bias, target, lse, n_valid, grad)
        kw = dict(label_smoothing=eps, z_loss_scale=s, ignore_index=ignore_index, reduction=reduction,
                  need_dx=ctx.needs_input_grad[0], need_dW=ctx.needs_input_grad[2],
                  need_db=bias is not None and ctx.needs_input_grad[3], logit_scale=logit_scale)
        if keep is not None:
            dx, dW, db = flce_backward_kept(*args, keep, **kw)
        else:
            dx, dW, db = flce_backward(*args, **kw)
        return dx, None, dW, db, None, None, None, None, None, None


def fused_linear_cross_entropy_loss(x, target, weight, bias=None, ignore_index=-100, label_smoothing=0.0,
                                    z_loss_scale=0.0, reduction="mean", logit_scale=1.0, keep_first_slab=False):
    """Functional form: x [N, H], target [N], weight [V, H], bias [V] or None."""
    return FusedLinearCrossEntropyFunction.apply(x, target, weight, bias, ignore_index, label_smoothing,
                                                 z_loss_scale, reduction, logit_scale, keep_first_slab)


class FusedLinearCrossEntropyLoss(torch.nn.Module):
    """Module form; x may be [..., H] and target [...]; they are flattened."""

    def __init__(self, ignore_index: int = -100, label_smoothing: float = 0.0, z_loss_scale: float = 0.0,
                 reduction: str = "mean", logit_scale: float = 1.0, keep_first_slab: bool = False):
        super().__init__()
        _reduction_code(reduction)
        self.logit_scale = logit_scale
        self.keep_first_slab = keep_first_slab
        self.ignore_index = ignore_index
        self.label_smoothing = label_smoothing
        self.z_loss_scale = z_loss_scale
        self.reduction = reduction

    def forward(self, x, target, weight, bias=None):
        return fused_linear_cross_entropy_loss(x.reshape(-1, x.shape[-1]), target.reshape(-1), weight, bias,
                                               self.ignore_index, self.label_smoothing, self.z_loss_scale,
                                               self.reduction, self.logit_scale, self.keep_first_slab)


class FusedLinearFunction(torch.autograd.Function):
    """y = act(x weight^T + bias) + residual; keeps the pre-activations if there is an activation.

    grad: whether a backward may follow.  needs_input_grad says which inputs require gradients, also under
    no_grad and inference_mode, and forward itself always runs without gradients."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, residual=None, activation="none", grad=True):
        y, z = flce_linear_forward(x, weight, bias, residual, activation, keep=grad and any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, weight, z)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dW = db = None
        if any(need[:3]):
            dx, dW, db = flce_linear_backward(x, weight, dy, z, ctx.activation, need[0], need[1], need[2])
        return dx, dW, db, dy if need[3] else None, None, None


class FusedGLUFunction(torch.autograd.Function):
    """h = act(x w_gate^T + b_gate) * (x w_up^T + b_up); keeps both projections.  grad: as in FusedLinearFunction."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", grad=True):
        h, g, u = flce_glu_forward(x, w_gate, w_up, b_gate, b_up, activation,
                                   keep=grad and any(ctx.needs_input_grad[:5]))
        ctx.save_for_backward(x, w_gate, w_up, g, u)
        ctx.activation = activation
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, w_gate, w_up, g, u = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dWg, dWu, dbg, dbu = flce_glu_backward(x, w_gate, w_up, g, u, dh, ctx.activation, need[0], need[1], need[2],
                                                   need[3] or need[4])
        return dx, dWg, dWu, dbg if need[3] else None, dbu if need[4] else None, None, None


def fused_linear(x, weight, bias=None, residual=None, activation="none"):
    """act(x weight^T + bias) + residual for x [..., H], residual [..., F]; differentiable."""
    lead, F = x.shape[:-1], weight.shape[0]
    if residual is not None:
        if residual.shape != (*lead, F):
            raise ValueError(f"residual must be {(*lead, F)}")
        residual = residual.reshape(-1, F)
    return FusedLinearFunction.apply(x.reshape(-1, x.shape[-1]), weight, bias, residual, activation,
                                     torch.is_grad_enabled()).reshape(*lead, F)


def fused_glu(x, w_gate, w_up, b_gate=None, b_up=None, activation="silu"):
    """act(x w_gate^T + b_gate) * (x w_up^T + b_up) for x [..., H]; differentiable."""
    return FusedGLUFunction.apply(x.reshape(-1, x.shape[-1]), w_gate, w_up, b_gate, b_up, activation,
                                  torch.is_grad_enabled()).reshape(*x.shape[:-1], w_gate.shape[0])


class GatedFeedForward(torch.nn.Module):
    """A gated feed-forward block: down(act(gate(x)) * up(x)) + residual, two fused calls."""

    def __init__(self, hidden: int, intermediate: int, activation: str = "silu", bias: bool = False, device=None,
                 dtype=None):
        super().__init__()
        _activation_code(activation)
        kw = dict(bias=bias, device=device, dtype=dtype)
        self.activation = activation
        self.gate_proj = torch.nn.Linear(hidden, intermediate, **kw)
        self.up_proj = torch.nn.Linear(hidden, intermediate, **kw)
        self.down_proj = torch.nn.Linear(intermediate, hidden, **kw)

    def forward(self, x, residual=None):
        h = fused_glu(x, self.gate_proj.weight, self.up_proj.weight, self.gate_proj.bias, self.up_proj.bias,
                      self.activation)
        return fused_linear(h, self.down_proj.weight, self.down_proj.bias, residual)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0) -> torch.Tensor:
    """Clips the parameters' gradients in place by their global norm, by the formula of
    torch.nn.utils.clip_grad_norm_; returns the norm before (a scalar tensor).  norm_type is 2 or infinity;
    the gradients are on one device, and no two of them share memory (no parameter comes twice)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.zeros((), dtype=torch.float32)
    return flce_clip_grad_norm(grads, max_norm, norm_type).reshape(())
