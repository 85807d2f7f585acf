"""Tensor-level helpers over the C ABI (PyTorch supplies memory and streams only).

``fused_kl_fwd_bwd`` / ``fused_kl_fwd`` allocate outputs and the workspace
with PyTorch on the inputs' device and call the library on the current
stream.  ``FusedChunkedKL`` is an autograd Function that computes the
gradients inside its forward (one fused library call) and scales them by the
upstream gradient in backward.
"""
from __future__ import annotations

import dataclasses
import functools
from operator import index as _int

import torch
from torch.autograd.function import once_differentiable

from . import (FcklCeProblem, FcklError, FcklNormProblem, FcklProblem, FCKL_BFLOAT, FCKL_FLOAT,
               FCKL_GRAD_BFLOAT, FCKL_GRAD_FLOAT, FCKL_LABELS_INT, FCKL_LABELS_LONG,
               FCKL_NORM_POST, FCKL_NORM_PRE, FCKL_OK, FCKL_REDUCE_MEAN, FCKL_REDUCE_SUM,
               fckl_block_norm_bwd, fckl_block_norm_fwd, fckl_block_norm_workspace_bytes, fckl_ce_bwd, fckl_ce_fwd, fckl_ce_fwd_bwd, fckl_ce_workspace_bytes, fckl_check,
               fckl_fwd, fckl_fwd_bwd, fckl_fwd_bwd_host, fckl_fwd_bwd_sliced,
               fckl_host_workspace_bytes, fckl_scale_gradient, fckl_workspace_bytes)

__all__ = ["make_problem", "alloc_workspace", "fused_kl_fwd", "fused_kl_fwd_bwd", "student_entropy",
           "select_top_rows", "fused_kl_rows", "arrays_to_device",
           "fused_kl_from_host", "alloc_host_workspace", "fused_kl_fwd_bwd_host",
           "fused_kl_fwd_bwd_sliced",
           "FusedChunkedKL", "fused_chunked_kl_loss", "fused_ce_fwd", "fused_ce_fwd_bwd",
           "fused_ce_bwd", "FusedCrossEntropy", "fused_cross_entropy_loss", "block_norm_fwd",
           "block_norm_bwd", "BlockNorm", "block_norm", "TailNorm"]


def _bits(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.bfloat16:
        return t
    if t.dtype in (torch.int16, torch.uint16):
        return t.view(torch.bfloat16)
    raise TypeError(f"expected bfloat16 (or its uint16 bits), got {t.dtype}")


def make_problem(hidden, W, topk_idx, T=1.0, chunk=0, teacher=0, n_valid_total=0,
                 dw_rows=0) -> FcklProblem:
    N, H = hidden.shape
    V = W.shape[0]
    K = topk_idx.shape[1]
    return FcklProblem(N, H, V, K, T, chunk, teacher, n_valid_total, dw_rows)


def alloc_workspace(prob: FcklProblem, device) -> torch.Tensor:
    nbytes = fckl_workspace_bytes(prob)
    if nbytes == 0:
        raise FcklError(1, "fckl_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _check_shapes(hidden, W, topk_idx=None, topk_logit=None, row_mask=None):
    """Shapes and dtypes the library reads without further checks: hidden [N,H],
    W [V,H], topk_idx int32 and topk_logit float32 [N,K], row_mask uint8 [N]."""
    if hidden.dim() != 2 or W.dim() != 2 or W.shape[1] != hidden.shape[1]:
        raise ValueError(f"hidden must be [N,H] and W [V,H]; got {tuple(hidden.shape)} "
                         f"and {tuple(W.shape)}")
    N = hidden.shape[0]
    if topk_idx is not None:
        if (topk_idx.dim() != 2 or tuple(topk_logit.shape) != tuple(topk_idx.shape)
                or topk_idx.shape[0] != N):
            raise ValueError(f"topk_idx and topk_logit must both be [N={N},K]; got "
                             f"{tuple(topk_idx.shape)} and {tuple(topk_logit.shape)}")
        if topk_idx.dtype != torch.int32 or topk_logit.dtype != torch.float32:
            raise TypeError("topk_idx must be int32 and topk_logit float32")
    if row_mask is not None:
        if row_mask.dtype != torch.uint8 or row_mask.numel() != N:
            raise TypeError(f"row_mask must be a uint8 tensor of N={N} entries")


def _check_placement(cuda, tensors):
    """Every named tensor contiguous and on one CUDA device (cuda=True) or on
    the host (cuda=False)."""
    devices = set()
    for name, t in tensors:
        if t is None:
            continue
        where = "CUDA" if cuda else "CPU"
        if t.is_cuda != cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {where} tensor")
        devices.add(t.device)
    if cuda and len(devices) > 1:
        raise ValueError(f"all tensors must be on one device; got {sorted(map(str, devices))}")


def _workspace(workspace, prob, device, host_inputs=False):
    """The caller's workspace (a contiguous uint8 tensor on ``device``; the
    library checks its size), or a new one of the size the problem needs."""
    if workspace is None:
        return (alloc_host_workspace if host_inputs else alloc_workspace)(prob, device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def _check_out(out, prob, device, with_loss=True):
    """Caller-supplied outputs: (loss[>=1],) dH [N,H], dW [V,H], contiguous float32
    tensors on the inputs' device."""
    names = ("loss", "dH", "dW") if with_loss else ("dH", "dW")
    if len(out) != len(names):
        raise ValueError("out must be (" + ", ".join(names) + ")")
    want = {"loss": None, "dH": (prob.N, prob.H), "dW": (prob.V, prob.H)}
    for name, t in zip(names, out):
        shape_ok = t.numel() >= 1 if want[name] is None else tuple(t.shape) == want[name]
        if (not shape_ok or t.dtype != torch.float32 or not t.is_contiguous()
                or t.device != device):
            raise ValueError(f"out {name} must be a contiguous float32 tensor on {device}"
                             + ("" if want[name] is None else f" of shape {want[name]}"))


def _check_inputs(hidden, W, topk_idx, topk_logit, row_mask):
    _check_shapes(hidden, W, topk_idx, topk_logit, row_mask)
    _check_placement(True, (("hidden", hidden), ("W", W), ("topk_idx", topk_idx),
                            ("topk_logit", topk_logit), ("row_mask", row_mask)))


def fused_kl_fwd_bwd(hidden, W, topk_idx, topk_logit, row_mask=None, T=1.0, chunk=0,
                     workspace=None, want_row_loss=False, check=True, out=None, teacher=0,
                     n_valid_total=0, dw_rows=0):
    """Returns (loss[1], row_loss[N] or None, dH[N,H] fp32, dW[V,H] fp32).

    ``out``: optional (loss, dH, dW) tensors to write into instead of allocating.
    ``n_valid_total``: N_v for the mean and gradient scale when these rows are one
    shard of a larger batch (0 = the valid rows of this call).
    ``dw_rows``: group chunks so that each dW GEMM covers at least this many
    rows (0 = one dW GEMM per chunk)."""
    hidden, W = _bits(hidden), _bits(W)
    _check_inputs(hidden, W, topk_idx, topk_logit, row_mask)
    prob = make_problem(hidden, W, topk_idx, T, chunk, teacher, n_valid_total, dw_rows)
    dev = hidden.device
    workspace = _workspace(workspace, prob, dev)
    if out is not None:
        _check_out(out, prob, dev)
        loss, dH, dW = out
    else:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        dH = torch.empty(prob.N, prob.H, dtype=torch.float32, device=dev)
        dW = torch.empty(prob.V, prob.H, dtype=torch.float32, device=dev)
    row_loss = torch.empty(prob.N, dtype=torch.float32, device=dev) if want_row_loss else None
    stream = torch.cuda.current_stream(dev).cuda_stream
    st = fckl_fwd_bwd(prob, hidden.data_ptr(), W.data_ptr(), topk_idx.data_ptr(),
                      topk_logit.data_ptr(), None if row_mask is None else row_mask.data_ptr(),
                      loss.data_ptr(), None if row_loss is None else row_loss.data_ptr(),
                      dH.data_ptr(), dW.data_ptr(), workspace.data_ptr(), workspace.numel(),
                      stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_fwd_bwd")
    if check:
        st = fckl_check(workspace.data_ptr(), stream)
        if st != FCKL_OK:
            raise FcklError(st, "fckl_check")
    return loss, row_loss, dH, dW


def fused_kl_fwd_bwd_sliced(hidden, W, topk_idx, topk_logit, row_mask=None, T=1.0, chunk=0,
                            workspace=None, n_slices=4, teacher=0, n_valid_total=0, out=None,
                            dw_rows=0):
    """fused_kl_fwd_bwd whose last dW launch is split into ``n_slices``
    vocabulary slices.  Returns (loss[1], dH, dW, slices) with slices a list of
    (row0, row1, event): dW[row0:row1] is final once ``event`` (a
    torch.cuda.Event recorded on the current stream) has completed."""
    hidden, W = _bits(hidden), _bits(W)
    _check_inputs(hidden, W, topk_idx, topk_logit, row_mask)
    prob = make_problem(hidden, W, topk_idx, T, chunk, teacher, n_valid_total, dw_rows)
    dev = hidden.device
    workspace = _workspace(workspace, prob, dev)
    if out is None:
        out = (torch.empty(1, dtype=torch.float32, device=dev),
               torch.empty(prob.N, prob.H, dtype=torch.float32, device=dev),
               torch.empty(prob.V, prob.H, dtype=torch.float32, device=dev))
    _check_out(out, prob, dev)
    loss, dH, dW = out
    stream = torch.cuda.current_stream(dev)
    events = [torch.cuda.Event() for _ in range(n_slices)]
    for e in events:
        e.record(stream)  # creates the CUDA event; the call records it again
    st, rows = fckl_fwd_bwd_sliced(prob, hidden.data_ptr(), W.data_ptr(), topk_idx.data_ptr(),
                                   topk_logit.data_ptr(),
                                   None if row_mask is None else row_mask.data_ptr(),
                                   loss.data_ptr(), None, dH.data_ptr(), dW.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), stream.cuda_stream,
                                   [e.cuda_event for e in events])
    if st != FCKL_OK:
        raise FcklError(st, "fckl_fwd_bwd_sliced")
    slices = [(rows[i], rows[i + 1], events[i]) for i in range(n_slices)]
    return loss, dH, dW, slices


def fused_kl_fwd(hidden, W, topk_idx, topk_logit, row_mask=None, T=1.0, chunk=0,
                 workspace=None, want_row_loss=False, check=True, teacher=0):
    """Returns (loss[1], row_loss[N] or None)."""
    hidden, W = _bits(hidden), _bits(W)
    _check_inputs(hidden, W, topk_idx, topk_logit, row_mask)
    prob = make_problem(hidden, W, topk_idx, T, chunk, teacher)
    dev = hidden.device
    workspace = _workspace(workspace, prob, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    row_loss = torch.empty(prob.N, dtype=torch.float32, device=dev) if want_row_loss else None
    stream = torch.cuda.current_stream(dev).cuda_stream
    st = fckl_fwd(prob, hidden.data_ptr(), W.data_ptr(), topk_idx.data_ptr(),
                  topk_logit.data_ptr(), None if row_mask is None else row_mask.data_ptr(),
                  loss.data_ptr(), None if row_loss is None else row_loss.data_ptr(),
                  workspace.data_ptr(), workspace.numel(), stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_fwd")
    if check:
        st = fckl_check(workspace.data_ptr(), stream)
        if st != FCKL_OK:
            raise FcklError(st, "fckl_check")
    return loss, row_loss


def alloc_host_workspace(prob: FcklProblem, device) -> torch.Tensor:
    nbytes = fckl_host_workspace_bytes(prob)
    if nbytes == 0:
        raise FcklError(1, "fckl_host_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fused_kl_fwd_bwd_host(hidden, W, topk_idx, topk_logit, row_mask=None, T=1.0, chunk=0,
                          workspace=None, out=None, loss_host=None, check=True, dw_rows=0):
    """Forward + backward from HOST inputs (contiguous CPU tensors; pinned for
    overlapped copies): hidden bf16 [N,H], topk_idx int32 [N,K], topk_logit
    float32 [N,K], row_mask uint8 [N] or None.  W is a CUDA bf16 tensor.  The
    library streams the inputs to the device chunk by chunk, overlapped with
    the kernels.  Returns (loss as a Python float, dH, dW); the loss read
    synchronises the stream."""
    hidden, W = _bits(hidden), _bits(W)
    _check_shapes(hidden, W, topk_idx, topk_logit, row_mask)
    _check_placement(False, (("hidden", hidden), ("topk_idx", topk_idx),
                             ("topk_logit", topk_logit), ("row_mask", row_mask)))
    _check_placement(True, (("W", W),))
    prob = make_problem(hidden, W, topk_idx, T, chunk, dw_rows=dw_rows)
    dev = W.device
    workspace = _workspace(workspace, prob, dev, host_inputs=True)
    if out is None:
        out = (torch.empty(prob.N, prob.H, dtype=torch.float32, device=dev),
               torch.empty(prob.V, prob.H, dtype=torch.float32, device=dev))
    _check_out(out, prob, dev, with_loss=False)
    dH, dW = out
    if loss_host is None:
        loss_host = torch.empty(1, dtype=torch.float32, pin_memory=True)
    stream = torch.cuda.current_stream(dev)
    st = fckl_fwd_bwd_host(prob, hidden.data_ptr(), W.data_ptr(), topk_idx.data_ptr(),
                           topk_logit.data_ptr(),
                           None if row_mask is None else row_mask.data_ptr(),
                           loss_host.data_ptr(), dH.data_ptr(), dW.data_ptr(),
                           workspace.data_ptr(), workspace.numel(), stream.cuda_stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_fwd_bwd_host")
    if check:
        st = fckl_check(workspace.data_ptr(), stream.cuda_stream)
        if st != FCKL_OK:
            raise FcklError(st, "fckl_check")
    else:
        stream.synchronize()
    return float(loss_host[0]), dH, dW


def fused_kl_from_host(dev_bufs: dict, host: dict, T=1.0, chunk=0, workspace=None, out=None):
    """End-to-end call from pinned host arrays: copies the inputs host->device on
    the current stream, runs fused forward+backward, and reads the loss back.
    ``dev_bufs`` holds preallocated device tensors with the same keys as
    ``host`` (hidden, W, topk_idx, topk_logit, row_mask).  Returns (loss as a
    Python float, dH, dW)."""
    for k, h in host.items():
        dev_bufs[k].copy_(h, non_blocking=True)
    loss, _, dH, dW = fused_kl_fwd_bwd(dev_bufs["hidden"], dev_bufs["W"], dev_bufs["topk_idx"],
                                       dev_bufs["topk_logit"], dev_bufs.get("row_mask"), T=T,
                                       chunk=chunk, workspace=workspace, check=False, out=out)
    return float(loss.item()), dH, dW


class FusedChunkedKL(torch.autograd.Function):
    """loss = FusedChunkedKL.apply(hidden_bf16, W_bf16, topk_idx, topk_logit, row_mask, T, chunk)

    Gradients flow to hidden and W (returned as fp32 tensors cast to the input
    dtype); the fused call computes them in forward."""

    @staticmethod
    def forward(ctx, hidden, W, topk_idx, topk_logit, row_mask, T, chunk):
        loss, _, dH, dW = fused_kl_fwd_bwd(hidden, W, topk_idx, topk_logit, row_mask, T, chunk)
        ctx.save_for_backward(dH, dW)
        ctx.dtypes = (hidden.dtype, W.dtype)
        return loss[0]

    @staticmethod
    def backward(ctx, grad_out):
        dH, dW = ctx.saved_tensors
        return ((dH * grad_out).to(ctx.dtypes[0]), (dW * grad_out).to(ctx.dtypes[1]),
                None, None, None, None, None)


def fused_chunked_kl_loss(hidden, W, topk_idx, topk_logit, row_mask=None, T=1.0, chunk=0,
                          norm=None):
    """``norm``: a TailNorm; ``hidden`` is then the residual stream, and the loss
    runs over its normed rows."""
    if norm is not None:
        hidden = norm(hidden)
    return FusedChunkedKL.apply(hidden, W, topk_idx, topk_logit, row_mask, T, chunk)


def arrays_to_device(hidden_bits, W_bits, topk_idx, topk_logit, row_mask, device="cuda"):
    """numpy arrays (bf16 bit patterns as uint16, int32 ids, float32 logits,
    uint8 mask or None) -> contiguous device tensors, in that order."""
    import numpy as np

    def t(a, dt):
        return torch.from_numpy(np.ascontiguousarray(a).view(dt))

    out = [t(hidden_bits, np.int16).to(device).view(torch.bfloat16),
           t(W_bits, np.int16).to(device).view(torch.bfloat16),
           t(topk_idx, np.int32).to(device),
           t(topk_logit, np.float32).to(device),
           None if row_mask is None else t(row_mask, np.uint8).to(device)]
    return tuple(out)


def student_entropy(hidden, W, row_mask=None, T=1.0, chunk=0, workspace=None, check=True):
    """Per-row student entropy H(softmax(W h / T)) in nats, [N] fp32 (0 for masked rows)."""
    from . import fckl_student_entropy
    hidden, W = _bits(hidden), _bits(W)
    _check_shapes(hidden, W, row_mask=row_mask)
    _check_placement(True, (("hidden", hidden), ("W", W), ("row_mask", row_mask)))
    N, H = hidden.shape
    prob = FcklProblem(N, H, W.shape[0], 1, T, chunk)
    dev = hidden.device
    workspace = _workspace(workspace, prob, dev)
    ent = torch.empty(N, dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    st = fckl_student_entropy(prob, hidden.data_ptr(), W.data_ptr(),
                              None if row_mask is None else row_mask.data_ptr(), ent.data_ptr(),
                              workspace.data_ptr(), workspace.numel(), stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_student_entropy")
    if check:
        st = fckl_check(workspace.data_ptr(), stream)
        if st != FCKL_OK:
            raise FcklError(st, "fckl_check")
    return ent


def select_top_rows(score, n_select, row_mask=None):
    """(rows int32 [n_select] ascending, padded with -1; count int32 [1]) on device."""
    from . import fckl_select_top_rows
    if score.dtype != torch.float32 or score.dim() != 1:
        raise TypeError("score must be a 1-D float32 tensor")
    if row_mask is not None and (row_mask.dtype != torch.uint8 or row_mask.numel() != score.numel()):
        raise TypeError("row_mask must be a uint8 tensor with one entry per score")
    _check_placement(True, (("score", score), ("row_mask", row_mask)))
    N = score.numel()
    rows = torch.empty(n_select, dtype=torch.int32, device=score.device)
    count = torch.empty(1, dtype=torch.int32, device=score.device)
    st = fckl_select_top_rows(score.data_ptr(), None if row_mask is None else row_mask.data_ptr(),
                              N, n_select, rows.data_ptr(), count.data_ptr(),
                              torch.cuda.current_stream(score.device).cuda_stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_select_top_rows")
    return rows, count


def fused_kl_rows(hidden, W, topk_idx, topk_logit, rows, T=1.0, chunk=0, workspace=None,
                  grads=True, want_row_loss=False, check=True, teacher=0, dw_rows=0):
    """Loss (and dH, dW) over the listed rows only.  Returns (loss, row_loss, dH, dW)."""
    from . import fckl_fwd_bwd_rows
    hidden, W = _bits(hidden), _bits(W)
    if rows.dtype != torch.int32 or rows.dim() != 1:
        raise TypeError("rows must be a 1-D int32 tensor")
    _check_inputs(hidden, W, topk_idx, topk_logit, None)
    _check_placement(True, (("hidden", hidden), ("rows", rows)))
    prob = make_problem(hidden, W, topk_idx, T, chunk, teacher, dw_rows=dw_rows)
    dev = hidden.device
    workspace = _workspace(workspace, prob, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    row_loss = torch.empty(prob.N, dtype=torch.float32, device=dev) if want_row_loss else None
    dH = torch.empty(prob.N, prob.H, dtype=torch.float32, device=dev) if grads else None
    dW = torch.empty(prob.V, prob.H, dtype=torch.float32, device=dev) if grads else None
    stream = torch.cuda.current_stream(dev).cuda_stream
    st = fckl_fwd_bwd_rows(prob, hidden.data_ptr(), W.data_ptr(), topk_idx.data_ptr(),
                           topk_logit.data_ptr(), rows.data_ptr(), rows.numel(), loss.data_ptr(),
                           None if row_loss is None else row_loss.data_ptr(),
                           None if dH is None else dH.data_ptr(),
                           None if dW is None else dW.data_ptr(), workspace.data_ptr(),
                           workspace.numel(), stream)
    if st != FCKL_OK:
        raise FcklError(st, "fckl_fwd_bwd_rows")
    if check:
        st = fckl_check(workspace.data_ptr(), stream)
        if st != FCKL_OK:
            raise FcklError(st, "fckl_check")
    return loss, row_loss, dH, dW


# ---------------------------------------------------------------- cross entropy
_REDUCTIONS = {"mean": FCKL_REDUCE_MEAN, "sum": FCKL_REDUCE_SUM}
_GRAD_TYPES = {torch.float32: FCKL_GRAD_FLOAT, torch.bfloat16: FCKL_GRAD_BFLOAT}
_LABEL_TYPES = {torch.int32: FCKL_LABELS_INT, torch.int64: FCKL_LABELS_LONG}


def _ptr(t):
    return None if t is None else t.data_ptr()


# The stream handle without building a torch.cuda.Stream (a call of a few
# microseconds on the GPU would wait for it).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_device(index, call, *args):
    """call(*args, stream) with device ``index`` current, on its current stream."""
    if index == torch.cuda.current_device():
        return call(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return call(*args, _raw_stream(index))


def _placed(index, tensors):
    """Whether every tensor (None aside) is contiguous on CUDA device ``index``."""
    for t in tensors:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            return False
    return index >= 0


# The caches below are keyed by plain numbers: a tensor would be remembered by its
# identity, and its later values never seen.  So options become float / int first.
@functools.lru_cache(maxsize=256)
def _ce_problem(*fields):
    """The problem of these sizes and options, and its workspace sizes without and
    with gradients."""
    prob = FcklCeProblem(*fields)
    return prob, fckl_ce_workspace_bytes(prob, False), fckl_ce_workspace_bytes(prob, True)


_norm_struct = functools.lru_cache(maxsize=256)(FcklNormProblem)


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(prob_fields):
    return fckl_block_norm_workspace_bytes(FcklNormProblem(*prob_fields))


def _ce_setup(hidden, W, labels, rows, T, label_smoothing, z_loss, ignore_index, reduction, chunk,
              n_valid_total, grad_dtype, workspace, gradients):
    """Checks, the problem and the workspace of a cross-entropy call.  ``rows``:
    (name, tensor or None) of the per-row float32 inputs."""
    if hidden.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        hidden, W = _bits(hidden), _bits(W)
    if hidden.dim() != 2 or W.dim() != 2 or W.shape[1] != hidden.shape[1]:
        _check_shapes(hidden, W)
    N, H = hidden.shape
    index = hidden.get_device()
    placed = _placed(index, (hidden, W, labels))
    if labels.dtype not in _LABEL_TYPES:
        raise TypeError(f"labels must be int32 or int64, got {labels.dtype}")
    if labels.shape != (N,):
        raise ValueError(f"labels must be [N={N}], got {tuple(labels.shape)}")
    for name, t in rows:
        if t is not None:
            if t.dtype != torch.float32 or t.shape != (N,):
                raise TypeError(f"{name} must be a float32 tensor [N={N}]")
            placed = placed and t.get_device() == index and t.is_contiguous()
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}, got {reduction!r}")
    if grad_dtype not in _GRAD_TYPES:
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    if not placed:
        _check_placement(True, [("hidden", hidden), ("W", W), ("labels", labels)] + list(rows))
    prob, *nbytes = _ce_problem(N, H, W.shape[0], float(T), float(label_smoothing), float(z_loss),
                                _REDUCTIONS[reduction], _int(ignore_index), _int(chunk),
                                _int(n_valid_total), _LABEL_TYPES[labels.dtype],
                                _GRAD_TYPES[grad_dtype])
    if workspace is None:
        if nbytes[gradients] == 0:
            raise FcklError(1, "fckl_ce_workspace_bytes")
        workspace = torch.empty(nbytes[gradients], dtype=torch.uint8, device=hidden.device)
    elif (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
          or workspace.device != hidden.device):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {hidden.device}")
    return hidden, W, prob, workspace


def _check_grad_out(name, t, shape, dtype, device):
    if (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()
            or t.device != device):
        raise ValueError(f"out {name} must be a contiguous {dtype} tensor {shape} on {device}")


def _finish(status, where, workspace, check):
    if status == FCKL_OK and check:
        where = "fckl_check"
        status = _on_device(workspace.get_device(), fckl_check, workspace.data_ptr())
    if status != FCKL_OK:
        raise FcklError(status, where)


def fused_ce_fwd(hidden, W, labels, row_weight=None, T=1.0, label_smoothing=0.0, z_loss=0.0,
                 ignore_index=-100, reduction="mean", chunk=0, workspace=None, check=True,
                 n_valid_total=0):
    """Cross entropy of softmax(hidden W^T / T) against ``labels`` (int32 or int64
    [N]; rows whose label is ``ignore_index`` are left out).  Returns (loss[1],
    row_loss[N], lse[N]), float32; row_loss is without ``row_weight`` (float32
    [N], the rows' weights in ``loss``).  ``reduction``: "mean" over the rows
    that count (``n_valid_total`` > 0 replaces their number) or "sum"."""
    hidden, W, prob, workspace = _ce_setup(hidden, W, labels, (("row_weight", row_weight),), T,
                                           label_smoothing, z_loss, ignore_index, reduction, chunk,
                                           n_valid_total, torch.float32, workspace, False)
    dev = hidden.device
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    row_loss = torch.empty(prob.N, dtype=torch.float32, device=dev)
    lse = torch.empty(prob.N, dtype=torch.float32, device=dev)
    st = _on_device(dev.index, fckl_ce_fwd, prob, hidden.data_ptr(), W.data_ptr(),
                    labels.data_ptr(), _ptr(row_weight), loss.data_ptr(), row_loss.data_ptr(),
                    lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    _finish(st, "fckl_ce_fwd", workspace, check)
    return loss, row_loss, lse


def _fused_ce_fwd_bwd(hidden, W, labels, row_weight, T, label_smoothing, z_loss, ignore_index,
                      reduction, chunk, workspace, check, out, grad_dtype, n_valid_total,
                      want=(True, True), want_lse=False):
    hidden, W, prob, workspace = _ce_setup(hidden, W, labels, (("row_weight", row_weight),), T,
                                           label_smoothing, z_loss, ignore_index, reduction, chunk,
                                           n_valid_total, grad_dtype, workspace, True)
    dev = hidden.device
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must be (loss, dH, dW)")
        loss, dH, dW = out
        _check_grad_out("loss", loss, (1,), torch.float32, dev)
        _check_grad_out("dH", dH, (prob.N, prob.H), grad_dtype, dev)
        _check_grad_out("dW", dW, (prob.V, prob.H), grad_dtype, dev)
    else:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        dH = torch.empty_like(hidden, dtype=grad_dtype) if want[0] else None
        dW = torch.empty_like(W, dtype=grad_dtype) if want[1] else None
    row_loss = torch.empty(prob.N, dtype=torch.float32, device=dev)
    lse = torch.empty(prob.N, dtype=torch.float32, device=dev) if want_lse else None
    st = _on_device(dev.index, fckl_ce_fwd_bwd, prob, hidden.data_ptr(), W.data_ptr(),
                    labels.data_ptr(), _ptr(row_weight), loss.data_ptr(), row_loss.data_ptr(),
                    _ptr(lse), _ptr(dH), _ptr(dW), workspace.data_ptr(), workspace.numel())
    _finish(st, "fckl_ce_fwd_bwd", workspace, check)
    return loss, row_loss, lse, dH, dW


def fused_ce_fwd_bwd(hidden, W, labels, row_weight=None, T=1.0, label_smoothing=0.0, z_loss=0.0,
                     ignore_index=-100, reduction="mean", chunk=0, workspace=None, check=True,
                     out=None, grad_dtype=torch.float32, n_valid_total=0):
    """fused_ce_fwd with the gradients of ``loss`` in the same call: returns
    (loss[1], row_loss[N], dH[N,H], dW[V,H]), the gradients in ``grad_dtype``
    (float32 or bfloat16; either way the dlogits are rounded to bfloat16 for the
    tensor cores, so float32 spares the result's own rounding and no more).
    ``out``: optional (loss, dH, dW) to write into."""
    loss, row_loss, _, dH, dW = _fused_ce_fwd_bwd(
        hidden, W, labels, row_weight, T, label_smoothing, z_loss, ignore_index, reduction, chunk,
        workspace, check, out, grad_dtype, n_valid_total)
    return loss, row_loss, dH, dW


def fused_ce_bwd(hidden, W, labels, lse, row_grad, T=1.0, label_smoothing=0.0, z_loss=0.0,
                 ignore_index=-100, chunk=0, workspace=None, check=True, out=None,
                 grad_dtype=torch.float32, want=(True, True)):
    """Gradients of sum(row_grad * row_loss) for the row losses and ``lse`` that
    fused_ce_fwd returned on the same inputs; row_grad float32 [N], of either
    sign.  Returns (dH[N,H], dW[V,H]) in ``grad_dtype`` (see fused_ce_fwd_bwd);
    ``want`` = (dH, dW): leave one out (None)."""
    if lse is None or row_grad is None:
        raise TypeError("lse and row_grad must be float32 tensors [N]")
    if not any(want):
        raise ValueError("want leaves out both gradients")
    hidden, W, prob, workspace = _ce_setup(hidden, W, labels,
                                           (("lse", lse), ("row_grad", row_grad)), T,
                                           label_smoothing, z_loss, ignore_index, "sum", chunk, 0,
                                           grad_dtype, workspace, True)
    dev = hidden.device
    if out is not None:
        if len(out) != 2:
            raise ValueError("out must be (dH, dW)")
        dH, dW = out
        _check_grad_out("dH", dH, (prob.N, prob.H), grad_dtype, dev)
        _check_grad_out("dW", dW, (prob.V, prob.H), grad_dtype, dev)
    else:
        dH = torch.empty_like(hidden, dtype=grad_dtype) if want[0] else None
        dW = torch.empty_like(W, dtype=grad_dtype) if want[1] else None
    st = _on_device(dev.index, fckl_ce_bwd, prob, hidden.data_ptr(), W.data_ptr(),
                    labels.data_ptr(), lse.data_ptr(), row_grad.data_ptr(), _ptr(dH), _ptr(dW),
                    workspace.data_ptr(), workspace.numel())
    _finish(st, "fckl_ce_bwd", workspace, check)
    return dH, dW


def _scale_gradient(t, factor):
    """t *= factor (a device float32 scalar) in place; free when the factor is 1."""
    if t is None:
        return
    st = _on_device(t.get_device(), fckl_scale_gradient, t.data_ptr(), t.numel(),
                    _GRAD_TYPES[t.dtype], factor.data_ptr())
    if st != FCKL_OK:
        raise FcklError(st, "fckl_scale_gradient")


def _option(name, value):
    """A differentiable call's option as a number: backward sees what forward saw."""
    if isinstance(value, torch.Tensor) and value.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} gets no gradient; detach it")
    return float(value)


class FusedCrossEntropy(torch.autograd.Function):
    """Cross entropy with gradients for hidden and W, in their own dtype (bf16).

    reduction "mean" / "sum": the fused call computes the gradients in forward;
    with grad_dtype bfloat16 the first backward multiplies them by the upstream
    factor (rounded once more unless it is a power of two) and hands them over, and
    later ones (retain_graph) compute them again from the saved log-sum-exps; with
    float32 they are kept and rounded once, after the factor.  reduction "none":
    forward returns the row losses, backward computes the gradients for the given
    upstream gradient."""

    @staticmethod
    def forward(ctx, hidden, W, labels, row_weight, reduction, ignore_index, check, opts,
                grad_dtype=torch.bfloat16, n_valid_total=0):
        want = ctx.needs_input_grad[:2]
        ctx.set_materialize_grads(False)
        ctx.reduction, ctx.ignore_index, ctx.check, ctx.opts = reduction, ignore_index, check, opts
        ctx.want, ctx.grads, ctx.n_valid_total = want, None, n_valid_total
        kw = dict(ignore_index=ignore_index, check=check, **opts)
        ctx.kept = reduction != "none" and any(want) and grad_dtype == torch.float32
        if reduction == "none":
            if row_weight is not None:
                raise ValueError('row_weight needs reduction "mean" or "sum"')
            _, value, lse = fused_ce_fwd(hidden, W, labels, reduction="sum", **kw)
        elif any(want):
            loss, _, lse, dH, dW = _fused_ce_fwd_bwd(
                hidden, W, labels, row_weight, reduction=reduction, workspace=None, out=None,
                grad_dtype=grad_dtype, n_valid_total=n_valid_total, want=want,
                want_lse=not ctx.kept, **kw)
            value = loss[0]
            if ctx.kept:
                ctx.save_for_backward(dH, dW)
                return value
            ctx.grads = (dH, dW)
        else:
            loss, _, lse = fused_ce_fwd(hidden, W, labels, row_weight, reduction=reduction,
                                        n_valid_total=n_valid_total, **kw)
            value = loss[0]
        ctx.save_for_backward(hidden, W, labels, row_weight, lse)
        return value

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        none = (None,) * 8
        if grad_out is None:
            return (None, None) + none
        if ctx.kept:        # the product in float32, rounded as it is stored
            return tuple(t if t is None else torch.mul(t, grad_out, out=torch.empty_like(
                t, dtype=torch.bfloat16)) for t in ctx.saved_tensors) + none
        hidden, W, labels, row_weight, lse = ctx.saved_tensors
        if ctx.grads is not None:
            (dH, dW), ctx.grads = ctx.grads, None
            for t in (dH, dW):
                _scale_gradient(t, grad_out)
            return (dH, dW) + none
        row_grad = grad_out
        if ctx.reduction != "none":
            row_grad = grad_out.expand(labels.shape[0])
            if row_weight is not None:
                row_grad = row_grad * row_weight
            if ctx.reduction == "mean":
                V, count = W.shape[0], ctx.n_valid_total
                if count == 0:
                    kept = (labels != ctx.ignore_index) & (labels >= 0) & (labels < V)
                    count = kept.sum().clamp(min=1)
                row_grad = row_grad / count
        dH, dW = fused_ce_bwd(hidden, W, labels, lse, row_grad.contiguous(),
                              ignore_index=ctx.ignore_index, check=ctx.check,
                              grad_dtype=torch.bfloat16, want=ctx.want, **ctx.opts)
        return (dH, dW) + none


def fused_cross_entropy_loss(hidden, W, labels, row_weight=None, T=1.0, label_smoothing=0.0,
                             z_loss=0.0, ignore_index=-100, reduction="mean", chunk=0, check=True,
                             norm=None, grad_dtype=torch.bfloat16, n_valid_total=0):
    """Differentiable fused_ce_fwd: the loss (a scalar), or with reduction "none"
    the row losses [N].  hidden and W are bfloat16, and so are their gradients;
    ``row_weight`` gets no gradient.  ``check=False`` leaves out the device-error
    check, which synchronises the stream (a step that is captured into a graph needs
    that, and, like every captured backward pass, no eager graph of the same leaves
    alive).  ``norm``: a TailNorm; ``hidden`` is then the residual stream, and the loss
    runs over its normed rows.

    ``n_valid_total``: > 0 replaces the number of rows that a mean divides by, e.g.
    that of all data-parallel ranks' rows: the ranks' losses and gradients then sum
    to those of the whole batch.
    ``grad_dtype``: what the gradients of a mean or sum are held in until backward
    brings their upstream factor (alpha in "alpha * loss + ..."): bfloat16, which
    costs nothing at a factor of 1 and a second rounding at one that is not a power
    of two, or float32, rounded once (twice the memory, one more pass)."""
    if grad_dtype not in _GRAD_TYPES:
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    if row_weight is not None and row_weight.requires_grad:
        raise ValueError("row_weight gets no gradient; detach it")
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f'reduction must be "mean", "sum" or "none", got {reduction!r}')
    if norm is not None:
        hidden = norm(hidden)
    opts = dict(T=_option("T", T), label_smoothing=_option("label_smoothing", label_smoothing),
                z_loss=_option("z_loss", z_loss), chunk=_int(chunk))
    if not torch.is_grad_enabled():  # (inside a Function's forward this cannot be told)
        hidden, W = hidden.detach(), W.detach()
    return FusedCrossEntropy.apply(hidden, W, labels, row_weight, reduction, _int(ignore_index),
                                   check, opts, grad_dtype, _int(n_valid_total))


# ---------------------------------------------------------------- norms around a block
_REAL_TYPES = {torch.float32: FCKL_FLOAT, torch.bfloat16: FCKL_BFLOAT}


def _norm_checks(x, block, post_weight, gate, pre_weight, dy=None, dv=None):
    """Shapes, dtypes and placement of a block_norm call, named one by one."""
    if x.dim() != 2:
        raise ValueError(f"x must be [N,H]; got {tuple(x.shape)}")
    N, H = x.shape
    rows = (("x", x), ("block", block), ("dy", dy), ("dv", dv))
    for name, t in rows:
        if t is not None and tuple(t.shape) != (N, H):
            raise ValueError(f"{name} must be [N={N},H={H}]; got {tuple(t.shape)}")
    if x.dtype not in _REAL_TYPES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if block is not None and block.dtype != torch.bfloat16:
        raise TypeError(f"block must be bfloat16, got {block.dtype}")
    if dv is not None and dv.dtype != x.dtype:
        raise TypeError(f"dv must have x's dtype {x.dtype}, got {dv.dtype}")
    if dy is not None and dy.dtype not in _REAL_TYPES:
        raise TypeError(f"dy must be float32 or bfloat16, got {dy.dtype}")
    weights = [(n, w) for n, w in (("post_weight", post_weight), ("gate", gate),
                                   ("pre_weight", pre_weight)) if w is not None]
    for name, w in weights:
        if tuple(w.shape) != (H,):
            raise ValueError(f"{name} must be [H={H}]; got {tuple(w.shape)}")
        if w.dtype not in _REAL_TYPES or w.dtype != weights[0][1].dtype:
            raise TypeError("post_weight, gate and pre_weight must all be float32 or all bfloat16")
    _check_placement(True, rows + tuple(weights))


def _norm_problem(x, block, post_weight, gate, pre_weight, scale, post, pre, eps, weight_offset,
                  dy=None, dv=None):
    """The fields of a block_norm call's problem, checked.  One quick pass over the tensors;
    only what it does not accept goes through the checks that name the fault."""
    shape, index, wt, ok = x.shape, x.get_device(), None, x.dim() == 2
    if ok:
        row = shape[1:]
        for w in (post_weight, gate, pre_weight):
            if w is not None:
                wt = wt or w.dtype
                ok = ok and w.dtype == wt and w.shape == row
        ok = (ok and x.dtype in _REAL_TYPES and (wt is None or wt in _REAL_TYPES)
              and (block is None or (block.shape == shape and block.dtype == torch.bfloat16))
              and (dy is None or (dy.shape == shape and dy.dtype in _REAL_TYPES))
              and (dv is None or (dv.shape == shape and dv.dtype == x.dtype))
              and _placed(index, (x, block, post_weight, gate, pre_weight, dy, dv)))
    if not ok:
        _norm_checks(x, block, post_weight, gate, pre_weight, dy, dv)
    return (shape[0], shape[1], float(scale), float(eps), float(weight_offset),
            (FCKL_NORM_POST if post else 0) | (FCKL_NORM_PRE if pre else 0),
            _REAL_TYPES[x.dtype], _REAL_TYPES[wt] if wt else FCKL_FLOAT,
            FCKL_BFLOAT if dy is None else _REAL_TYPES[dy.dtype])


def block_norm_fwd(x, block=None, post_weight=None, gate=None, pre_weight=None, scale=1.0,
                   post=None, pre=True, eps=1e-6, weight_offset=0.0, want_residual=True):
    """Joins a block's output to the residual stream and norms the result:
    v = x + scale * gate * (block * rho(block) * post_weight), y = v * rho(v) *
    pre_weight with rho(z) = 1/sqrt(mean(z^2) + eps) over a row.

    x [N,H] float32 or bfloat16, block [N,H] bfloat16 (None: a plain norm of x),
    weights and gate [H] float32 or bfloat16 (None: ones; ``weight_offset`` is
    added to the two norm weights).  ``post`` (default: whether post_weight is
    given) and ``pre``: which norms there are.  Returns (v in x's dtype, y
    bfloat16); v is x itself without a block and None without ``want_residual``;
    y is None without ``pre``."""
    post = post_weight is not None if post is None else bool(post)
    fields = _norm_problem(x, block, post_weight, gate, pre_weight, scale, post, pre, eps,
                           weight_offset)
    dev = x.device
    v = torch.empty_like(x) if block is not None and (want_residual or not pre) else None
    y = torch.empty_like(x, dtype=torch.bfloat16) if pre else None
    st = _on_device(dev.index, fckl_block_norm_fwd, _norm_struct(*fields), x.data_ptr(), _ptr(block),
                    _ptr(post_weight), _ptr(gate), _ptr(pre_weight), _ptr(v), _ptr(y))
    if st != FCKL_OK:
        raise FcklError(st, "fckl_block_norm_fwd")
    return (x if block is None else v), y


def block_norm_bwd(x, block=None, dy=None, dv=None, post_weight=None, gate=None, pre_weight=None,
                   scale=1.0, post=None, pre=True, eps=1e-6, weight_offset=0.0,
                   want=(True, True, True, True, True), workspace=None):
    """Gradients of block_norm_fwd's inputs from dy (float32 or bfloat16, with
    ``pre``) and dv (x's dtype, or None).  Returns (dx, dblock, dpost_weight,
    dgate, dpre_weight), the last three float32; None for what is not there or
    not in ``want``."""
    post = post_weight is not None if post is None else bool(post)
    if pre and dy is None:
        raise ValueError("dy is required with a pre-norm")
    if not pre and (dy is not None or dv is None):
        raise ValueError("without a pre-norm there is dv and no dy")
    fields = _norm_problem(x, block, post_weight, gate, pre_weight, scale, post, pre, eps,
                           weight_offset, dy, dv)
    dev, H = x.device, fields[1]
    if workspace is None:
        nbytes = _norm_workspace_bytes(fields)
        if nbytes == 0:
            raise FcklError(1 if H % 8 == 0 and H <= 8192 else 2,
                            "fckl_block_norm_workspace_bytes")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
          or workspace.device != dev):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    dx = torch.empty_like(x) if want[0] else None
    dblock = torch.empty_like(block) if want[1] and block is not None else None
    # one allocation for the weights' gradients
    want1 = want[2] and post_weight is not None
    wantg = want[3] and gate is not None
    want2 = want[4] and pre_weight is not None
    d1 = dg = d2 = None
    n = want1 + wantg + want2
    if n:
        sums = torch.empty(n, H, dtype=torch.float32, device=dev).unbind()
        if want1:
            d1 = sums[0]
        if wantg:
            dg = sums[1 if want1 else 0]
        if want2:
            d2 = sums[-1]
    elif dx is None and dblock is None:
        return None, None, None, None, None
    st = _on_device(dev.index, fckl_block_norm_bwd, _norm_struct(*fields), x.data_ptr(), _ptr(block),
                    _ptr(post_weight), _ptr(gate), _ptr(pre_weight), _ptr(dy), _ptr(dv), _ptr(dx),
                    _ptr(dblock), _ptr(d1), _ptr(dg), _ptr(d2), workspace.data_ptr(),
                    workspace.numel())
    if st != FCKL_OK:
        raise FcklError(st, "fckl_block_norm_bwd")
    return dx, dblock, d1, dg, d2


class BlockNorm(torch.autograd.Function):
    """(v, y), y alone (no block) or v alone (no pre-norm) of block_norm_fwd, with
    gradients for x, block, the weights and the gate in their own dtypes."""

    @staticmethod
    def forward(ctx, x, block, post_weight, gate, pre_weight, opts):
        ctx.set_materialize_grads(False)
        ctx.opts = opts
        ctx.save_for_backward(x, block, post_weight, gate, pre_weight)
        v, y = block_norm_fwd(x, block, post_weight, gate, pre_weight, **opts)
        ctx.single = block is None or y is None
        return y if block is None else v if y is None else (v, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        x, block, post_weight, gate, pre_weight = ctx.saved_tensors
        opts = dict(ctx.opts)
        if not ctx.single:
            dv, dy = grads
        else:
            dv, dy = (None, grads[0]) if opts["pre"] else (grads[0], None)
        if dv is None and dy is None:
            return (None,) * 6
        if dy is None:              # y took no part in what is differentiated
            opts["pre"] = False
        want = ctx.needs_input_grad[:5]
        if not opts["pre"]:
            want = want[:4] + (False,)
            pre_weight_in = None
        else:
            pre_weight_in = pre_weight
        out = block_norm_bwd(x, block, None if dy is None else dy.contiguous(),
                             None if dv is None else dv.contiguous(), post_weight, gate,
                             pre_weight_in, want=want, **opts)
        weights = (post_weight, gate, pre_weight)
        return out[:2] + tuple(g if g is None else g.to(w.dtype)
                               for g, w in zip(out[2:], weights)) + (None,)


def block_norm(x, block=None, post_weight=None, gate=None, pre_weight=None, scale=1.0, post=None,
               pre=True, eps=1e-6, weight_offset=0.0):
    """Differentiable block_norm_fwd: (v, y)."""
    if block is None and not pre:
        raise ValueError("without a block there must be a pre-norm")
    opts = dict(scale=_option("scale", scale),
                post=post_weight is not None if post is None else bool(post), pre=bool(pre),
                eps=_option("eps", eps), weight_offset=_option("weight_offset", weight_offset))
    out = BlockNorm.apply(x, block, post_weight, gate, pre_weight, opts)
    if block is None:
        return x, out
    return out if pre else (out, None)


@dataclasses.dataclass
class TailNorm:
    """The end of a student between its residual stream and its projection, for
    the losses' ``norm`` option: the last block's output (if any) joins the
    stream and the stream is normed (see block_norm_fwd)."""
    pre_weight: torch.Tensor = None
    block: torch.Tensor = None
    post_weight: torch.Tensor = None
    gate: torch.Tensor = None
    scale: float = 1.0
    post: bool = None
    eps: float = 1e-6
    weight_offset: float = 0.0

    def __call__(self, x):
        return block_norm(x, self.block, self.post_weight, self.gate, self.pre_weight, self.scale,
                          self.post, True, self.eps, self.weight_offset)[1]
