"""Python binding of the cross entropy of a large vocabulary: argument
marshalling only.

The logits x W^T of the last norm's rows are made in tiles and never stored;
what comes out is the loss, each row's logarithm of the sum of exponentials,
and the gradients of x and W. Formulas, types and rules:
include/mhc_cross_entropy.h. All arithmetic runs in the gfx950 kernels; a
missing library raises ImportError.
"""

from __future__ import annotations

import functools
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._call import address, on, require, stream_handle, workspace_of
from ._lib import check_cross_entropy
from .linear import _launch_arg

_DTYPES = {torch.bfloat16: _lib.MHC_LINEAR_BF16, torch.float16: _lib.MHC_LINEAR_F16}
REDUCTIONS = {"none": _lib.MHC_REDUCTION_NONE, "sum": _lib.MHC_REDUCTION_SUM,
              "mean": _lib.MHC_REDUCTION_MEAN}
IGNORE_INDEX = -100


class LossOut(NamedTuple):
    """What `linear_cross_entropy` returns."""
    loss: torch.Tensor  # fp32, [M] ("none") or a scalar
    lse: torch.Tensor   # [M] fp32


class LossGrads(NamedTuple):
    """What `linear_cross_entropy_grads` returns."""
    loss: torch.Tensor         # fp32, [M] ("none") or a scalar
    lse: torch.Tensor          # [M] fp32
    grad_x: torch.Tensor       # [M, K] in x's type
    grad_weight: torch.Tensor  # [V, K] in x's type


def _inputs(x, weight, targets, reduction) -> tuple[int, int, int, int, int]:
    """(M, V, K, the ABI's dtype and reduction) after checking the inputs."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must have shape [M, K]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must have shape [V, K]")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x must be bfloat16 or float16 (got {x.dtype})")
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)} (got {reduction!r})")
    M, K, V = int(x.shape[0]), int(x.shape[1]), int(weight.shape[0])
    require(x, "x", x.dtype, (M, K), x.device)
    require(weight, "weight", x.dtype, (V, K), x.device)
    require(targets, "targets", torch.int64, (M,), x.device)
    return M, V, K, _DTYPES[x.dtype], REDUCTIONS[reduction]


def _loss_shape(M: int, reduction: int) -> tuple:
    return (M,) if reduction == _lib.MHC_REDUCTION_NONE else ()


def _rows(t, name, shape, device):
    if t is not None:
        require(t, name, torch.float32, shape, device)


@functools.lru_cache(maxsize=4096)
def _workspace(call: str, M: int, V: int, K: int, dtype: int) -> int:
    """Workspace bytes of a call with the policy's launch (they follow from the
    sizes alone)."""
    return getattr(_lib.cross_entropy_lib(), f"mhc_cross_entropy_{call}_workspace_bytes")(
        M, V, K, dtype, None)


def mhc_cross_entropy_workspace_bytes(call: str, M: int, V: int, K: int, dtype: int,
                                      launch=None) -> int:
    """Workspace bytes that "fwd", "bwd" or "grads" needs (dtype: the ABI's
    number)."""
    if call not in ("fwd", "bwd", "grads"):
        raise ValueError(f'call must be "fwd", "bwd" or "grads" (got {call!r})')
    got = getattr(_lib.cross_entropy_lib(), f"mhc_cross_entropy_{call}_workspace_bytes")(
        M, V, K, dtype, _launch_arg(launch))
    if got < 0:
        raise ValueError(f"invalid M={M}, V={V}, K={K}, dtype={dtype} or launch")
    return int(got)


def _space(call, sizes, launch, workspace, device, stream):
    need = 0
    if workspace is None:
        need = _workspace(call, *sizes) if launch is None else \
            mhc_cross_entropy_workspace_bytes(call, *sizes, launch)
    return workspace_of(workspace, need, device, stream)


def mhc_cross_entropy_fwd(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                          loss: torch.Tensor, lse: torch.Tensor, *,
                          ignore_index: int = IGNORE_INDEX, reduction: str = "mean",
                          workspace: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None, launch=None,
                          start_event: int | None = None, stop_event: int | None = None
                          ) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse [M]) <- cross entropy of x [M, K] . weight [V, K]^T against
    targets [M]; loss is [M] ("none") or a scalar. Without a workspace one is
    allocated. Asynchronous."""
    M, V, K, dtype, how = _inputs(x, weight, targets, reduction)
    dev = x.device
    require(loss, "loss", torch.float32, _loss_shape(M, how), dev)
    require(lse, "lse", torch.float32, (M,), dev)
    ws, ws_bytes, _owner = _space("fwd", (M, V, K, dtype), launch, workspace, dev, stream)
    with on(dev):
        st = _lib.cross_entropy_lib().mhc_cross_entropy_fwd(
            x.data_ptr(), weight.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(),
            ws, ws_bytes, M, V, K, dtype, how, int(ignore_index), stream_handle(dev, stream),
            _launch_arg(launch), start_event, stop_event)
    check_cross_entropy(st)
    return loss, lse


def mhc_cross_entropy_bwd(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                          lse: torch.Tensor, grad_loss: torch.Tensor | None = None, *,
                          grad_lse: torch.Tensor | None = None,
                          grad_x: torch.Tensor | None = None,
                          grad_weight: torch.Tensor | None = None,
                          ignore_index: int = IGNORE_INDEX, reduction: str = "mean",
                          workspace: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None, launch=None,
                          start_event: int | None = None, stop_event: int | None = None) -> None:
    """Writes those of grad_x [M, K] and grad_weight [V, K] that are given, from
    the forward's lse and the gradients of loss (None stands for 1) and lse; the
    logits are made again. Without a workspace one is allocated.
    Asynchronous."""
    M, V, K, dtype, how = _inputs(x, weight, targets, reduction)
    dev = x.device
    require(lse, "lse", torch.float32, (M,), dev)
    _rows(grad_loss, "grad_loss", _loss_shape(M, how), dev)
    _rows(grad_lse, "grad_lse", (M,), dev)
    if grad_x is not None:
        require(grad_x, "grad_x", x.dtype, (M, K), dev)
    if grad_weight is not None:
        require(grad_weight, "grad_weight", x.dtype, (V, K), dev)
    ws, ws_bytes, _owner = _space("bwd", (M, V, K, dtype), launch, workspace, dev, stream)
    with on(dev):
        st = _lib.cross_entropy_lib().mhc_cross_entropy_bwd(
            x.data_ptr(), weight.data_ptr(), targets.data_ptr(), lse.data_ptr(),
            address(grad_loss), address(grad_lse), address(grad_x), address(grad_weight), ws,
            ws_bytes, M, V, K, dtype, how, int(ignore_index), stream_handle(dev, stream),
            _launch_arg(launch), start_event, stop_event)
    check_cross_entropy(st)


def mhc_cross_entropy_grads(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                            loss: torch.Tensor, lse: torch.Tensor,
                            grad_loss: torch.Tensor | None = None, *,
                            grad_x: torch.Tensor | None = None,
                            grad_weight: torch.Tensor | None = None,
                            ignore_index: int = IGNORE_INDEX, reduction: str = "mean",
                            workspace: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None, launch=None,
                            start_event: int | None = None, stop_event: int | None = None) -> None:
    """Writes loss and lse [M], and those of grad_x [M, K] and grad_weight
    [V, K] that are given, for a gradient of the loss that is known beforehand
    (None stands for 1). Without a workspace one is allocated. Asynchronous."""
    M, V, K, dtype, how = _inputs(x, weight, targets, reduction)
    dev = x.device
    require(loss, "loss", torch.float32, _loss_shape(M, how), dev)
    require(lse, "lse", torch.float32, (M,), dev)
    _rows(grad_loss, "grad_loss", _loss_shape(M, how), dev)
    if grad_x is not None:
        require(grad_x, "grad_x", x.dtype, (M, K), dev)
    if grad_weight is not None:
        require(grad_weight, "grad_weight", x.dtype, (V, K), dev)
    ws, ws_bytes, _owner = _space("grads", (M, V, K, dtype), launch, workspace, dev, stream)
    with on(dev):
        st = _lib.cross_entropy_lib().mhc_cross_entropy_grads(
            x.data_ptr(), weight.data_ptr(), targets.data_ptr(), address(grad_loss),
            loss.data_ptr(), lse.data_ptr(), address(grad_x), address(grad_weight), ws, ws_bytes,
            M, V, K, dtype, how, int(ignore_index), stream_handle(dev, stream),
            _launch_arg(launch), start_event, stop_event)
    check_cross_entropy(st)


# ---------------------------------------------------------------------------
# Allocating conveniences and autograd
# ---------------------------------------------------------------------------

def _new(x, targets, reduction):
    shape = tuple(targets.shape) if reduction == "none" else ()
    return (x.new_empty(shape, dtype=torch.float32),
            x.new_empty((x.shape[0],), dtype=torch.float32))


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                         ignore_index: int = IGNORE_INDEX, reduction: str = "mean") -> LossOut:
    """The loss with freshly allocated outputs (no autograd)."""
    _inputs(x, weight, targets, reduction)
    loss, lse = _new(x, targets, reduction)
    mhc_cross_entropy_fwd(x, weight, targets, loss, lse, ignore_index=ignore_index,
                          reduction=reduction)
    return LossOut(loss, lse)


def linear_cross_entropy_backward(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                                  lse: torch.Tensor, grad_loss: torch.Tensor | None = None, *,
                                  grad_lse: torch.Tensor | None = None,
                                  ignore_index: int = IGNORE_INDEX, reduction: str = "mean"
                                  ) -> tuple[torch.Tensor, torch.Tensor]:
    """Backward with freshly allocated gradients: (grad_x, grad_weight)."""
    grad_x, grad_weight = torch.empty_like(x), torch.empty_like(weight)
    mhc_cross_entropy_bwd(x, weight, targets, lse, grad_loss, grad_lse=grad_lse, grad_x=grad_x,
                          grad_weight=grad_weight, ignore_index=ignore_index, reduction=reduction)
    return grad_x, grad_weight


def linear_cross_entropy_grads(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                               grad_loss: torch.Tensor | None = None, *,
                               ignore_index: int = IGNORE_INDEX, reduction: str = "mean"
                               ) -> LossGrads:
    """The loss and its gradients in one call, with freshly allocated outputs:
    for a gradient of the loss that is known beforehand (None stands for 1; of
    "none" a weight for each row). The logits are made once, where
    `linear_cross_entropy` and its backward make them twice."""
    _inputs(x, weight, targets, reduction)
    loss, lse = _new(x, targets, reduction)
    grad_x, grad_weight = torch.empty_like(x), torch.empty_like(weight)
    mhc_cross_entropy_grads(x, weight, targets, loss, lse, grad_loss, grad_x=grad_x,
                            grad_weight=grad_weight, ignore_index=ignore_index,
                            reduction=reduction)
    return LossGrads(loss, lse, grad_x, grad_weight)


class LinearCrossEntropy(torch.autograd.Function):
    """Autograd wrapper: (loss, lse); forward and backward both run the gfx950
    kernels."""

    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, reduction):
        o = linear_cross_entropy(x, weight, targets, ignore_index=ignore_index,
                                 reduction=reduction)
        ctx.save_for_backward(x, weight, targets, o.lse)
        ctx.how = dict(ignore_index=ignore_index, reduction=reduction)
        ctx.set_materialize_grads(False)
        return o.loss, o.lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, grad_lse):
        x, weight, targets, lse = ctx.saved_tensors
        need_x, need_w, *_ = ctx.needs_input_grad
        grad_x = torch.empty_like(x) if need_x else None
        grad_weight = torch.empty_like(weight) if need_w else None
        if grad_loss is None and grad_lse is None:
            return None, None, None, None, None
        if grad_loss is None:
            grad_loss = lse.new_zeros(lse.shape if ctx.how["reduction"] == "none" else ())
        if need_x or need_w:
            mhc_cross_entropy_bwd(x, weight, targets, lse, grad_loss.contiguous(),
                                  grad_lse=None if grad_lse is None else grad_lse.contiguous(),
                                  grad_x=grad_x, grad_weight=grad_weight, **ctx.how)
        return grad_x, grad_weight, None, None, None


def linear_cross_entropy_autograd(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                                  *, ignore_index: int = IGNORE_INDEX, reduction: str = "mean"
                                  ) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) with gradients of both for x and weight."""
    return LinearCrossEntropy.apply(x, weight, targets, ignore_index, reduction)
