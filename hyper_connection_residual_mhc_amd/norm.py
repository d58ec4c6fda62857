"""Python binding of the root-mean-square norm: argument marshalling only.

One pass over a row adds the residual or collapses the residual streams (the
bits of `ops.h_aggregate`), norms it, and writes it in the input's type or in
8 bits (e4m3 or integers) with scales that `linear.linear` takes. Formulas, types and
rules: include/mhc_rms_norm.h. All arithmetic runs in the gfx950 kernels; a
missing library raises ImportError.
"""

from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._call import address, on, require, stream_handle, workspace_of
from ._lib import check_norm

_DTYPES = {torch.float32: _lib.MHC_NORM_F32, torch.bfloat16: _lib.MHC_NORM_BF16,
           torch.float16: _lib.MHC_NORM_F16}
_FORMATS = {None: _lib.MHC_NORM_SAME, "row": _lib.MHC_NORM_E4M3_ROW, "mx": _lib.MHC_NORM_E4M3_MX,
            "int8": _lib.MHC_NORM_I8_ROW}
_CODES = {"row": torch.float8_e4m3fn, "mx": torch.float8_e4m3fn, "int8": torch.int8}
SUPPORTED_HC = (2, 4, 8)


class RMSNormOut(NamedTuple):
    """What `rms_norm` returns; a field that was not asked for is None."""
    y: torch.Tensor                 # [T, H] in x's type, or float8_e4m3fn, or int8
    scales: torch.Tensor | None     # "row", "int8": [T] fp32; "mx": [T, ceil(H / 32)] float8_e8m0fnu
    stored: torch.Tensor | None     # [T, H]: x + residual, or the collapsed streams
    rstd: torch.Tensor | None       # [T] fp32


def _shapes(x: torch.Tensor, pre) -> tuple[int, int, int]:
    want = 2 if pre is None else 3
    if not isinstance(x, torch.Tensor) or x.dim() != want:
        raise ValueError("x must have shape [T, H], or [T, n, H] with pre")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x must be float32, bfloat16 or float16 (got {x.dtype})")
    if pre is None:
        return int(x.shape[0]), 0, int(x.shape[1])
    if x.shape[1] not in SUPPORTED_HC:
        raise ValueError("streams must have shape [T, n, H] with n in {2, 4, 8}")
    return int(x.shape[0]), int(x.shape[1]), int(x.shape[2])


def _check_inputs(x, weight, residual, pre, quant) -> tuple[int, int, int]:
    """(T, n, H) of a forward call whose inputs are sound."""
    T, n, H = _shapes(x, pre)
    if quant not in _FORMATS:
        raise ValueError(f'quant must be None, "row", "mx" or "int8" (got {quant!r})')
    dev, dt = x.device, x.dtype
    require(x, "x", dt, (T, n, H) if n else (T, H), dev)
    _check_weight(weight, dt, H, dev)
    if residual is not None:
        require(residual, "residual", dt, (T, H), dev)
    if pre is not None:
        require(pre, "pre", torch.float32, (T, n), dev)
    return T, n, H


def _check_weight(weight, dtype: torch.dtype, H: int, device: torch.device) -> None:
    fp32 = isinstance(weight, torch.Tensor) and weight.dtype is torch.float32
    require(weight, "weight", torch.float32 if fp32 else dtype, (H,), device)


def _launch_fwd(x, weight, out, eps, residual, pre, scales, stored, rstd, quant, T, n, H, stream,
                start_event, stop_event) -> None:
    dev = x.device
    with on(dev):
        st = _lib.norm_lib().mhc_rms_norm_fwd(
            x.data_ptr(), address(residual), address(pre), n, weight.data_ptr(),
            _DTYPES[weight.dtype], float(eps), out.data_ptr(), address(scales), address(stored),
            address(rstd), T, H, _DTYPES[x.dtype], _FORMATS[quant], stream_handle(dev, stream),
            start_event, stop_event)
    check_norm(st)


def mhc_rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, *,
                     eps: float = 1e-6, residual: torch.Tensor | None = None,
                     pre: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                     stored: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                     quant: str | None = None, stream: torch.cuda.Stream | None = None,
                     start_event: int | None = None, stop_event: int | None = None
                     ) -> torch.Tensor:
    """out <- norm of x [T, H], of x + residual, or of streams x [T, n, H]
    collapsed with pre [T, n]; writes scales, stored and rstd where given.
    quant: None, "row", "mx" or "int8". Asynchronous."""
    T, n, H = _check_inputs(x, weight, residual, pre, quant)
    dev, dt = x.device, x.dtype
    require(out, "out", dt if quant is None else _CODES[quant], (T, H), dev)
    if stored is not None:
        require(stored, "stored", dt, (T, H), dev)
    if rstd is not None:
        require(rstd, "rstd", torch.float32, (T,), dev)
    if quant in ("row", "int8"):
        require(scales, "scales", torch.float32, (T,), dev)
    elif quant == "mx":
        require(scales, "scales", torch.float8_e8m0fnu, (T, -(-H // 32)), dev)
    elif scales is not None:
        raise ValueError("scales need quant")
    _launch_fwd(x, weight, out, eps, residual, pre, scales, stored, rstd, quant, T, n, H, stream,
                start_event, stop_event)
    return out


def mhc_rms_norm_bwd_workspace_bytes(T: int, H: int) -> int:
    """Workspace bytes a backward call of T rows of H elements needs."""
    got = _lib.norm_lib().mhc_rms_norm_bwd_workspace_bytes(int(T), int(H))
    if got < 0:
        raise ValueError(f"invalid T={T} or H={H}")
    return int(got)


def mhc_rms_norm_bwd(grad_y: torch.Tensor, stored: torch.Tensor, weight: torch.Tensor,
                     rstd: torch.Tensor, grad_x: torch.Tensor, grad_weight: torch.Tensor, *,
                     grad_stored: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None, start_event: int | None = None,
                     stop_event: int | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(grad_x [T, H], grad_weight [H] fp32) <- backward of the norm of the
    rows `stored`; grad_stored is added to grad_x where given. Without a
    workspace one is allocated. Asynchronous."""
    T, H = _check_bwd_inputs(grad_y, stored, weight, rstd, grad_stored)
    dev = stored.device
    require(grad_x, "grad_x", stored.dtype, (T, H), dev)
    require(grad_weight, "grad_weight", torch.float32, (H,), dev)
    _launch_bwd(grad_y, stored, weight, rstd, grad_stored, grad_x, grad_weight, workspace, T, H,
                stream, start_event, stop_event)
    return grad_x, grad_weight


def _check_bwd_inputs(grad_y, stored, weight, rstd, grad_stored) -> tuple[int, int]:
    T, _, H = _shapes(stored, None)
    dev, dt = stored.device, stored.dtype
    require(stored, "stored", dt, (T, H), dev)
    require(grad_y, "grad_y", dt, (T, H), dev)
    _check_weight(weight, dt, H, dev)
    require(rstd, "rstd", torch.float32, (T,), dev)
    if grad_stored is not None:
        require(grad_stored, "grad_stored", dt, (T, H), dev)
    return T, H


def _launch_bwd(grad_y, stored, weight, rstd, grad_stored, grad_x, grad_weight, workspace, T, H,
                stream, start_event, stop_event) -> None:
    dev = stored.device
    lib = _lib.norm_lib()
    need = lib.mhc_rms_norm_bwd_workspace_bytes(T, H) if workspace is None else 0
    ws, ws_bytes, _owner = workspace_of(workspace, need, dev, stream)
    with on(dev):
        st = lib.mhc_rms_norm_bwd(
            grad_y.data_ptr(), stored.data_ptr(), weight.data_ptr(), _DTYPES[weight.dtype],
            rstd.data_ptr(), address(grad_stored), grad_x.data_ptr(), grad_weight.data_ptr(), ws,
            ws_bytes, T, H, _DTYPES[stored.dtype], stream_handle(dev, stream), start_event,
            stop_event)
    check_norm(st)


# ---------------------------------------------------------------------------
# Allocating conveniences and autograd
# ---------------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
             residual: torch.Tensor | None = None, pre: torch.Tensor | None = None,
             quant: str | None = None, return_rstd: bool = False) -> RMSNormOut:
    """The norm with freshly allocated outputs (no autograd); `stored` is
    returned with a residual or pre."""
    T, n, H = _check_inputs(x, weight, residual, pre, quant)
    scales = stored = rstd = None
    if quant is None:
        y = x.new_empty((T, H)) if n else torch.empty_like(x)
    else:
        y = x.new_empty((T, H), dtype=_CODES[quant])
        if quant != "mx":
            scales = x.new_empty((T,), dtype=torch.float32)
        else:
            scales = x.new_empty((T, -(-H // 32)), dtype=torch.float8_e8m0fnu)
    if n or residual is not None:
        stored = x.new_empty((T, H)) if n else torch.empty_like(x)
    if return_rstd:
        rstd = x.new_empty((T,), dtype=torch.float32)
    _launch_fwd(x, weight, y, eps, residual, pre, scales, stored, rstd, quant, T, n, H, None, None,
                None)
    return RMSNormOut(y, scales, stored, rstd)


def rms_norm_backward(grad_y: torch.Tensor, stored: torch.Tensor, weight: torch.Tensor,
                      rstd: torch.Tensor, *, grad_stored: torch.Tensor | None = None
                      ) -> tuple[torch.Tensor, torch.Tensor]:
    """Backward with freshly allocated gradients: (grad_x in stored's type,
    grad_weight in fp32)."""
    T, H = _check_bwd_inputs(grad_y, stored, weight, rstd, grad_stored)
    grad_x = torch.empty_like(stored)
    grad_weight = stored.new_empty((H,), dtype=torch.float32)
    _launch_bwd(grad_y, stored, weight, rstd, grad_stored, grad_x, grad_weight, None, T, H, None,
                None, None)
    return grad_x, grad_weight


class RMSNorm(torch.autograd.Function):
    """Autograd wrapper: (y, stored) of x, of x + residual, or of streams x
    with pre, whose gradients run through h_aggregate's backward. stored is x
    itself where neither is given."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual, pre):
        o = rms_norm(x, weight, eps, residual=residual, pre=pre, return_rstd=True)
        stored = x if o.stored is None else o.stored
        ctx.save_for_backward(stored, weight, o.rstd, *((x, pre) if pre is not None else ()))
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        if o.stored is None:
            return o.y, None
        return o.y, o.stored

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_stored):
        stored, weight, rstd, *streams = ctx.saved_tensors
        if grad_y is None:
            grad_x, grad_weight = grad_stored, None
        else:
            if grad_stored is not None:
                grad_stored = grad_stored.contiguous()
            grad_x, grad_weight = rms_norm_backward(grad_y.contiguous(), stored, weight, rstd,
                                                    grad_stored=grad_stored)
            grad_weight = grad_weight.to(weight.dtype)
        grad_pre = None
        grad_residual = grad_x if ctx.has_residual else None
        if streams and grad_x is not None:
            from .ops import h_aggregate_backward
            grad_x, grad_pre = h_aggregate_backward(streams[0], streams[1], grad_x.contiguous())
        return grad_x, grad_weight, None, grad_residual, grad_pre


def rms_norm_autograd(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                      residual: torch.Tensor | None = None, pre: torch.Tensor | None = None
                      ) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(y, stored) with gradients for x, weight, residual and pre; stored is
    None where neither a residual nor pre is given (the row is x itself)."""
    return RMSNorm.apply(x, weight, eps, residual, pre)
