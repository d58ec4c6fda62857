"""Python binding of the matrix product with bias, activation and residual in
its epilogue: argument marshalling only.

16-bit operands, or 8-bit operands with the scales that `norm.rms_norm` writes
(e4m3 "row" and "int8": fp32, one a row; e4m3 "mx": e8m0, one for 32 columns). Formulas, types and
rules: include/mhc_linear.h. All arithmetic runs in the gfx950 kernels; a
missing library raises ImportError.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Mapping, NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._call import address, on, require, stream_handle, workspace_of
from ._lib import check_linear, mhc_linear_launch

_DTYPES = {torch.bfloat16: _lib.MHC_LINEAR_BF16, torch.float16: _lib.MHC_LINEAR_F16}
ACTIVATIONS = {"none": _lib.MHC_ACT_NONE, "relu": _lib.MHC_ACT_RELU, "silu": _lib.MHC_ACT_SILU,
               "gelu": _lib.MHC_ACT_GELU}


class LinearOut(NamedTuple):
    """What `linear` returns; z is None where it was not asked for."""
    out: torch.Tensor
    z: torch.Tensor | None


def _launch_arg(launch):
    if launch is None:
        return None
    if isinstance(launch, mhc_linear_launch):
        return ctypes.pointer(launch)
    if isinstance(launch, Mapping):
        return ctypes.pointer(mhc_linear_launch(**{k: int(v) for k, v in launch.items()}))
    raise TypeError("launch must be None, an mhc_linear_launch or a mapping of its fields")


def _act(activation: str) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)} (got {activation!r})")
    return ACTIVATIONS[activation]


def _operands(x: torch.Tensor, weight: torch.Tensor, x_scales, weight_scales
              ) -> tuple[int, int, int, int, torch.dtype]:
    """(M, N, K, the ABI's dtype, the type of the output) after checking x,
    weight and their scales."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must have shape [M, K]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must have shape [N, K]")
    M, K, N = int(x.shape[0]), int(x.shape[1]), int(weight.shape[0])
    dev = x.device
    if x.dtype in _DTYPES:
        if x_scales is not None or weight_scales is not None:
            raise ValueError("scales need float8_e4m3fn or int8 operands")
        require(x, "x", x.dtype, (M, K), dev)
        require(weight, "weight", x.dtype, (N, K), dev)
        return M, N, K, _DTYPES[x.dtype], x.dtype
    if x.dtype not in (torch.float8_e4m3fn, torch.int8):
        raise TypeError(f"x must be bfloat16, float16, float8_e4m3fn or int8 (got {x.dtype})")
    require(x, "x", x.dtype, (M, K), dev)
    require(weight, "weight", x.dtype, (N, K), dev)
    if not isinstance(x_scales, torch.Tensor) or not isinstance(weight_scales, torch.Tensor):
        raise ValueError("float8_e4m3fn and int8 operands need x_scales and weight_scales")
    if x.dtype == torch.int8 or x_scales.dtype == torch.float32:
        require(x_scales, "x_scales", torch.float32, (M,), dev)
        require(weight_scales, "weight_scales", torch.float32, (N,), dev)
        abi = _lib.MHC_LINEAR_I8_ROW if x.dtype == torch.int8 else _lib.MHC_LINEAR_E4M3_ROW
        return M, N, K, abi, torch.bfloat16
    blocks = -(-K // 32)
    require(x_scales, "x_scales", torch.float8_e8m0fnu, (M, blocks), dev)
    require(weight_scales, "weight_scales", torch.float8_e8m0fnu, (N, blocks), dev)
    return M, N, K, _lib.MHC_LINEAR_E4M3_MX, torch.bfloat16


@functools.lru_cache(maxsize=4096)
def _fwd_workspace(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace bytes of a forward call with the policy's launch (they follow
    from the sizes alone)."""
    return _lib.linear_lib().mhc_linear_fwd_workspace_bytes(M, N, K, dtype, None)


@functools.lru_cache(maxsize=4096)
def _bwd_workspace(M: int, N: int, K: int, dtype: int) -> int:
    return _lib.linear_lib().mhc_linear_bwd_workspace_bytes(M, N, K, dtype)


def mhc_linear_plan(M: int, N: int, K: int, dtype: int, launch=None) -> dict:
    """Host-only: the launch shape a forward call would use."""
    plan = mhc_linear_launch()
    check_linear(_lib.linear_lib().mhc_linear_plan(M, N, K, dtype, _launch_arg(launch),
                                                   ctypes.byref(plan)))
    return plan.as_dict()


def mhc_linear_fwd_workspace_bytes(M: int, N: int, K: int, dtype: int, launch=None) -> int:
    """Workspace bytes a forward call needs (dtype: the ABI's number)."""
    got = _lib.linear_lib().mhc_linear_fwd_workspace_bytes(M, N, K, dtype, _launch_arg(launch))
    if got < 0:
        raise ValueError(f"invalid M={M}, N={N}, K={K}, dtype={dtype} or launch")
    return int(got)


def mhc_linear_bwd_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace bytes a backward call needs (dtype: the ABI's number)."""
    got = _lib.linear_lib().mhc_linear_bwd_workspace_bytes(M, N, K, dtype)
    if got < 0:
        raise ValueError(f"invalid M={M}, N={N}, K={K} or dtype={dtype}")
    return int(got)


def mhc_linear_fwd(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, *,
                   bias: torch.Tensor | None = None, activation: str = "none",
                   residual: torch.Tensor | None = None, x_scales: torch.Tensor | None = None,
                   weight_scales: torch.Tensor | None = None, z: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None, launch=None,
                   start_event: int | None = None, stop_event: int | None = None) -> torch.Tensor:
    """out [M, N] <- act(x [M, K] . weight [N, K]^T + bias [N]) + residual
    [M, N]; z, where given, takes the value before the activation. Without a
    workspace one is allocated. Asynchronous."""
    sizes = _check_fwd_inputs(x, weight, bias, residual, x_scales, weight_scales)
    M, N, _, _, kind = sizes
    require(out, "out", kind, (M, N), x.device)
    if z is not None:
        require(z, "z", kind, (M, N), x.device)
    _launch_fwd(x, weight, out, bias, activation, residual, x_scales, weight_scales, z, sizes,
                workspace, stream, _launch_arg(launch), start_event, stop_event)
    return out


def _check_fwd_inputs(x, weight, bias, residual, x_scales, weight_scales):
    sizes = _operands(x, weight, x_scales, weight_scales)
    M, N, _, _, kind = sizes
    if bias is not None:
        require(bias, "bias", kind, (N,), x.device)
    if residual is not None:
        require(residual, "residual", kind, (M, N), x.device)
    return sizes


def _launch_fwd(x, weight, out, bias, activation, residual, x_scales, weight_scales, z, sizes,
                workspace, stream, launch, start_event, stop_event) -> None:
    M, N, K, dtype, _ = sizes
    act = _act(activation)
    dev = x.device
    lib = _lib.linear_lib()
    need = 0
    if workspace is None:
        need = _fwd_workspace(M, N, K, dtype) if launch is None else \
            lib.mhc_linear_fwd_workspace_bytes(M, N, K, dtype, launch)
    ws, ws_bytes, _owner = workspace_of(workspace, need, dev, stream)
    with on(dev):
        st = lib.mhc_linear_fwd(
            x.data_ptr(), address(x_scales), weight.data_ptr(), address(weight_scales),
            address(bias), address(residual), out.data_ptr(), address(z), ws, ws_bytes, M, N, K,
            dtype, act, stream_handle(dev, stream), launch, start_event, stop_event)
    check_linear(st)


def mhc_linear_bwd(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *,
                   grad_x: torch.Tensor | None = None, grad_weight: torch.Tensor | None = None,
                   grad_bias: torch.Tensor | None = None, activation: str = "none",
                   z: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None, start_event: int | None = None,
                   stop_event: int | None = None) -> None:
    """Writes those of grad_x [M, K], grad_weight [N, K] and grad_bias [N]
    that are given; z as the forward wrote it, unless the activation is
    "none". Without a workspace one is allocated. Asynchronous."""
    M, N, K, dtype, kind = _operands(x, weight, None, None)
    act = _act(activation)
    dev = x.device
    require(grad_out, "grad_out", kind, (M, N), dev)
    if activation != "none":
        require(z, "z", kind, (M, N), dev)
    if grad_x is not None:
        require(grad_x, "grad_x", kind, (M, K), dev)
    if grad_weight is not None:
        require(grad_weight, "grad_weight", kind, (N, K), dev)
    if grad_bias is not None:
        require(grad_bias, "grad_bias", kind, (N,), dev)
    ws, ws_bytes, _owner = workspace_of(
        workspace, _bwd_workspace(M, N, K, dtype) if workspace is None else 0, dev, stream)
    with on(dev):
        st = _lib.linear_lib().mhc_linear_bwd(
            grad_out.data_ptr(), x.data_ptr(), weight.data_ptr(),
            z.data_ptr() if activation != "none" else None, address(grad_x),
            address(grad_weight), address(grad_bias), ws, ws_bytes, M, N, K, dtype, act,
            stream_handle(dev, stream), start_event, stop_event)
    check_linear(st)


# ---------------------------------------------------------------------------
# Allocating conveniences and autograd
# ---------------------------------------------------------------------------

def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *,
           activation: str = "none", residual: torch.Tensor | None = None,
           x_scales: torch.Tensor | None = None, weight_scales: torch.Tensor | None = None,
           return_z: bool = False) -> LinearOut:
    """The product with freshly allocated outputs (no autograd). return_z:
    also the value before the activation, which the backward needs unless
    the activation is "none". The launch is the policy's; where a row's bytes
    must not depend on the batch, `mhc_linear_fwd` takes a launch by name."""
    sizes = _check_fwd_inputs(x, weight, bias, residual, x_scales, weight_scales)
    M, N, _, _, kind = sizes
    out = x.new_empty((M, N), dtype=kind)
    z = torch.empty_like(out) if return_z and activation != "none" else None
    _launch_fwd(x, weight, out, bias, activation, residual, x_scales, weight_scales, z, sizes,
                None, None, None, None, None)
    return LinearOut(out, z)


def linear_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *,
                    activation: str = "none", z: torch.Tensor | None = None, bias: bool = False
                    ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """Backward with freshly allocated gradients: (grad_x, grad_weight,
    grad_bias; the last None unless bias). The residual's gradient is
    grad_out itself."""
    grad_x, grad_weight = torch.empty_like(x), torch.empty_like(weight)
    grad_bias = x.new_empty((weight.shape[0],)) if bias else None
    mhc_linear_bwd(grad_out, x, weight, grad_x=grad_x, grad_weight=grad_weight,
                   grad_bias=grad_bias, activation=activation, z=z)
    return grad_x, grad_weight, grad_bias


class Linear(torch.autograd.Function):
    """Autograd wrapper (16-bit operands): forward and backward both run the
    gfx950 kernels."""

    @staticmethod
    def forward(ctx, x, weight, bias, activation, residual):
        o = linear(x, weight, bias, activation=activation, residual=residual, return_z=True)
        ctx.save_for_backward(x, weight, o.z)
        ctx.activation = activation
        return o.out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, weight, z = ctx.saved_tensors
        need_x, need_w, need_b, _, need_r = ctx.needs_input_grad
        grads = [torch.empty_like(x) if need_x else None,
                 torch.empty_like(weight) if need_w else None,
                 torch.empty((weight.shape[0],), dtype=x.dtype, device=x.device)
                 if need_b else None]
        if any(g is not None for g in grads):
            mhc_linear_bwd(grad_out.contiguous(), x, weight, grad_x=grads[0],
                           grad_weight=grads[1], grad_bias=grads[2], activation=ctx.activation,
                           z=z)
        return (*grads, None, grad_out if need_r else None)


def linear_autograd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *,
                    activation: str = "none", residual: torch.Tensor | None = None
                    ) -> torch.Tensor:
    """act(x weight^T + bias) + residual with gradients for all four."""
    return Linear.apply(x, weight, bias, activation, residual)
