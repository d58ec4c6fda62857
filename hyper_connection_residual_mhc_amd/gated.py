"""Python binding of the gated feed-forward block: argument marshalling only.

Both projections of a row, the activation of one and the product of the two in
one kernel, act(x Wg^T + gate_bias) * (x Wu^T + up_bias), for 16-bit operands or
for 8-bit ones with the scales that `norm.rms_norm` writes; the block's last
projection is `linear.linear`. Formulas, types and rules: include/mhc_gated.h.
All arithmetic runs in the gfx950 kernels; a missing library raises
ImportError.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._call import address, on, require, stream_handle, workspace_of
from ._lib import check_gated, mhc_linear_launch
from .linear import _act, _launch_arg, _operands


class GatedOut(NamedTuple):
    """What `gated` returns; gate and up are None where they were not asked for."""
    out: torch.Tensor
    gate: torch.Tensor | None
    up: torch.Tensor | None


def _check_operands(x, gate_weight, up_weight, x_scales, gate_scales, up_scales):
    """(M, N, K, the ABI's dtype, the type of the output)."""
    sizes = _operands(x, gate_weight, x_scales, gate_scales)
    _, N, K, _, _ = sizes
    dev = x.device
    require(up_weight, "up_weight", x.dtype, (N, K), dev)
    if gate_scales is not None:
        require(up_scales, "up_scales", gate_scales.dtype, tuple(gate_scales.shape), dev)
    elif up_scales is not None:
        raise ValueError("scales need float8_e4m3fn or int8 operands")
    return sizes


def _check_fwd_inputs(x, gate_weight, up_weight, gate_bias, up_bias, x_scales, gate_scales,
                      up_scales):
    sizes = _check_operands(x, gate_weight, up_weight, x_scales, gate_scales, up_scales)
    _, N, _, _, kind = sizes
    if gate_bias is not None:
        require(gate_bias, "gate_bias", kind, (N,), x.device)
    if up_bias is not None:
        require(up_bias, "up_bias", kind, (N,), x.device)
    return sizes


@functools.lru_cache(maxsize=4096)
def _fwd_workspace(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace bytes of a forward call with the policy's launch (they follow
    from the sizes alone)."""
    return _lib.gated_lib().mhc_gated_fwd_workspace_bytes(M, N, K, dtype, None)


@functools.lru_cache(maxsize=4096)
def _bwd_workspace(M: int, N: int, K: int, dtype: int) -> int:
    return _lib.gated_lib().mhc_gated_bwd_workspace_bytes(M, N, K, dtype)


def mhc_gated_plan(M: int, N: int, K: int, dtype: int, launch=None) -> dict:
    """Host-only: the launch shape a forward call would use."""
    plan = mhc_linear_launch()
    check_gated(_lib.gated_lib().mhc_gated_plan(M, N, K, dtype, _launch_arg(launch),
                                                ctypes.byref(plan)))
    return plan.as_dict()


def mhc_gated_fwd_workspace_bytes(M: int, N: int, K: int, dtype: int, launch=None) -> int:
    """Workspace bytes a forward call needs (dtype: the ABI's number)."""
    got = _lib.gated_lib().mhc_gated_fwd_workspace_bytes(M, N, K, dtype, _launch_arg(launch))
    if got < 0:
        raise ValueError(f"invalid M={M}, N={N}, K={K}, dtype={dtype} or launch")
    return int(got)


def mhc_gated_bwd_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace bytes a backward call needs (dtype: the ABI's number)."""
    got = _lib.gated_lib().mhc_gated_bwd_workspace_bytes(M, N, K, dtype)
    if got < 0:
        raise ValueError(f"invalid M={M}, N={N}, K={K} or dtype={dtype}")
    return int(got)


def mhc_gated_fwd(x: torch.Tensor, gate_weight: torch.Tensor, up_weight: torch.Tensor,
                  out: torch.Tensor, *, gate_bias: torch.Tensor | None = None,
                  up_bias: torch.Tensor | None = None, activation: str = "silu",
                  x_scales: torch.Tensor | None = None, gate_scales: torch.Tensor | None = None,
                  up_scales: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  up: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None, launch=None,
                  start_event: int | None = None, stop_event: int | None = None) -> torch.Tensor:
    """out [M, N] <- act(x [M, K] . gate_weight [N, K]^T + gate_bias [N]) *
    (x . up_weight [N, K]^T + up_bias [N]); gate and up, where given, take the
    two values before the activation and the product. Without a workspace one
    is allocated. Asynchronous."""
    sizes = _check_fwd_inputs(x, gate_weight, up_weight, gate_bias, up_bias, x_scales,
                              gate_scales, up_scales)
    M, N, _, _, kind = sizes
    for name, t in (("out", out), ("gate", gate), ("up", up)):
        if t is not None or name == "out":
            require(t, name, kind, (M, N), x.device)
    _launch_fwd(x, gate_weight, up_weight, out, gate_bias, up_bias, activation, x_scales,
                gate_scales, up_scales, gate, up, sizes, workspace, stream, _launch_arg(launch),
                start_event, stop_event)
    return out


def _launch_fwd(x, gate_weight, up_weight, out, gate_bias, up_bias, activation, x_scales,
                gate_scales, up_scales, gate, up, sizes, workspace, stream, launch, start_event,
                stop_event) -> None:
    M, N, K, dtype, _ = sizes
    act = _act(activation)
    dev = x.device
    lib = _lib.gated_lib()
    need = 0
    if workspace is None:
        need = _fwd_workspace(M, N, K, dtype) if launch is None else \
            lib.mhc_gated_fwd_workspace_bytes(M, N, K, dtype, launch)
    ws, ws_bytes, _owner = workspace_of(workspace, need, dev, stream)
    with on(dev):
        st = lib.mhc_gated_fwd(
            x.data_ptr(), address(x_scales), gate_weight.data_ptr(), address(gate_scales),
            up_weight.data_ptr(), address(up_scales), address(gate_bias), address(up_bias),
            out.data_ptr(), address(gate), address(up), ws, ws_bytes, M, N, K, dtype, act,
            stream_handle(dev, stream), launch, start_event, stop_event)
    check_gated(st)


def mhc_gated_bwd(grad_out: torch.Tensor, x: torch.Tensor, gate_weight: torch.Tensor,
                  up_weight: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, *,
                  grad_x: torch.Tensor | None = None,
                  grad_gate_weight: torch.Tensor | None = None,
                  grad_up_weight: torch.Tensor | None = None,
                  grad_gate_bias: torch.Tensor | None = None,
                  grad_up_bias: torch.Tensor | None = None, activation: str = "silu",
                  workspace: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None, start_event: int | None = None,
                  stop_event: int | None = None) -> None:
    """Writes those of grad_x [M, K], grad_gate_weight and grad_up_weight [N, K]
    (both or neither), grad_gate_bias and grad_up_bias [N] that are given; gate
    and up as the forward wrote them. Without a workspace one is allocated.
    Asynchronous."""
    M, N, K, dtype, kind = _check_operands(x, gate_weight, up_weight, None, None, None)
    act = _act(activation)
    dev = x.device
    for name, t in (("grad_out", grad_out), ("gate", gate), ("up", up)):
        require(t, name, kind, (M, N), dev)
    for name, t, shape in (("grad_x", grad_x, (M, K)), ("grad_gate_weight", grad_gate_weight, (N, K)),
                           ("grad_up_weight", grad_up_weight, (N, K)),
                           ("grad_gate_bias", grad_gate_bias, (N,)),
                           ("grad_up_bias", grad_up_bias, (N,))):
        if t is not None:
            require(t, name, kind, shape, dev)
    ws, ws_bytes, _owner = workspace_of(
        workspace, _bwd_workspace(M, N, K, dtype) if workspace is None else 0, dev, stream)
    with on(dev):
        st = _lib.gated_lib().mhc_gated_bwd(
            grad_out.data_ptr(), x.data_ptr(), gate_weight.data_ptr(), up_weight.data_ptr(),
            gate.data_ptr(), up.data_ptr(), address(grad_x), address(grad_gate_weight),
            address(grad_up_weight), address(grad_gate_bias), address(grad_up_bias), ws, ws_bytes,
            M, N, K, dtype, act, stream_handle(dev, stream), start_event, stop_event)
    check_gated(st)


# ---------------------------------------------------------------------------
# Allocating conveniences and autograd
# ---------------------------------------------------------------------------

def gated(x: torch.Tensor, gate_weight: torch.Tensor, up_weight: torch.Tensor,
          gate_bias: torch.Tensor | None = None, up_bias: torch.Tensor | None = None, *,
          activation: str = "silu", x_scales: torch.Tensor | None = None,
          gate_scales: torch.Tensor | None = None, up_scales: torch.Tensor | None = None,
          return_z: bool = False) -> GatedOut:
    """The block's first half with freshly allocated outputs (no autograd).
    return_z: also gate and up, which the backward needs."""
    sizes = _check_fwd_inputs(x, gate_weight, up_weight, gate_bias, up_bias, x_scales,
                              gate_scales, up_scales)
    M, N, _, _, kind = sizes
    out = x.new_empty((M, N), dtype=kind)
    gate = torch.empty_like(out) if return_z else None
    up = torch.empty_like(out) if return_z else None
    _launch_fwd(x, gate_weight, up_weight, out, gate_bias, up_bias, activation, x_scales,
                gate_scales, up_scales, gate, up, sizes, None, None, None, None, None)
    return GatedOut(out, gate, up)


def gated_backward(grad_out: torch.Tensor, x: torch.Tensor, gate_weight: torch.Tensor,
                   up_weight: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, *,
                   activation: str = "silu", bias: bool = False
                   ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor | None,
                              torch.Tensor | None]:
    """Backward with freshly allocated gradients: (grad_x, grad_gate_weight,
    grad_up_weight, grad_gate_bias, grad_up_bias; the last two None unless
    bias)."""
    grad_x, grad_g, grad_u = (torch.empty_like(t) for t in (x, gate_weight, up_weight))
    grad_gb = x.new_empty((gate_weight.shape[0],)) if bias else None
    grad_ub = x.new_empty((gate_weight.shape[0],)) if bias else None
    mhc_gated_bwd(grad_out, x, gate_weight, up_weight, gate, up, grad_x=grad_x,
                  grad_gate_weight=grad_g, grad_up_weight=grad_u, grad_gate_bias=grad_gb,
                  grad_up_bias=grad_ub, activation=activation)
    return grad_x, grad_g, grad_u, grad_gb, grad_ub


class Gated(torch.autograd.Function):
    """Autograd wrapper (16-bit operands): forward and backward both run the
    gfx950 kernels."""

    @staticmethod
    def forward(ctx, x, gate_weight, up_weight, gate_bias, up_bias, activation):
        o = gated(x, gate_weight, up_weight, gate_bias, up_bias, activation=activation,
                  return_z=True)
        ctx.save_for_backward(x, gate_weight, up_weight, o.gate, o.up)
        ctx.activation = activation
        return o.out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, gate_weight, up_weight, gate, up = ctx.saved_tensors
        need_x, need_g, need_u, need_gb, need_ub, _ = ctx.needs_input_grad
        N = gate_weight.shape[0]
        grad_x = torch.empty_like(x) if need_x else None
        # the weights' gradients come from one launch
        weights = need_g or need_u
        grad_g = torch.empty_like(gate_weight) if weights else None
        grad_u = torch.empty_like(up_weight) if weights else None
        grad_gb = x.new_empty((N,)) if need_gb else None
        grad_ub = x.new_empty((N,)) if need_ub else None
        if need_x or weights or need_gb or need_ub:
            mhc_gated_bwd(grad_out.contiguous(), x, gate_weight, up_weight, gate, up,
                          grad_x=grad_x, grad_gate_weight=grad_g, grad_up_weight=grad_u,
                          grad_gate_bias=grad_gb, grad_up_bias=grad_ub,
                          activation=ctx.activation)
        return (grad_x, grad_g if need_g else None, grad_u if need_u else None, grad_gb, grad_ub,
                None)


def gated_autograd(x: torch.Tensor, gate_weight: torch.Tensor, up_weight: torch.Tensor,
                   gate_bias: torch.Tensor | None = None, up_bias: torch.Tensor | None = None, *,
                   activation: str = "silu") -> torch.Tensor:
    """act(x gate_weight^T + gate_bias) * (x up_weight^T + up_bias) with
    gradients for all five."""
    return Gated.apply(x, gate_weight, up_weight, gate_bias, up_bias, activation)
