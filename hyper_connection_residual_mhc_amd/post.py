"""Python binding of the write-back into the residual streams: argument
marshalling only.

Formulas, types and rules: include/mhc_post.h. All arithmetic runs in the
gfx950 kernels; a missing library raises ImportError.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._call import on, require, stream_handle
from ._lib import check_post
from .ops import _shapes_n


def _check_inputs(residual: torch.Tensor, comb: torch.Tensor, post: torch.Tensor,
                  y: torch.Tensor) -> tuple[int, int, int]:
    T, n, H = _shapes_n(residual)
    dev = residual.device
    require(residual, "residual", torch.bfloat16, (T, n, H), dev)
    require(comb, "comb", torch.float32, (T, n, n), dev)
    require(post, "post", torch.float32, (T, n), dev)
    require(y, "y", torch.bfloat16, (T, H), dev)
    return T, n, H


def mhc_post_fwd(residual: torch.Tensor, comb: torch.Tensor, post: torch.Tensor, y: torch.Tensor,
                 out: torch.Tensor, stream: torch.cuda.Stream | None = None,
                 start_event: int | None = None, stop_event: int | None = None) -> torch.Tensor:
    """out [T, n, H] bf16 <- comb [T, n, n] . residual [T, n, H] + post [T, n]
    (x) y [T, H]; the gates are fp32, the rest bf16. Asynchronous."""
    T, n, H = _check_inputs(residual, comb, post, y)
    require(out, "out", torch.bfloat16, (T, n, H), residual.device)
    return _launch_fwd(residual, comb, post, y, out, T, n, H, stream, start_event, stop_event)


def _launch_fwd(residual, comb, post, y, out, T, n, H, stream, start_event, stop_event
                ) -> torch.Tensor:
    dev = residual.device
    with on(dev):
        st = _lib.post_lib().mhc_post_fwd(
            residual.data_ptr(), comb.data_ptr(), post.data_ptr(), y.data_ptr(), out.data_ptr(),
            T, n, H, stream_handle(dev, stream), start_event, stop_event)
    check_post(st)
    return out


def mhc_post_bwd(grad_out: torch.Tensor, residual: torch.Tensor, comb: torch.Tensor,
                 post: torch.Tensor, y: torch.Tensor, grad_residual: torch.Tensor,
                 grad_comb: torch.Tensor, grad_post: torch.Tensor, grad_y: torch.Tensor,
                 stream: torch.cuda.Stream | None = None, start_event: int | None = None,
                 stop_event: int | None = None
                 ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(grad_residual [T, n, H] bf16, grad_comb [T, n, n] fp32, grad_post
    [T, n] fp32, grad_y [T, H] bf16) <- backward. Asynchronous."""
    T, n, H = _check_inputs(residual, comb, post, y)
    dev = residual.device
    require(grad_out, "grad_out", torch.bfloat16, (T, n, H), dev)
    require(grad_residual, "grad_residual", torch.bfloat16, (T, n, H), dev)
    require(grad_comb, "grad_comb", torch.float32, (T, n, n), dev)
    require(grad_post, "grad_post", torch.float32, (T, n), dev)
    require(grad_y, "grad_y", torch.bfloat16, (T, H), dev)
    with on(dev):
        st = _lib.post_lib().mhc_post_bwd(
            grad_out.data_ptr(), residual.data_ptr(), comb.data_ptr(), post.data_ptr(),
            y.data_ptr(), grad_residual.data_ptr(), grad_comb.data_ptr(), grad_post.data_ptr(),
            grad_y.data_ptr(), T, n, H, stream_handle(dev, stream), start_event, stop_event)
    check_post(st)
    return grad_residual, grad_comb, grad_post, grad_y


# ---------------------------------------------------------------------------
# Allocating conveniences and autograd
# ---------------------------------------------------------------------------

def post_update(residual: torch.Tensor, comb: torch.Tensor, post: torch.Tensor,
                y: torch.Tensor) -> torch.Tensor:
    """The write-back with a freshly allocated output (no autograd)."""
    T, n, H = _check_inputs(residual, comb, post, y)
    return _launch_fwd(residual, comb, post, y, torch.empty_like(residual), T, n, H, None, None,
                       None)


def post_update_backward(grad_out: torch.Tensor, residual: torch.Tensor, comb: torch.Tensor,
                         post: torch.Tensor, y: torch.Tensor
                         ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward with freshly allocated gradients: (grad_residual, grad_comb,
    grad_post, grad_y)."""
    return mhc_post_bwd(grad_out, residual, comb, post, y, torch.empty_like(residual),
                        torch.empty_like(comb), torch.empty_like(post), torch.empty_like(y))


class PostUpdate(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the gfx950 kernels."""

    @staticmethod
    def forward(ctx, residual, comb, post, y):
        ctx.save_for_backward(residual, comb, post, y)
        return post_update(residual, comb, post, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        grads = post_update_backward(grad_out.contiguous(), *ctx.saved_tensors)
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad))


def post_update_autograd(residual: torch.Tensor, comb: torch.Tensor, post: torch.Tensor,
                         y: torch.Tensor) -> torch.Tensor:
    return PostUpdate.apply(residual, comb, post, y)
