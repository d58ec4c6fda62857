"""What the bindings of the norm, the product and the write-back share: checks
of a call's tensors, and the stream and device it runs on.

A small call takes less time on the GPU than its marshalling on the host, so
the checks here cost little where nothing is wrong (one tensor 0.3 us, against
0.6 for `ops._require`, which names what is) and the device is switched only
where it is another than the current one (1.2 us).
"""

from __future__ import annotations

import contextlib

import torch

from .ops import _require

_NOTHING = contextlib.nullcontext()


def require(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: torch.device
            ) -> None:
    """Raises unless t is a contiguous GPU tensor of this dtype, shape and
    device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.device == device and t.is_contiguous()):
        _require(t, name, dtype, shape, device)


def stream_handle(device: torch.device, stream: torch.cuda.Stream | None) -> int:
    """The raw handle of `stream`, or of torch's current one on `device`."""
    if stream is not None:
        return int(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(device.index)


def on(device: torch.device):
    """Context in which `device` is the current one."""
    return _NOTHING if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def address(t: torch.Tensor | None) -> int | None:
    """Data address of an optional tensor."""
    return None if t is None else t.data_ptr()


def workspace_of(workspace: torch.Tensor | None, need: int, device: torch.device,
                 stream: torch.cuda.Stream | None) -> tuple[int | None, int, torch.Tensor | None]:
    """(address, bytes, owner) of the caller's workspace, or of a fresh one of
    `need` bytes. A fresh one belongs to `stream`: memory of torch's current
    stream may still be in use there when `stream` starts to write."""
    if workspace is None:
        if need <= 0:
            return None, 0, None
        with _NOTHING if stream is None else torch.cuda.stream(stream):
            workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
