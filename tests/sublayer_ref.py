"""Plain fp64 forms of the operators around the collapse (norm, product,
write-back) and the tools their tests share. Nothing here uses the package's
kernels: the formulas are those of the C headers, written with torch on the
CPU in double precision."""

from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}
# half of the smallest subnormal: the rounding error next to zero
HALF_TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150,
             torch.float8_e4m3fn: 2.0 ** -10}
U32 = 2.0 ** -24  # half a step of fp32, relative


def d(t: torch.Tensor | None) -> torch.Tensor | None:
    """The tensor's values in fp64 on the CPU."""
    return None if t is None else t.detach().cpu().to(torch.float32).double() \
        if t.dtype in (torch.float8_e4m3fn, torch.float8_e8m0fnu) else t.detach().cpu().double()


def rounding(ref: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """What one rounding of `ref` to dtype may be off."""
    return ref.abs() * HALF_STEP[dtype] + HALF_TINY[dtype]


def assert_within(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what: str) -> None:
    """|got - ref| <= tol everywhere; the worst place in the message. Where ref
    is not finite, got is the same infinity or a NaN too."""
    g = d(got)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)} != {tuple(ref.shape)}"
    if not g.numel():
        return
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN in other places"
    same = ~fine & ~torch.isnan(ref)
    assert torch.equal(g[same], ref[same]), f"{what}: infinities in other places"
    over = torch.where(fine, (g - ref).abs() - tol, torch.zeros_like(ref))
    over = torch.where(torch.isnan(over), torch.full_like(over, math.inf), over)
    over = torch.where(fine, over, torch.full_like(over, -1.0))
    worst = int(over.argmax())
    assert float(over.max()) <= 0, (
        f"{what}: {int((over > 0).sum())} of {g.numel()} outside; worst at flat index {worst}: got "
        f"{float(g.flatten()[worst])!r}, want {float(ref.flatten()[worst])!r} within "
        f"{float(tol.expand_as(ref).flatten()[worst])!r}")


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def norm(s: torch.Tensor, w: torch.Tensor, eps: float) -> tuple[torch.Tensor, torch.Tensor]:
    """(y [T, H], rstd [T]) of the stored rows s, all fp64."""
    rstd = 1 / torch.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * w, rstd


def norm_grads(g, s, w, rstd, grad_stored=None):
    """(grad_x, grad_weight) by the formulas of mhc_rms_norm.h."""
    u = g * w
    c = (u * s).mean(1, keepdim=True) * rstd[:, None] ** 2
    gx = rstd[:, None] * (u - s * c)
    return (gx if grad_stored is None else gx + grad_stored), (g * s * rstd[:, None]).sum(0)


def mx_power(amax: torch.Tensor) -> torch.Tensor:
    """The smallest integer p in [-127, 127] with amax <= 448 * 2^p."""
    m, e = torch.frexp(amax.double() / 448)
    p = torch.where(m == 0.5, e - 1, e)
    return torch.where(m == 0, torch.full_like(p, -127), p).clamp(-127, 127)


def block_amax(v: torch.Tensor) -> torch.Tensor:
    """Largest magnitude of each 32 consecutive columns (the last block may be short)."""
    v = torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 32))
    return v.view(v.shape[0], -1, 32).amax(2)


# ---------------------------------------------------------------------------
# Write-back
# ---------------------------------------------------------------------------

def post(r, comb, gate, y):
    return torch.einsum("tij,tjh->tih", comb, r) + gate[:, :, None] * y[:, None]


def post_grads(g, r, comb, gate, y):
    """(grad_residual, grad_comb, grad_post, grad_y) by the formulas of mhc_post.h."""
    return (torch.einsum("tij,tih->tjh", comb, g), torch.einsum("tih,tjh->tij", g, r),
            torch.einsum("tih,th->ti", g, y), torch.einsum("ti,tih->th", gate, g))


# ---------------------------------------------------------------------------
# Differences
# ---------------------------------------------------------------------------

def differences(f, x: torch.Tensor, step: float = 1e-5) -> torch.Tensor:
    """Central differences of the scalar f at every element of x (fp64)."""
    out = torch.empty_like(x)
    flat, of = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        up = float(f())
        flat[i] = keep - step
        of[i] = (up - float(f())) / (2 * step)
        flat[i] = keep
    return out


# ---------------------------------------------------------------------------
# Device tensors
# ---------------------------------------------------------------------------

def normal(gen: torch.Generator, *shape, dtype=torch.bfloat16, scale: float = 1.0) -> torch.Tensor:
    """Seeded normal values on the CPU, rounded to dtype."""
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * scale).to(dtype)


def shifted(t: torch.Tensor, dev, elements: int = 1) -> torch.Tensor:
    """A contiguous device copy whose data starts `elements` elements past an
    aligned address."""
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device=dev)
    view = buf[elements:].view(t.shape)
    view.copy_(t)
    return view


class Guarded:
    """A device tensor between two 1-KiB regions of a fixed byte."""

    EDGE = 1024

    def __init__(self, shape, dtype, dev, fill: int = 0xA5):
        self.fill = fill
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        self.bytes = torch.full((n + 2 * self.EDGE,), fill, dtype=torch.uint8, device=dev)
        self.n = n
        self.t = self.bytes[self.EDGE:self.EDGE + n].view(dtype).view(shape)

    def untouched(self) -> bool:
        b = self.bytes.cpu()
        return bool((b[:self.EDGE] == self.fill).all() and (b[self.EDGE + self.n:] == self.fill).all())


def same_bytes(a: torch.Tensor, b: torch.Tensor) -> bool:
    a, b = a.contiguous().cpu(), b.contiguous().cpu()
    return a.shape == b.shape and torch.equal(a.flatten().view(torch.uint8), b.flatten().view(torch.uint8))


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------

def tail(a: torch.Tensor) -> torch.Tensor:
    """The normal distribution's tail past a."""
    return 0.5 * torch.special.erfc(a * 0.5 ** 0.5)


def act(z: torch.Tensor, name: str) -> torch.Tensor:
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * tail(-z) if name == "gelu" else z


def act_slope(z: torch.Tensor, name: str) -> torch.Tensor:
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return tail(-z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def linear(x, w, bias=None, activation="none", residual=None):
    """(out, z), all fp64."""
    z = x @ w.t()
    z = z if bias is None else z + bias
    out = act(z, activation)
    return (out if residual is None else out + residual), z


def linear_grads(g, x, w, z, activation):
    """(grad_x, grad_weight, grad_bias, gz) without the rounding of gz."""
    gz = g * act_slope(z, activation)
    return gz @ w, gz.t() @ x, gz.sum(0), gz


def dequantise(q: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values of e4m3 codes with fp32 row scales or e8m0 scales of 32 columns."""
    v = d(q)
    if scales.dtype == torch.float32:
        return v * d(scales)[:, None]
    return v * d(scales).repeat_interleave(32, 1)[:, :q.shape[1]]


def quantise(v: torch.Tensor, kind: str) -> tuple[torch.Tensor, torch.Tensor]:
    """fp32 rows on the CPU in e4m3 with "row" or "mx" scales."""
    if kind == "row":
        s = (v.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        return (v / s[:, None]).to(torch.float8_e4m3fn), s
    p = mx_power(block_amax(v))
    scale = (2.0 ** p.double()).repeat_interleave(32, 1)[:, :v.shape[1]]
    return (v.double() / scale).float().to(torch.float8_e4m3fn), (p + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
