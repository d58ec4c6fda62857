"""The product's backward at the limits of 16 bits (include/mhc_linear.h). Where z passed its range:
a pre-activation beyond +-65520 is stored as an infinity in fp16 while the
forward's output, made from the fp32 value, may be finite, so the slope at an
infinite z is the activation's limit. And where its products are rounded: grad_bias sums them
before that."""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
from gpu_util import say

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
INF, NAN = float("inf"), float("nan")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("activation", ["relu", "silu", "gelu"])
def test_slope_of_infinite_z(device, kind, activation):
    """With unit matrices for x and the weight both products give gz itself: the slope is 1 at +inf and far to the
    right, 0 at -inf and far to the left, NaN at NaN alone (in its row and column of the gradients)."""
    from hyper_connection_residual_mhc_amd import linear as L
    say(f"slope at infinities {kind} {activation}")
    t = TYPES[kind]
    size = 16
    eye = torch.eye(size, dtype=t)
    g = torch.arange(1, size * size + 1).view(size, size).remainder(7).add(1).to(t)  # exact in both types
    z = torch.zeros(size, size, dtype=t)
    far = torch.finfo(t).max
    # infinities together with values of every size in the same rows and columns
    z[0::4], z[1::4], z[2::4], z[3::4] = INF, -INF, far, -far
    want = torch.where(z > 0, g, torch.zeros_like(g))
    for with_nan in (False, True):
        if with_nan:
            z[5, 9] = NAN
        gx, gw, gb = L.linear_backward(g.to(device), eye.to(device), eye.to(device), activation=activation,
                                       z=z.to(device), bias=True)
        gx, gw, gb = gx.cpu(), gw.cpu().t(), gb.cpu()
        rows = torch.arange(size) != (5 if with_nan else -1)
        columns = torch.arange(size) != (9 if with_nan else -1)
        assert torch.equal(gx[rows], want[rows]) and torch.equal(gw[:, columns], want[:, columns])
        assert torch.equal(gb[columns].float(), want.float().sum(0)[columns])   # 16 terms of at most 7: exact
        if with_nan:
            assert torch.isnan(gx[5]).all() and torch.isnan(gw[:, 9]).all() and torch.isnan(gb[9])


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["relu", "silu", "gelu"])
def test_gradients_where_fp16_z_overflows(device, activation):
    """A training step whose forward is finite has finite gradients: z reaches -76800 and is stored as -inf, the
    output there is 0 and so is the slope."""
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(7)
    M, N, K = 40, 24, 48
    x, w = R.normal(gen, M, K, dtype=torch.float16), R.normal(gen, N, K, dtype=torch.float16, scale=0.2)
    x[3], w[5] = 0, 0
    x[3, 0], w[5, 0] = 256, -300
    g = R.normal(gen, M, N, dtype=torch.float16)
    leaves = [v.to(device).requires_grad_() for v in (x, w)]
    out = L.linear_autograd(*leaves, activation=activation)
    assert float(out.detach()[3, 5]) == 0 and torch.isfinite(out.detach()).all()
    z = L.linear(x.to(device), w.to(device), activation=activation, return_z=True).z
    assert torch.isinf(z[3, 5])
    gx, gw = (v.cpu() for v in torch.autograd.grad(out, leaves, g.to(device)))
    assert torch.isfinite(gx).all() and torch.isfinite(gw).all()
    # against fp64: gz is off by the slope's 1e-4 at most (values of z up to 16 rounded to fp16 move it by less
    # than 1.13 * 2^-8 at most) and its rounding; both sums have M or N terms
    xv, wv, gv = R.d(x), R.d(w), R.d(g)
    wx, ww, _, gz = R.linear_grads(gv, xv, wv, R.linear(xv, wv)[1], activation)
    dz = gv.abs() * (R.d(z).clamp(-16, 16).abs() * 2.0 ** -11 * 1.13 + 1e-4) + gz.abs() * 2.0 ** -11
    if activation == "relu":
        dz = gz.abs() * 2.0 ** -11
    tol = dz @ wv.abs() + gz.abs() @ wv.abs() * 2.0 ** -18
    R.assert_within(gx, wx, tol + R.rounding(wx.abs() + tol, torch.float16), "grad_x")
    tol = dz.t() @ xv.abs() + gz.abs().t() @ xv.abs() * 2.0 ** -18
    R.assert_within(gw, ww, tol + R.rounding(ww.abs() + tol, torch.float16), "grad_weight")


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_bias_gradient_sums_before_the_rounding(device, activation):
    """grad_bias adds grad_out * act'(z) before its rounding to 16 bits: over equal rows it is within half a step of
    the exact sum, which the sum of the rounded products is not."""
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(5)
    M, N, t = 1000, 200, torch.float16
    g, z = (R.normal(gen, 1, N, dtype=t, scale=s).expand(M, N).contiguous() for s in (0.01, 1.0))
    gb = L.linear_backward(g.to(device), torch.ones(M, 8, dtype=t, device=device), torch.ones(N, 8, dtype=t, device=device),
                           activation=activation, z=z.to(device), bias=True)[2]
    each = (R.d(g) * R.act_slope(R.d(z), activation))[0]
    want = each * M
    # the slope (1e-5 fitted tail, 2^-20 of its parts), the product, and additions of at most 1000 / 4 + 4 + 256 equal
    # terms, each off by at most half a step of fp32
    tol = R.d(g)[0].abs() * M * (1e-5 + 8 * 2.0 ** -20) + want.abs() * (2 + 510) * R.U32
    rounded = (each.to(t).double() * M).to(t).double()
    assert bool(((rounded - want).abs() > tol + R.rounding(want.abs() + tol, t)).any())
    R.assert_within(gb, want, tol + R.rounding(want.abs() + tol, t), "grad_bias")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 70])
def test_forward_of_infinite_z(device, M):
    """A bias of -inf or +inf, as a mask of columns: relu and gelu give 0 and inf, silu NaN and inf, and the other
    columns are what they are without it."""
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(M)
    x, w = R.normal(gen, M, 96).to(device), R.normal(gen, 40, 96).to(device)
    bias = R.normal(gen, 40)
    masked = bias.clone()
    masked[5], masked[11] = -INF, INF
    rest = [n for n in range(40) if n not in (5, 11)]
    for activation in ("relu", "gelu", "silu"):
        plain = L.linear(x, w, bias.to(device), activation=activation).out.cpu()
        out = L.linear(x, w, masked.to(device), activation=activation).out.cpu()
        assert R.same_bytes(out[:, rest], plain[:, rest])
        assert (out[:, 11] == INF).all()
        assert torch.isnan(out[:, 5]).all() if activation == "silu" else (out[:, 5] == 0).all()
