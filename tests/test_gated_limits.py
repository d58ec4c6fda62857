"""The gated block's backward (include/mhc_gated.h) around the largest dg and du whose
weights' gradients are loaded straight into LDS: 2^31 bytes of them side by side. Past
that the products take other kernels, whose places in memory no longer fit 32 bits.
"""

from __future__ import annotations

import math

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from test_linear import STEP, additions

BF16 = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("N", [13056, 13120, 13101])
def test_backward_of_2_to_the_31_bytes(device, N):
    """40960 rows: 13056 columns stay 8 MiB below, 13120 and 13101 pass it. The products of two bf16 values are exact in
    fp32 and round to 16 bits once, as here; fp64 on the GPU."""
    from hyper_connection_residual_mhc_amd import gated as G
    M, K = 40960, 72
    half = -(-N // 64) * 64
    assert (M * half * 4 > 2 ** 31 - 1) == (N > 13056)
    say(f"gated backward M={M} N={N} K={K}")
    gen = torch.Generator(device=device).manual_seed(N)
    d, u, g = (torch.randn(M, N, device=device, generator=gen).to(BF16) for _ in range(3))
    x, wg, wu = (torch.randn(s, K, device=device, generator=gen).to(BF16) for s in (M, N, N))
    got = G.gated_backward(d, x, wg, wu, g, u, bias=True, activation="none")
    xv, wgv, wuv = x.double(), wg.double(), wu.double()
    sizes = additions(2 * half, 32) * STEP, additions(M, 32) * STEP
    # the biases' sums: about 1024 blocks of 512 columns, each of four waves every fourth row, then every fourth part
    parts = 1024 // math.ceil(half / 512)
    long = math.ceil(math.ceil(M / parts) / 4) + 4 + math.ceil(parts / 4) + 4
    want = torch.zeros(M, K, dtype=torch.float64, device=device)
    size = torch.zeros_like(want)
    for other, weight, p, bias in ((u, wgv, got[1], got[3]), (g, wuv, got[2], got[4])):
        f = d.double() * other.double()
        bound = f.abs().sum(0) * long * STEP
        assert float(((bias.double() - f.sum(0)).abs() - bound - (f.sum(0).abs() + bound) * R.HALF_STEP[BF16]).max()) <= 0
        f = f.to(BF16).double()
        wanted, tol = f.t() @ xv, f.abs().t() @ xv.abs() * sizes[1]
        assert float(((p.double() - wanted).abs() - tol - (wanted.abs() + tol) * R.HALF_STEP[BF16] - R.HALF_TINY[BF16]).max()) <= 0
        want += f @ weight
        size += f.abs() @ weight.abs()
    tol = size * sizes[0]
    assert float(((got[0].double() - want).abs() - tol - (want.abs() + tol) * R.HALF_STEP[BF16] - R.HALF_TINY[BF16]).max()) <= 0
