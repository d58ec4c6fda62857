"""The norm where sums of squares leave the range of fp32 (include/mhc_rms_norm.h)."""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [64, 1279, 7168, 20008])
def test_sums_past_the_range(device, dtype, H):
    """Rows of huge values have rstd 0, rows of tiny ones inf with eps 0; just inside the range the norm is right, and
    every row is the same as alone."""
    from hyper_connection_residual_mhc_amd import norm
    gen = torch.Generator().manual_seed(H)
    x = (R.normal(gen, 5, H, dtype=torch.float32).clamp(-4, 4) + 0.01) * torch.tensor([1e22, 1e16, 1.0, 1e-16, 1e-30])[:, None]
    x, w = x.to(dtype).to(device), torch.ones(H, device=device)
    o = norm.rms_norm(x, w, 0.0, return_rstd=True)
    assert float(o.rstd[0]) == 0 and not o.y[0].float().any()
    assert float(o.rstd[4]) == float("inf")
    _, want = R.norm(R.d(x), R.d(w), 0.0)
    # at most 8 * ceil(H / 512) + 13 roundings in the sum of squares (64 threads hold up to 512 columns, longer rows
    # have more), half of them in rstd, and four more; squares of 1e-16 are far above the subnormals
    tol = want * ((8 * (H // 512 + 1) + 13) / 2 + 4) * R.U32
    assert ((R.d(o.rstd) - want).abs() <= tol)[1:4].all()
    for t in range(5):
        one = norm.rms_norm(x[t:t + 1], w, 0.0, return_rstd=True)
        assert R.same_bytes(one.y, o.y[t:t + 1]) and R.same_bytes(one.rstd, o.rstd[t:t + 1])
