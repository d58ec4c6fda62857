"""The end of a wide tile, whose bias and residual are loaded before they are needed: the
same bytes as the 128 x 128 tiles give, whose sums have the same order, at edges where
rows or columns end inside a tile, a wave or a chunk of 8, at any alignment of what is
read, and nothing written outside."""

from __future__ import annotations

import itertools

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from test_linear import LARGE, MEDIUM

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("M,N", [(256, 256), (512, 768), (257, 264), (300, 520), (129, 259), (1, 9), (128, 8), (127, 15), (513, 1001),
                                 (385, 771), (300, 5)])
def test_same_bytes_as_other_tiles(device, kind, M, N):
    from hyper_connection_residual_mhc_amd import linear as L
    t, K = TYPES[kind], 200
    gen = torch.Generator().manual_seed(M + N)
    x, w = R.normal(gen, M, K, dtype=t).to(device), R.normal(gen, N, K, dtype=t, scale=K ** -0.5).to(device)
    b, r = R.normal(gen, N, dtype=t), R.normal(gen, M, N, dtype=t)
    for has_b, has_r, has_z, activation in itertools.product((False, True), (False, True), (False, True),
                                                             ("none", "relu", "silu", "gelu")):
        say(f"wide epilogue {kind} M={M} N={N} bias={has_b} residual={has_r} z={has_z} {activation}")
        made = []
        for kernel, place in ((MEDIUM, lambda v: v.to(device)), (LARGE, lambda v: v.to(device)),
                              (LARGE, lambda v: R.shifted(v, device))):
            out, z = R.Guarded((M, N), t, device), R.Guarded((M, N), t, device)
            L.mhc_linear_fwd(x, w, out.t, bias=place(b) if has_b else None, residual=place(r) if has_r else None,
                             z=z.t if has_z else None, activation=activation, launch={"kernel": kernel, "splits": 1})
            assert out.untouched() and z.untouched()
            made.append((out.t, z.t))
        for out, z in made[1:]:
            assert R.same_bytes(out, made[0][0]) and (not has_z or R.same_bytes(z, made[0][1]))


@pytest.mark.gpu
def test_many_tiles_to_a_block(device):
    """More tiles than compute units, ragged at both ends: a block's next tile begins while one ends."""
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator(device=device).manual_seed(3)
    M, N, K = 4100, 4803, 136
    x, w, b, r = (torch.randn(s, device=device, generator=gen).to(torch.bfloat16) for s in ((M, K), (N, K), (N,), (M, N)))
    for bias, residual in ((b, r), (b, None), (None, r)):
        got = []
        for kernel in (MEDIUM, LARGE):
            out = torch.empty(M, N, dtype=torch.bfloat16, device=device)
            L.mhc_linear_fwd(x, w, out, bias=bias, residual=residual, activation="silu", launch={"kernel": kernel, "splits": 1})
            got.append(out)
        assert R.same_bytes(*got)
