"""8-bit integers with a scale for each token and channel: the norm's rows
(MHC_NORM_I8_ROW in include/mhc_rms_norm.h) and the product of them
(MHC_LINEAR_I8_ROW in include/mhc_linear.h).

Tolerances. The sum of a product is an exact integer (at most 131071 * 2^14 <
2^31), so what is left is its rounding to fp32, the product of the two scales,
the product with them, bias and residual (half a step of fp32 each), the
activation as in test_linear.py, and half a step of bf16. A code of the norm is
the nearest integer to a value that is off by the norm's own error and two
roundings, so the value it stands for is off by half a scale and that.
"""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from hyper_connection_residual_mhc_amd import _lib
from hyper_connection_residual_mhc_amd._lib import MHC_ERROR_ALIASING, MHC_ERROR_INVALID_VALUE, MHC_SUCCESS
from test_gated import act_error, quantise_int8
from test_linear import LARGE, MEDIUM, NARROW, ROWS, SMALL, STEP
from test_linear import BASE, GAP, SCALES, fwd_args
from test_rms_norm import EPS, WIDTHS, make as make_norm, rstd_rel, want_stored
from test_rms_norm import fwd_args as norm_args

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# Host rules (CPU)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [{}, {"x": BASE + 1, "w": BASE + GAP + 3}, {"K": 131071, "M": 1}, {"act": 3, "bias": BASE + 6 * GAP}])
def test_valid_products(built_library, kw):
    lib = _lib.linear_lib()
    assert lib.mhc_linear_validate_fwd(*fwd_args(dtype=6, **{**SCALES, **kw})) == MHC_SUCCESS, lib.mhc_linear_last_error_message()


@pytest.mark.parametrize("kw", [{"K": 131072}, {"xs": None}, {"ws": None}, {"xs": BASE + 4 * GAP + 2}, {"dtype": 7}, {"dtype": 5}])
def test_refused_products(built_library, kw):
    lib = _lib.linear_lib()
    assert lib.mhc_linear_validate_fwd(*fwd_args(**{"dtype": 6, **SCALES, **kw})) == MHC_ERROR_INVALID_VALUE
    assert lib.mhc_linear_bwd_workspace_bytes(5, 5, 5, 6) == -1


def test_overlapping_products(built_library):
    lib = _lib.linear_lib()
    assert lib.mhc_linear_validate_fwd(*fwd_args(dtype=6, **{**SCALES, "ws": BASE + 2 * GAP})) == MHC_ERROR_ALIASING


def test_norm_arguments(built_library):
    v = _lib.norm_lib().mhc_rms_norm_validate_fwd
    assert v(*norm_args(out_format=4, scales=BASE + 3 * GAP)) == MHC_SUCCESS
    for kw in ({"scales": None}, {"scales": BASE + 3 * GAP + 2}, {"out_format": 5}):
        assert v(*norm_args(**{"out_format": 4, "scales": BASE + 3 * GAP, **kw})) == MHC_ERROR_INVALID_VALUE, kw


def test_constants_match_the_headers(built_library):
    from hyper_connection_residual_mhc_amd import _build
    text = _build.LINEAR_HEADER.read_text()
    assert f"#define MHC_LINEAR_I8_ROW {_lib.MHC_LINEAR_I8_ROW} " in text
    assert f"#define MHC_LINEAR_MAX_K_I8 {_lib.MHC_LINEAR_MAX_K_I8}\n" in text
    assert f"#define MHC_NORM_I8_ROW {_lib.MHC_NORM_I8_ROW} " in _build.NORM_HEADER.read_text()
    assert _lib.MHC_LINEAR_MAX_K_I8 * 128 * 128 < 1 << 31


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import linear as L, norm
    x, w = torch.zeros(2, 8, dtype=torch.int8), torch.zeros(4, 8, dtype=torch.int8)
    with pytest.raises(TypeError):
        L.linear(x, w, x_scales=torch.ones(2), weight_scales=torch.ones(4))      # not on a GPU
    with pytest.raises(ValueError, match="int4"):
        norm.rms_norm(torch.zeros(2, 8), torch.ones(8), quant="int4")


# ---------------------------------------------------------------------------
# Product (GPU)
# ---------------------------------------------------------------------------

def check(device, M, N, K, seed, activation="none", bias=True, residual=True, launch=None, extreme=False,
          place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(seed)
    if extreme:
        x, w = (torch.randint(0, 2, (r, K), generator=gen, dtype=torch.int8) * -128 for r in (M, N))
        x[0], w[0] = -128, -128                            # the largest sum there is
        xs, ws = (torch.rand(r, generator=gen) * 2.0 ** -16 for r in (M, N))
    else:
        (x, xs), (w, ws) = quantise_int8(torch.randn(M, K, generator=gen)), quantise_int8(torch.randn(N, K, generator=gen) * K ** -0.5)
    b = R.normal(gen, N) if bias else None
    r = R.normal(gen, M, N) if residual else None
    up = [None if t is None else place(t, device) for t in (x, w, b, r, xs, ws)]
    out, z = (torch.empty(M, N, dtype=BF16, device=device) for _ in range(2))
    L.mhc_linear_fwd(up[0], up[1], out, bias=up[2], residual=up[3], x_scales=up[4], weight_scales=up[5],
                     activation=activation, z=z, launch=launch)
    torch.cuda.synchronize()
    total = x.double() @ w.double().t()
    want = total * (xs.double()[:, None] * ws.double())
    dz = want.abs() * 2 * STEP
    if bias:
        want = want + R.d(b)
        dz = dz + want.abs() * STEP
    R.assert_within(z, want, dz + R.rounding(want.abs() + dz, BF16), "z")
    tol, want = act_error(want, dz, activation), R.act(want, activation)
    if residual:
        want = want + R.d(r)
        tol = tol + (want.abs() + tol) * STEP
    R.assert_within(out, want, tol + R.rounding(want.abs() + tol, BF16), "out")
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ROWS, NARROW, SMALL, MEDIUM, LARGE])
def test_product_depths(device, kernel):
    M, N = (5, 40) if kernel == ROWS else (70, 72) if kernel in (NARROW, SMALL) else (140, 264)
    for k, K in enumerate((1, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 520, 1279, 2048)):
        say(f"int8 kernel={kernel} K={K}")
        check(device, M, N, K, seed=k, launch={"kernel": kernel})


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [NARROW, SMALL, MEDIUM, LARGE])
def test_product_tiles(device, kernel):
    bm, bn = {NARROW: (64, 32), SMALL: (64, 64), MEDIUM: (128, 128), LARGE: (256, 256)}[kernel]
    for k, (M, N) in enumerate(((1, 1), (bm - 1, bn - 1), (bm, bn), (bm + 1, bn + 1), (bm + 17, 3 * bn - 9), (5 * bm + 3, 2 * bn))):
        say(f"int8 kernel={kernel} M={M} N={N}")
        check(device, M, N, 384, seed=k, launch={"kernel": kernel, "splits": 1})


@pytest.mark.gpu
def test_product_rows(device):
    for M in (1, 2, 3, 8, 15, 16, 17):
        for N, K in ((1, 300), (7, 4100), (16, 640), (100, 64), (1001, 1279)):
            say(f"int8 M={M} N={N} K={K}")
            check(device, M, N, K, seed=M + N)


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
def test_product_epilogues(device, activation):
    for M, N in ((3, 50), (128, 128), (150, 200)):
        for bias in (False, True):
            for residual in (False, True):
                check(device, M, N, 256, 11, activation, bias, residual)


@pytest.mark.gpu
def test_product_of_the_largest_sums(device):
    """Codes of -128 over the longest sum, on every kernel and in parts: nothing wraps around."""
    for kernel, M, N, K, splits in ((ROWS, 3, 20, 131071, 1), (NARROW, 20, 20, 131071, 3), (SMALL, 20, 40, 131071, 64),
                                    (MEDIUM, 20, 40, 131071, 1), (LARGE, 20, 40, 131056, 2)):
        say(f"int8 kernel={kernel} K={K} splits={splits}")
        check(device, M, N, K, 3, extreme=True, bias=False, residual=False, launch={"kernel": kernel, "splits": splits})


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1100, 1300, 1600 - 7), (600, 1801, 2000 + 24)])
def test_product_rows_that_are_no_whole_pieces(device, M, N, K):
    check(device, M, N, K, seed=M)


@pytest.mark.gpu
def test_a_row_depends_on_nothing_else(device):
    """Whatever kernel, split, batch and alignment: the same bytes, since the sums are exact."""
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(7)
    M, N, K = 300, 200, 1000
    (x, xs), (w, ws) = quantise_int8(torch.randn(M, K, generator=gen)), quantise_int8(torch.randn(N, K, generator=gen))
    b = R.normal(gen, N).to(device)
    x, xs, w, ws = (t.to(device) for t in (x, xs, w, ws))
    want = L.linear(x, w, b, activation="gelu", x_scales=xs, weight_scales=ws).out
    for kernel in (NARROW, SMALL, MEDIUM, LARGE):
        for splits in (1, 2, 5):
            out = torch.empty_like(want)
            L.mhc_linear_fwd(x, w, out, bias=b, activation="gelu", x_scales=xs, weight_scales=ws,
                             launch={"kernel": kernel, "splits": splits})
            assert R.same_bytes(out, want), (kernel, splits)
    for rows in ([0], [299, 4], list(range(17, 40))):
        got = L.linear(x[rows].contiguous(), w, b, activation="gelu", x_scales=xs[rows].contiguous(), weight_scales=ws).out
        assert R.same_bytes(got, want[rows])
    got = L.linear(R.shifted(x.cpu(), device), R.shifted(w.cpu(), device, 3), b, activation="gelu", x_scales=xs, weight_scales=ws).out
    assert R.same_bytes(got, want)


@pytest.mark.gpu
def test_product_writes_nothing_else(device):
    from hyper_connection_residual_mhc_amd import linear as L
    for M, N, K in ((3, 40, 256), (70, 72, 256), (300, 264, 512), (129, 1001, 1279)):
        (x, xs), (w, ws) = (quantise_int8(torch.randn(r, K)) for r in (M, N))
        out = R.Guarded((M, N), BF16, device)
        work = R.Guarded((max(1, L.mhc_linear_fwd_workspace_bytes(M, N, K, 6)),), torch.uint8, device)
        L.mhc_linear_fwd(x.to(device), w.to(device), out.t, x_scales=xs.to(device), weight_scales=ws.to(device), workspace=work.t)
        assert out.untouched() and work.untouched()
    empty = L.linear(torch.empty(0, 64, dtype=torch.int8, device=device), w[:, :64].contiguous().to(device),
                     x_scales=torch.empty(0, device=device), weight_scales=ws.to(device))
    assert empty.out.shape == (0, w.shape[0])


# ---------------------------------------------------------------------------
# Norm (GPU)
# ---------------------------------------------------------------------------

def check_norm(o, v, rel):
    scale = R.d(o.scales)
    want = (v.abs().amax(1) / 127).clamp_min(2.0 ** -126)
    R.assert_within(o.scales, want, want * (rel + 2 * R.U32), "scales")
    q = o.y.cpu().double()
    assert o.y.dtype == torch.int8 and q.abs().max() <= 127
    tol = v.abs() * (rel + 3 * R.U32) + scale[:, None] * (0.5 + 127 * 2 * R.U32)
    R.assert_within((q * scale[:, None]).float(), v, tol + v.abs() * R.U32, "values")


@pytest.mark.gpu
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("source", ["plain", "add", "streams"])
def test_norm_widths(device, H, source):
    from hyper_connection_residual_mhc_amd import norm
    T = 3
    say(f"norm int8 {source} H={H}")
    for k, dtype in enumerate((BF16,) if source == "streams" else (BF16, torch.float16, torch.float32)):
        x, residual, pre, weight = make_norm(T, H, dtype, source, seed=H + k, n=(2, 4, 8)[H % 3])
        up = lambda t: None if t is None else t.to(device)  # noqa: E731
        o = norm.rms_norm(up(x), up(weight), EPS, residual=up(residual), pre=up(pre), quant="int8", return_rstd=True)
        s = want_stored(x, residual, pre)
        assert o.stored is None if source == "plain" else R.same_bytes(o.stored, s)
        v, _ = R.norm(R.d(s), R.d(weight), EPS)
        check_norm(o, v, rstd_rel(H) + 2 * R.U32)
        # into guarded tensors: the same bytes and nothing else
        out, scales = R.Guarded((T, H), torch.int8, device), R.Guarded((T,), torch.float32, device)
        norm.mhc_rms_norm_fwd(up(x), up(weight), out.t, eps=EPS, residual=up(residual), pre=up(pre), scales=scales.t, quant="int8")
        assert out.untouched() and scales.untouched() and R.same_bytes(out.t, o.y) and R.same_bytes(scales.t, o.scales)


@pytest.mark.gpu
def test_norm_codes_at_ties_and_extremes(device):
    """Ties go to the even integer; a row of zeros has codes 0; a row with an infinity or a NaN has scale infinity and
    codes 0, and a product with it is NaN."""
    from hyper_connection_residual_mhc_amd import linear as L, norm
    H = 64
    x = torch.zeros(5, H)
    x[0, 0], x[0, 1:9] = 127.0, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5, 0.25])
    x[0] *= 1.0 / float((x[0].double() ** 2).mean().sqrt())
    x[2, 3], x[3, 4], x[4, 5] = float("inf"), float("nan"), 1.0
    w = torch.ones(H, device=device)
    o = norm.rms_norm(x.to(device), w, 0.0 + 1e-30, quant="int8")
    q = o.y.cpu()
    assert q[0, 0] == 127 and q[0, 8] == 0
    # 0.25 is no tie; the halves may fall to either side by the rounding of the norm, by one code at most
    assert all(abs(float(a) - b) <= 0.5 + 1e-4 for a, b in zip(q[0, 1:8], (0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5)))
    assert not q[1:4].any() and q[4, 5] == 127 and not q[4, :5].any()
    s = o.scales.cpu()
    assert s[1] == 2.0 ** -126 and torch.isinf(s[2]) and torch.isinf(s[3])
    weight, scales = quantise_int8(torch.randn(40, H))
    out = L.linear(o.y, weight.to(device), x_scales=o.scales, weight_scales=scales.to(device)).out.cpu()
    assert torch.isnan(out[2:4]).all() and torch.isfinite(out[[0, 1, 4]]).all() and not out[1].any()


@pytest.mark.gpu
def test_norm_then_product_captured(device):
    """The 8-bit projection of a sublayer, captured and replayed."""
    from hyper_connection_residual_mhc_amd import linear as L, norm
    gen = torch.Generator().manual_seed(8)
    T, H, N = 20, 1288, 300
    x, r = R.normal(gen, T, H).to(device), R.normal(gen, T, H).to(device)
    weight = torch.ones(H, device=device)
    w, ws = (t.to(device) for t in quantise_int8(torch.randn(N, H, generator=gen) * H ** -0.5))

    def step(x):
        o = norm.rms_norm(x, weight, residual=r, quant="int8")
        return o.stored, o.scales, L.linear(o.y, w, activation="silu", x_scales=o.scales, weight_scales=ws).out

    step(x)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for k in range(4):
        new = (x * (k + 1)).contiguous()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, step(new)):
            assert R.same_bytes(p, q), k
