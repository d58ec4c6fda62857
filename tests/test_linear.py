"""The matrix product with bias, activation and residual (include/mhc_linear.h)
against its fp64 form, forward and backward, and the rules of the call.

Tolerances. The products of two operand values are exact in fp32. A term of a
sum over k goes through at most L additions: the 32 (16-bit) or 128 (8-bit)
terms of one matrix instruction, the chain of instructions over K, and the
joins of a block's waves or of a split's parts. Each addition is taken to be
off by at most one step of fp32, 2^-23 of its result, so a sum is off by at
most L 2^-23 of the sum of its terms' magnitudes. The 8-bit matrix instruction
first lines up the products of each 8 consecutive k: with 2^E the largest of
their powers of two, the bits of every product below 2^(E - 13) are dropped
(measured: 2^E + 2^(E-13) - 2^E comes back whole, 2^(E-14) as 0, 1.5 * 2^(E-13)
as 2^(E-13), for every place in the 8 and for no place outside). A product
loses less than 2^(E-13) and the largest, at least 2^E, none, so a group of 8
is off by at most 7 * 2^-13 of its largest product. Then come a rounding each
for scale, bias and residual, the activation (its slope is at most 1.13; its
exponential and reciprocal are good to 2^-21 of the tail or the sigmoid, the
fitted tail to 1e-5), and half a step of the output's type.
"""

from __future__ import annotations

import math

import pytest
import torch

import sublayer_ref as R
from hyper_connection_residual_mhc_amd import _lib
from hyper_connection_residual_mhc_amd._lib import (MHC_ERROR_ALIASING, MHC_ERROR_INVALID_VALUE,
                                                    MHC_SUCCESS)
from gpu_util import say

BF16, F16 = torch.bfloat16, torch.float16
STEP = 2.0 ** -23
ABI = {"bf16": 1, "f16": 2, "row": 3, "mx": 4}
ROWS, NARROW, SMALL, MEDIUM, LARGE = 1, 2, 3, 4, 5


def additions(K: int, wide: int) -> int:
    """Additions that a term of a sum over K goes through, at most."""
    return wide + math.ceil(K / wide) + 64 + 16


def dropped(xv: torch.Tensor, wv: torch.Tensor) -> torch.Tensor:
    """What the 8-bit instruction drops of x w^T, at most: [M, N]."""
    K = xv.shape[1]
    x, w = (torch.nn.functional.pad(v.abs(), (0, -K % 8)).view(v.shape[0], -1, 8) for v in (xv, wv))
    total = torch.zeros(xv.shape[0], wv.shape[0], dtype=torch.float64)
    for g in range(x.shape[1]):
        largest = x[:, None, g, 0] * w[None, :, g, 0]
        for k in range(1, 8):
            largest = torch.maximum(largest, x[:, None, g, k] * w[None, :, g, k])
        total += largest
    return total * 7 * 2.0 ** -13


# ---------------------------------------------------------------------------
# The fp64 form itself, and host rules (CPU)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_formula_gradients_are_the_differences_of_the_forward(name):
    gen = torch.Generator().manual_seed(3)
    M, N, K = 3, 4, 5
    x, w, b, g = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((M, K), (N, K), (N,), (M, N)))

    def loss():
        return (R.linear(x, w, b, name)[0] * g).sum()

    z = R.linear(x, w, b)[1]
    assert z.abs().min() > 1e-3                            # no kink of relu within a step
    gx, gw, gb, _ = R.linear_grads(g, x, w, z, name)
    for leaf, grad in ((x, gx), (w, gw), (b, gb)):
        assert torch.allclose(grad, R.differences(loss, leaf), rtol=0, atol=1e-7)


BASE = 1 << 36
GAP = 1 << 31


@pytest.fixture(scope="module")
def lib(built_library):
    return _lib.linear_lib()


def fwd_args(**kw):
    a = dict(x=BASE, xs=None, w=BASE + GAP, ws=None, bias=None, residual=None, out=BASE + 2 * GAP, z=None,
             workspace=BASE + 3 * GAP, workspace_bytes=1 << 30, M=20, N=40, K=50, dtype=1, act=0, launch=None)
    a.update(kw)
    return list(a.values())


SCALES = dict(xs=BASE + 4 * GAP, ws=BASE + 5 * GAP)


@pytest.mark.parametrize("kw", [
    {}, {"dtype": 2}, {"bias": BASE + 6 * GAP, "residual": BASE + 7 * GAP, "z": BASE + 8 * GAP, "act": 3},
    {"dtype": 3, **SCALES}, {"dtype": 4, **SCALES}, {"dtype": 4, "xs": BASE + 4 * GAP + 1, "ws": BASE + 5 * GAP + 3},
    {"dtype": 3, **SCALES, "x": BASE + 1, "w": BASE + GAP + 1}, {"M": 0, "x": None, "w": None, "out": None},
    {"M": 1, "N": 1, "K": 1, "workspace": None, "workspace_bytes": 0}, {"K": 1 << 21, "M": 1},
])
def test_valid_forward_arguments(lib, kw):
    assert lib.mhc_linear_validate_fwd(*fwd_args(**kw)) == MHC_SUCCESS, lib.mhc_linear_last_error_message()


@pytest.mark.parametrize("kw", [
    {"M": -1}, {"M": 1 << 31}, {"N": 0}, {"N": 1 << 31}, {"K": 0}, {"K": (1 << 21) + 1}, {"dtype": 0}, {"dtype": 5},
    {"act": -1}, {"act": 4}, {"x": None}, {"w": None}, {"out": None}, {"x": BASE + 1}, {"out": BASE + 2 * GAP + 1},
    {"bias": BASE + 6 * GAP + 1}, {"dtype": 3}, {"dtype": 4}, {"dtype": 3, "xs": BASE + 4 * GAP},
    {"dtype": 3, "xs": BASE + 4 * GAP + 2, "ws": BASE + 5 * GAP}, {**SCALES}, {"M": 1 << 30, "N": 1 << 30},
    {"M": 64, "K": 4096, "workspace_bytes": 0}, {"M": 64, "K": 4096, "workspace": None},
])
def test_refused_forward_arguments(lib, kw):
    assert lib.mhc_linear_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_INVALID_VALUE
    assert lib.mhc_linear_last_error_message() != b""


@pytest.mark.parametrize("kw", [
    {"out": BASE}, {"out": BASE + GAP}, {"z": BASE + 2 * GAP}, {"residual": BASE + 2 * GAP}, {"bias": BASE + 2 * GAP},
    {"dtype": 4, "xs": BASE + 2 * GAP, "ws": BASE + 5 * GAP}, {"M": 64, "K": 4096, "workspace": BASE},
])
def test_overlapping_forward_arguments(lib, kw):
    assert lib.mhc_linear_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_ALIASING


@pytest.mark.parametrize("M, N, launch, fits", [
    (1, 1 << 26, None, True), (1, (1 << 26) + 1, None, False), (16, (1 << 26) + 1, {"kernel": ROWS}, False),
    (1 << 29, 32, None, True), ((1 << 29) + 1, 32, None, False),            # tiles of 64 x 32
    (1 << 28, 32, {"kernel": NARROW, "splits": 2}, True), ((1 << 28) + 1, 32, {"kernel": NARROW, "splits": 2}, False),
    (1 << 29, 256, None, True), ((1 << 29) + 1, 256, None, False),          # tiles of 256 x 256
    ((1 << 31) - 1, (1 << 31) - 1, None, False),
])
def test_launches_hold_their_tiles(lib, M, N, launch, fits):
    from hyper_connection_residual_mhc_amd import linear as L
    if fits:
        assert L.mhc_linear_plan(M, N, 128, 1, launch)["kernel"]
        return
    with pytest.raises(_lib.MhcError):
        L.mhc_linear_plan(M, N, 128, 1, launch)
    assert lib.mhc_linear_validate_fwd(*fwd_args(M=M, N=N, K=128, launch=L._launch_arg(launch))) == MHC_ERROR_INVALID_VALUE


def test_launches(lib):
    from hyper_connection_residual_mhc_amd import linear as L
    bad = [{"kernel": 6}, {"kernel": -1}, {"splits": -1}, {"splits": 65}, {"kernel": 1, "splits": 2}]
    for launch in bad:
        with pytest.raises(_lib.MhcError):
            L.mhc_linear_plan(8, 64, 64, 1, launch)
        assert lib.mhc_linear_validate_fwd(*fwd_args(M=8, launch=L._launch_arg(launch))) == MHC_ERROR_INVALID_VALUE
        with pytest.raises(ValueError):
            L.mhc_linear_fwd_workspace_bytes(8, 64, 64, 1, launch)
    with pytest.raises(_lib.MhcError):
        L.mhc_linear_plan(17, 64, 64, 1, {"kernel": ROWS})
    for kernel in (NARROW, SMALL, MEDIUM, LARGE):
        for dtype in (1, 4):
            p = L.mhc_linear_plan(100, 100, 4096, dtype, {"kernel": kernel, "splits": 3})
            assert p == {"kernel": kernel, "splits": 3}
            need = 100 * 100 * 4 * 3                        # each part's sums, from a multiple of 256 bytes on
            assert L.mhc_linear_fwd_workspace_bytes(100, 100, 4096, dtype, p) == -(-need // 256) * 256
            assert L.mhc_linear_plan(100, 100, 60, dtype, {"kernel": kernel, "splits": 8})["splits"] == 1
            # every part has a tile of the sum: 5 tiles in 4 parts are 3 parts of 2
            assert L.mhc_linear_plan(100, 100, 640 // (1 if dtype == 4 else 2), dtype,
                                     {"kernel": kernel, "splits": 4})["splits"] == 3
    for M, N, K in ((1, 1, 1), (16, 7168, 4096), (17, 24, 28672), (300, 1000, 5000), (8192, 8192, 8192)):
        p = L.mhc_linear_plan(M, N, K, 1)
        assert p["kernel"] and p["splits"] >= 1
        assert L.mhc_linear_plan(M, N, K, 1, p) == p


def bwd_args(**kw):
    a = dict(grad_out=BASE, x=BASE + GAP, w=BASE + 2 * GAP, z=BASE + 3 * GAP, gx=BASE + 4 * GAP, gw=BASE + 5 * GAP,
             gb=BASE + 6 * GAP, workspace=BASE + 7 * GAP, workspace_bytes=1 << 30, M=20, N=40, K=50, dtype=1, act=3)
    a.update(kw)
    return list(a.values())


def test_backward_arguments(lib):
    v = lib.mhc_linear_validate_bwd
    for kw in ({}, {"act": 0, "z": None}, {"gx": None}, {"gw": None}, {"gb": None}, {"gx": None, "gw": None, "gb": None},
               {"M": 0, "grad_out": None, "x": None, "w": None, "z": None, "workspace": None, "workspace_bytes": 0}):
        assert v(*bwd_args(**kw)) == MHC_SUCCESS, kw
    for kw in ({"z": None}, {"dtype": 3}, {"dtype": 4}, {"M": -1}, {"N": 0}, {"K": 0}, {"M": (1 << 21) + 1},
               {"N": (1 << 21) + 1}, {"act": 9}, {"x": None}, {"workspace_bytes": 100}, {"workspace": None},
               {"workspace": BASE + 7 * GAP + 8}, {"gw": BASE + 5 * GAP + 1}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
    for kw in ({"gx": BASE}, {"gx": BASE + 5 * GAP}, {"gb": BASE + 2 * GAP}, {"workspace": BASE + GAP}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_ALIASING, kw
    assert lib.mhc_linear_bwd_workspace_bytes(0, 5, 5, 1) == 0
    assert lib.mhc_linear_bwd_workspace_bytes(5, 5, 5, 3) == -1


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import linear as L
    x, w = torch.zeros(2, 8, dtype=BF16), torch.zeros(4, 8, dtype=BF16)
    with pytest.raises(TypeError):
        L.linear(x, w)                                     # not on a GPU
    with pytest.raises(TypeError):
        L.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        L.linear(x[0], w)
    with pytest.raises(ValueError):
        L.linear(x, w, x_scales=torch.ones(2))


# ---------------------------------------------------------------------------
# Forward (GPU)
# ---------------------------------------------------------------------------

def make(kind, M, N, K, seed, bias=True, residual=True):
    """Host operands and their fp64 values."""
    gen = torch.Generator().manual_seed(seed)
    t = F16 if kind == "f16" else BF16
    x = torch.randn(M, K, generator=gen)
    w = torch.randn(N, K, generator=gen) * K ** -0.5
    xs = ws = None
    if kind in ("row", "mx"):
        (x, xs), (w, ws) = R.quantise(x, kind), R.quantise(w, kind)
        xv, wv = R.dequantise(x, xs), R.dequantise(w, ws)
    else:
        x, w = x.to(t), w.to(t)
        xv, wv = R.d(x), R.d(w)
    b = R.normal(gen, N, dtype=t) if bias else None
    r = R.normal(gen, M, N, dtype=t) if residual else None
    return dict(x=x, weight=w, bias=b, residual=r, x_scales=xs, weight_scales=ws), xv, wv, t


def check_forward(o, z, ops, xv, wv, t, activation, kind):
    b, r = R.d(ops["bias"]), R.d(ops["residual"])
    want, wz = R.linear(xv, wv, b, activation, r)
    K = xv.shape[1]
    size = xv.abs() @ wv.abs().t()
    dz = size * additions(K, 128 if kind in ("row", "mx") else 32) * STEP
    if kind in ("row", "mx"):
        dz = dz + dropped(xv, wv)
    if kind == "row":
        dz = dz + size * 4 * STEP
    if b is not None:
        dz = dz + (size + b.abs()) * STEP
    a = wz.abs()
    tol = dz
    if activation == "gelu":
        tol = 1.13 * dz + a * R.tail(a) * (1e-5 + (4 + a * a) * 2.0 ** -21) + want.abs() * 2 * STEP + a * 2 * STEP
    elif activation == "silu":
        tol = 1.1 * dz + R.act(wz, "silu").abs() * (4 + a) * 2.0 ** -21
    if r is not None:
        tol = tol + (R.act(wz, activation).abs() + r.abs() + tol) * STEP
    R.assert_within(o, want, tol + R.rounding(want.abs() + tol, t), "out")
    if z is not None:
        R.assert_within(z, wz, dz + R.rounding(a + dz, t), "z")


def run_forward(device, kind, M, N, K, seed, activation="none", bias=True, residual=True, launch=None,
                place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import linear as L
    ops, xv, wv, t = make(kind, M, N, K, seed, bias, residual)
    up = {k: None if v is None else place(v, device) for k, v in ops.items()}
    out, z = torch.empty(M, N, dtype=t, device=device), torch.empty(M, N, dtype=t, device=device)
    L.mhc_linear_fwd(up["x"], up["weight"], out, bias=up["bias"], residual=up["residual"], x_scales=up["x_scales"],
                     weight_scales=up["weight_scales"], activation=activation, z=z, launch=launch)
    torch.cuda.synchronize()
    check_forward(out, z, ops, xv, wv, t, activation, kind)
    return out


DEPTHS = [1, 7, 8, 16, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 160, 200, 256, 520, 1279, 2048]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
@pytest.mark.parametrize("kernel", [ROWS, NARROW, SMALL, MEDIUM, LARGE])
def test_forward_depths(device, kernel, kind):
    """Every length of the sum around the tiles' borders, on every kernel."""
    M, N = (5, 40) if kernel == ROWS else (70, 72) if kernel in (NARROW, SMALL) else (140, 264)
    for k, K in enumerate(DEPTHS):
        say(f"forward {kind} kernel={kernel} K={K}")
        run_forward(device, kind, M, N, K, seed=k, launch={"kernel": kernel})


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ROWS, NARROW, SMALL, MEDIUM, LARGE])
def test_forward_block_scales(device, kernel):
    """Scales that differ from block to block by up to 2^16, over one to nine passes of the tiles and in parts."""
    from hyper_connection_residual_mhc_amd import linear as L
    M, N = (7, 40) if kernel == ROWS else (300, 290)
    for passes in range(1, 10):
        for splits in (1,) if kernel == ROWS or passes < 4 else (1, 2):
            K = 128 * passes
            say(f"block scales kernel={kernel} K={K} splits={splits}")
            gen = torch.Generator().manual_seed(passes)
            x, w = (torch.randn(r, K, generator=gen).to(torch.float8_e4m3fn) for r in (M, N))
            xs, ws = (torch.randint(119, 136, (r, K // 32), generator=gen, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                      for r in (M, N))
            out, z = torch.empty(M, N, dtype=BF16, device=device), torch.empty(M, N, dtype=BF16, device=device)
            L.mhc_linear_fwd(x.to(device), w.to(device), out, x_scales=xs.to(device), weight_scales=ws.to(device), z=z,
                             launch={"kernel": kernel, "splits": splits})
            torch.cuda.synchronize()
            check_forward(out, z, dict(bias=None, residual=None), R.dequantise(x, xs), R.dequantise(w, ws), BF16, "none", "mx")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx"])
@pytest.mark.parametrize("kernel", [NARROW, SMALL, MEDIUM, LARGE])
def test_forward_tiles(device, kernel, kind):
    """Rows and columns around the tiles' borders, and tiles in every place of the grid."""
    bm, bn = {NARROW: (64, 32), SMALL: (64, 64), MEDIUM: (128, 128), LARGE: (256, 256)}[kernel]
    for k, (M, N) in enumerate(((1, 1), (bm - 1, bn - 1), (bm, bn), (bm + 1, bn + 1), (bm + 17, 3 * bn - 9),
                                (5 * bm + 3, 2 * bn), (9 * bm, bn + 7))):
        say(f"forward {kind} kernel={kernel} M={M} N={N}")
        run_forward(device, kind, M, N, 192, seed=k, launch={"kernel": kernel, "splits": 1})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
def test_forward_rows(device, kind):
    """One to seventeen rows, odd widths."""
    for M in (1, 2, 3, 8, 15, 16, 17):
        for N, K in ((1, 300), (7, 4100), (16, 640), (100, 64), (1001, 1279)):
            say(f"forward {kind} M={M} N={N} K={K}")
            run_forward(device, kind, M, N, K, seed=M + N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
@pytest.mark.parametrize("splits", [2, 3, 7, 64])
def test_forward_splits(device, splits, kind):
    for kernel, M, N in ((NARROW, 70, 24), (SMALL, 65, 130), (MEDIUM, 100, 136), (LARGE, 257, 300)):
        for K in (128, 1000, 2304):
            say(f"forward {kind} kernel={kernel} splits={splits} K={K}")
            run_forward(device, kind, M, N, K, seed=splits, activation="silu", launch={"kernel": kernel, "splits": splits})


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "row"])
def test_forward_epilogues(device, kind, activation):
    for M, N in ((3, 50), (128, 128), (150, 200)):
        for bias in (False, True):
            for residual in (False, True):
                run_forward(device, kind, M, N, 256, 11, activation, bias, residual)
                run_forward(device, kind, M, N, 256, 12, activation, bias, residual, launch={"kernel": 0, "splits": 2}
                            if M > 16 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
def test_forward_alignment_and_edges(device, kind):
    """Operands one element past alignment give the same bytes (the sums' order is the same); nothing outside out,
    z and the workspace is written."""
    from hyper_connection_residual_mhc_amd import linear as L
    for M, N, K in ((3, 40, 256), (70, 72, 256), (300, 264, 512), (129, 1001, 1279)):
        ops, *_, t = make(kind, M, N, K, 5)
        up = {k: None if v is None else v.to(device) for k, v in ops.items()}
        want = L.linear(**{**up, "bias": up["bias"]}, activation="relu", return_z=True)
        moved = {k: None if v is None else R.shifted(v, device) for k, v in ops.items()}
        got = L.linear(**moved, activation="relu", return_z=True)
        assert R.same_bytes(got.out, want.out) and R.same_bytes(got.z, want.z)
        for fill in (0xA5, 0x3C):
            out, z = R.Guarded((M, N), t, device, fill), R.Guarded((M, N), t, device, fill)
            need = L.mhc_linear_fwd_workspace_bytes(M, N, K, ABI[kind])
            ws = R.Guarded((max(need, 1),), torch.uint8, device, fill)
            L.mhc_linear_fwd(up["x"], up["weight"], out.t, bias=up["bias"], residual=up["residual"],
                             x_scales=up["x_scales"], weight_scales=up["weight_scales"], activation="relu", z=z.t,
                             workspace=ws.t)
            assert out.untouched() and z.untouched() and ws.untouched()
            assert R.same_bytes(out.t, want.out) and R.same_bytes(z.t, want.z)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
@pytest.mark.parametrize("M,N,K", [(1100, 1300, 1600 - 7), (2050, 700, 1999), (600, 1801, 2000 + 24),
                                   (2050, 1700, 1999), (1100, 3001, 2024)])
def test_forward_rows_that_are_no_whole_pieces(device, kind, M, N, K):
    """Products long enough for their operands to be copied into whole rows first; fp64 on the GPU. The workspace
    is larger than a call without copies needs, and nothing outside it is written."""
    from hyper_connection_residual_mhc_amd import linear as L
    say(f"forward {kind} M={M} N={N} K={K}")
    ops, xv, wv, t = make(kind, M, N, K, seed=M, residual=False)
    up = {k: None if v is None else v.to(device) for k, v in ops.items()}
    out = R.Guarded((M, N), t, device)
    ws = R.Guarded((L.mhc_linear_fwd_workspace_bytes(M, N, K, ABI[kind]),), torch.uint8, device, 0xFF)
    L.mhc_linear_fwd(up["x"], up["weight"], out.t, bias=up["bias"], x_scales=up["x_scales"],
                     weight_scales=up["weight_scales"], workspace=ws.t)
    assert out.untouched() and ws.untouched()
    x, w, b = (v.to(device) for v in (xv, wv, R.d(ops["bias"])))
    want, size = x @ w.t() + b, x.abs() @ w.abs().t() + b.abs()
    tol = size * (additions(K, 128 if kind in ("row", "mx") else 32) + 6) * STEP
    if kind in ("row", "mx"):
        tol = tol + size * 7 * 2.0 ** -13                  # at most the largest product of each 8, so at most their sum
    tol = tol + (want.abs() + tol) * R.HALF_STEP[t] + R.HALF_TINY[t]
    over = (out.t.double() - want).abs() - tol
    assert float(over.max()) <= 0, int((over > 0).sum())


@pytest.mark.gpu
def test_rows_do_not_depend_on_the_batch(device):
    """With a named tile kernel and one part a row's bytes are the same whatever M is and where it stands."""
    from hyper_connection_residual_mhc_amd import linear as L
    for kind in ("bf16", "mx"):
        for kernel in (SMALL, MEDIUM, LARGE):
            ops, *_ = make(kind, 300, 136, 1000, 6, residual=False)
            up = {k: None if v is None else v.to(device) for k, v in ops.items()}
            launch = {"kernel": kernel, "splits": 1}

            def run(rows):
                out = torch.empty(len(rows), 136, dtype=BF16, device=device)
                xs = up["x_scales"]
                L.mhc_linear_fwd(up["x"].view(torch.uint8 if kind == "mx" else BF16)[rows].contiguous().view(up["x"].dtype),
                                 up["weight"], out, bias=up["bias"],
                                 x_scales=None if xs is None else xs.view(torch.uint8)[rows].contiguous().view(xs.dtype),
                                 weight_scales=up["weight_scales"], launch=launch)
                return out

            everything = run(list(range(300)))
            for rows in ([0], [299], [5, 150, 77], list(range(100, 229))):
                assert R.same_bytes(run(rows), everything[rows])


@pytest.mark.gpu
def test_forward_nothing_and_extremes(device):
    from hyper_connection_residual_mhc_amd import linear as L
    w = torch.randn(40, 64).to(BF16).to(device)
    assert L.linear(torch.empty(0, 64, dtype=BF16, device=device), w).out.shape == (0, 40)
    for M in (4, 130):
        x = torch.ones(M, 64, dtype=BF16)
        x[1, 3], x[2, 5] = float("inf"), float("nan")
        o = L.linear(x.to(device), w.abs()).out.cpu()
        assert torch.isinf(o[1]).all() and torch.isnan(o[2]).all()
        assert torch.isfinite(o[0]).all() and torch.isfinite(o[3:]).all()
        # infinite sums through the activations: gelu and relu of +-inf are inf and 0
        eye = torch.eye(64, dtype=BF16, device=device)
        y = torch.zeros(M, 64, dtype=BF16)
        y[:, 0], y[:, 1], y[:, 2], y[:, 3] = 3e38, -3e38, 60.0, -60.0
        for name in ("relu", "gelu", "silu"):
            o = L.linear(y.to(device), eye, activation=name).out.cpu()
            assert (o[:, 0] == y[:, 0]).all() and (o[:, 1] == 0).all(), name
            assert (o[:, 2] == 60).all() and (o[:, 3].abs() < 1e-20).all(), name


@pytest.mark.gpu
def test_forward_long_rows(device):
    """Operands past 2^32 bytes: the last rows of a weight of 4.3 GB, and of an x and out as long."""
    from hyper_connection_residual_mhc_amd import linear as L
    K = 4096
    N = (1 << 19) + 64
    gen = torch.Generator().manual_seed(1)
    tailw = R.normal(gen, 64, K)
    w = torch.zeros(N, K, dtype=BF16, device=device)
    w[-64:] = tailw.to(device)
    for M in (2, 64):
        x = R.normal(gen, M, K)
        o = L.linear(x.to(device), w).out
        want = R.d(x) @ R.d(tailw).t()
        size = R.d(x).abs() @ R.d(tailw).abs().t()
        tol = size * additions(K, 32) * STEP
        R.assert_within(o[:, -64:], want, tol + R.rounding(want.abs() + tol, BF16), "last columns")
        assert not o[:, :-64].any()
        o = L.linear(w, x.to(device)).out
        want, size = want.t(), size.t()
        tol = size * additions(K, 32) * STEP
        R.assert_within(o[-64:], want, tol + R.rounding(want.abs() + tol, BF16), "last rows")
        assert not o[:-64].any()


# ---------------------------------------------------------------------------
# Backward (GPU)
# ---------------------------------------------------------------------------

def check_backward(device, kind, M, N, K, activation, seed, bias=True, place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import linear as L
    ops, xv, wv, t = make(kind, M, N, K, seed, bias, False)
    gen = torch.Generator().manual_seed(seed + 1)
    g = R.normal(gen, M, N, dtype=t)
    z = R.linear(xv, wv, R.d(ops["bias"]))[1].to(t)
    gx, gw, gb = L.linear_backward(place(g, device), place(ops["x"], device), place(ops["weight"], device),
                                   activation=activation, z=None if activation == "none" else place(z, device), bias=bias)
    torch.cuda.synchronize()
    zv = R.d(z)
    wx, ww, wb, gz = R.linear_grads(R.d(g), xv, wv, zv, activation)
    # gz: the slope (its parts are good to 2^-21 and the fitted tail to 1e-5), a product, a rounding to 16 bits
    dslope = 0.0 if activation in ("none", "relu") else 1e-5 + (4 + zv.abs()) * 2.0 ** -20
    dg = torch.zeros_like(gz) if activation == "none" else R.d(g).abs() * dslope + gz.abs() * 2 * STEP
    dr = dg if activation in ("none", "relu") else dg + R.rounding(gz.abs() + dg, t)
    ax = gz.abs() + dr
    tol = dr @ wv.abs() + (ax @ wv.abs()) * additions(N, 32) * STEP
    R.assert_within(gx, wx, tol + R.rounding(wx.abs() + tol, t), "grad_x")
    tol = dr.t() @ xv.abs() + (ax.t() @ xv.abs()) * additions(M, 32) * STEP
    R.assert_within(gw, ww, tol + R.rounding(ww.abs() + tol, t), "grad_weight")
    if bias:
        rows = max(32, math.ceil(M / 256))
        tol = dg.sum(0) + ax.sum(0) * (math.ceil(rows / 4) + 4 + math.ceil(M / rows)) * STEP
        R.assert_within(gb, wb, tol + R.rounding(wb.abs() + tol, t), "grad_bias")
    else:
        assert gb is None
    return gx, gw, gb


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
def test_backward_sizes(device, kind, activation):
    for k, (M, N, K) in enumerate(((1, 1, 1), (1, 64, 40), (3, 7, 9), (16, 17, 33), (64, 64, 64), (65, 130, 31),
                                   (129, 100, 257), (300, 520, 200), (2, 1001, 1279), (700, 24, 600))):
        say(f"backward {kind} {activation} M={M} N={N} K={K}")
        check_backward(device, kind, M, N, K, activation, seed=k, bias=k % 3 != 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3800, 3704, 3528), (3801, 3704, 3592), (2100, 2050, 1000), (130, 1024, 3000), (1500, 801, 1001), (900, 1024, 1003), (1031, 1025, 1024),
                                   (3800, 3701, 3525)])
@pytest.mark.parametrize("activation", ["none", "relu"])
def test_backward_large_tiles(device, M, N, K, activation):
    """Sizes at which the products take the large and the middling tiles, with ragged edges and with rows that are
    copied first; fp64 on the GPU."""
    from hyper_connection_residual_mhc_amd import linear as L
    say(f"backward M={M} N={N} K={K} {activation}")
    gen = torch.Generator(device=device).manual_seed(M)
    g, x, w = (torch.randn(s, device=device, generator=gen).to(BF16) for s in ((M, N), (M, K), (N, K)))
    z = torch.randn((M, N), device=device, generator=gen).to(BF16)
    gx, gw, gb = L.linear_backward(g, x, w, bias=True, activation=activation, z=z)
    if activation == "relu":
        g = torch.where(z > 0, g, torch.zeros_like(g))     # exact: the slope is 0 or 1
    for got, want, size, length in ((gx, g.double() @ w.double(), g.double().abs() @ w.double().abs(), N),
                                    (gw, g.double().t() @ x.double(), g.double().abs().t() @ x.double().abs(), M)):
        tol = size * additions(length, 32) * STEP
        tol = tol + (want.abs() + tol) * R.HALF_STEP[BF16] + R.HALF_TINY[BF16]
        over = (got.double() - want).abs() - tol
        assert float(over.max()) <= 0, int((over > 0).sum())
    want = g.double().sum(0)
    rows = max(32, math.ceil(M / 256))
    tol = g.double().abs().sum(0) * (math.ceil(rows / 4) + 4 + math.ceil(M / rows)) * STEP
    assert float(((gb.double() - want).abs() - tol - (want.abs() + tol) * R.HALF_STEP[BF16]).max()) <= 0


@pytest.mark.gpu
def test_backward_nothing(device):
    from hyper_connection_residual_mhc_amd import linear as L
    x, w = torch.empty(0, 24, dtype=BF16, device=device), torch.ones(40, 24, dtype=BF16, device=device)
    g = torch.empty(0, 40, dtype=BF16, device=device)
    gw, gb = R.Guarded((40, 24), BF16, device), R.Guarded((40,), BF16, device)
    L.mhc_linear_bwd(g, x, w, grad_x=torch.empty_like(x), grad_weight=gw.t, grad_bias=gb.t, activation="gelu", z=g)
    assert gw.untouched() and gb.untouched() and not gw.t.any() and not gb.t.any()


@pytest.mark.gpu
def test_backward_alignment_and_edges(device):
    from hyper_connection_residual_mhc_amd import linear as L
    for M, N, K in ((70, 72, 80), (33, 1001, 129)):
        a = check_backward(device, "bf16", M, N, K, "silu", seed=3)
        b = check_backward(device, "bf16", M, N, K, "silu", seed=3, place=R.shifted)
        for p, q in zip(a, b):
            assert R.same_bytes(p, q)
        gen = torch.Generator().manual_seed(1)
        g, z, x, w = (R.normal(gen, *s).to(device) for s in ((M, N), (M, N), (M, K), (N, K)))
        outs = [R.Guarded(s, BF16, device) for s in ((M, K), (N, K), (N,))]
        ws = R.Guarded((L.mhc_linear_bwd_workspace_bytes(M, N, K, 1),), torch.uint8, device)
        L.mhc_linear_bwd(g, x, w, grad_x=outs[0].t, grad_weight=outs[1].t, grad_bias=outs[2].t, activation="silu", z=z,
                         workspace=ws.t)
        want = L.linear_backward(g, x, w, activation="silu", z=z, bias=True)
        assert ws.untouched()
        for o, q in zip(outs, want):
            assert o.untouched() and R.same_bytes(o.t, q)
        # each gradient alone
        for k in range(3):
            one = [torch.empty_like(q) if i == k else None for i, q in enumerate(want)]
            L.mhc_linear_bwd(g, x, w, grad_x=one[0], grad_weight=one[1], grad_bias=one[2], activation="silu", z=z)
            assert R.same_bytes(one[k], want[k])


@pytest.mark.gpu
def test_autograd_streams_and_graphs(device):
    from hyper_connection_residual_mhc_amd import linear as L
    gen = torch.Generator().manual_seed(2)
    M, N, K = 150, 264, 320
    x, w, b, r, g = (R.normal(gen, *s).to(device) for s in ((M, K), (N, K), (N,), (M, N), (M, N)))

    def both(x):
        o = L.linear(x, w, b, activation="gelu", residual=r, return_z=True)
        return (o.out, *L.linear_backward(g, x, w, activation="gelu", z=o.z, bias=True))

    want = both(x)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    out = L.linear_autograd(leaves[0], leaves[1], leaves[2], activation="gelu", residual=leaves[3])
    got = torch.autograd.grad(out, leaves, g)
    for p, q in zip((out, *got), (*want, g)):
        assert R.same_bytes(p, q)
    out = L.linear_autograd(x, leaves[1], activation="none")
    gw, = torch.autograd.grad(out, leaves[1], g)
    assert R.same_bytes(gw, L.linear_backward(g, x, w)[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bufs = [torch.empty_like(t) for t in (*want, r)]
    L.mhc_linear_fwd(x, w, bufs[0], bias=b, activation="gelu", residual=r, z=bufs[4], stream=side)
    L.mhc_linear_bwd(g, x, w, grad_x=bufs[1], grad_weight=bufs[2], grad_bias=bufs[3], activation="gelu", z=bufs[4],
                     stream=side)
    side.synchronize()
    for p, q in zip(bufs, want):
        assert R.same_bytes(p, q)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(buf)
        small = L.linear(buf[:4], w, b).out
    for k in range(4):
        new = (x * (k + 1)).contiguous()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((*got, small), (*both(new), L.linear(new[:4], w, b).out)):
            assert R.same_bytes(p, q), k
