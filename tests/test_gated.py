"""The gated feed-forward block (include/mhc_gated.h) against its fp64 form,
forward and backward, and the rules of the call.

Tolerances. Each projection is a sum as in test_linear.py, and off by no more
(`projection`). The activation and its error are those of that file too
(`act_error`, `slope_error`). out is one product of the two values: with errors
da and du of its factors it is off by |u| da + |a| du + da du and one rounding
to fp32, then by half a step of its type. In the backward a product or two of
fp32 (half a step each) stand in front of the rounding to 16 bits, which the
products over it see in full; grad_x sums over both blocks.
"""

from __future__ import annotations

import math

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from hyper_connection_residual_mhc_amd import _lib
from hyper_connection_residual_mhc_amd._lib import (MHC_ERROR_ALIASING, MHC_ERROR_INVALID_VALUE,
                                                    MHC_SUCCESS)
from test_linear import LARGE, MEDIUM, NARROW, ROWS, SMALL, STEP, additions, dropped

BF16, F16 = torch.bfloat16, torch.float16
ABI = {"bf16": 1, "f16": 2, "row": 3, "mx": 4, "int8": 6}
EIGHT = ("row", "mx", "int8")


def quantise_int8(v):
    s = (v.abs().amax(1) / 127).clamp_min(2.0 ** -126)
    return (v / s[:, None]).round().to(torch.int8), s


def act_error(z, dz, name):
    """How far act(z) may be off where z is off by dz."""
    a = z.abs()
    if name == "gelu":
        return 1.13 * dz + a * R.tail(a) * (1e-5 + (4 + a * a) * 2.0 ** -21) + R.act(z, name).abs() * 2 * STEP + a * 2 * STEP
    if name == "silu":
        return 1.1 * dz + R.act(z, name).abs() * (4 + a) * 2.0 ** -21
    return dz


def slope_error(z, name):
    return torch.zeros_like(z) if name in ("none", "relu") else 1e-5 + (4 + z.abs()) * 2.0 ** -20


def gated(x, wg, wu, bg, bu, name):
    """(out, gate, up), all fp64."""
    g, u = x @ wg.t(), x @ wu.t()
    g, u = (g if bg is None else g + bg), (u if bu is None else u + bu)
    return R.act(g, name) * u, g, u


def gated_grads(d, x, wg, wu, g, u, name):
    """(grad_x, grad_wg, grad_wu, grad_bg, grad_bu, dg, du) without the rounding of dg and du."""
    dg, du = d * u * R.act_slope(g, name), d * R.act(g, name)
    return dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, dg.sum(0), du.sum(0), dg, du


# ---------------------------------------------------------------------------
# The fp64 form itself, and host rules (CPU)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_formula_gradients_are_the_differences_of_the_forward(name):
    gen = torch.Generator().manual_seed(4)
    M, N, K = 3, 4, 5
    x, wg, wu, bg, bu, d = (torch.randn(s, generator=gen, dtype=torch.float64)
                            for s in ((M, K), (N, K), (N, K), (N,), (N,), (M, N)))

    def loss():
        return (gated(x, wg, wu, bg, bu, name)[0] * d).sum()

    _, g, u = gated(x, wg, wu, bg, bu, name)
    assert g.abs().min() > 1e-3                            # no kink of relu within a step
    for leaf, grad in zip((x, wg, wu, bg, bu), gated_grads(d, x, wg, wu, g, u, name)):
        assert torch.allclose(grad, R.differences(loss, leaf), rtol=0, atol=1e-7)


BASE = 1 << 36
GAP = 1 << 31


@pytest.fixture(scope="module")
def lib(built_library):
    return _lib.gated_lib()


def fwd_args(**kw):
    a = dict(x=BASE, xs=None, wg=BASE + GAP, gs=None, wu=BASE + 2 * GAP, us=None, bg=None, bu=None, out=BASE + 3 * GAP,
             gate=None, up=None, workspace=BASE + 4 * GAP, workspace_bytes=1 << 30, M=20, N=40, K=50, dtype=1, act=2,
             launch=None)
    a.update(kw)
    return list(a.values())


SCALES = dict(xs=BASE + 5 * GAP, gs=BASE + 6 * GAP, us=BASE + 7 * GAP)


@pytest.mark.parametrize("kw", [
    {}, {"dtype": 2}, {"bg": BASE + 8 * GAP, "bu": BASE + 9 * GAP}, {"bu": BASE + 9 * GAP, "act": 0},
    {"gate": BASE + 8 * GAP, "up": BASE + 9 * GAP, "act": 3}, {"up": BASE + 9 * GAP}, {"dtype": 3, **SCALES},
    {"dtype": 4, **SCALES}, {"dtype": 6, **SCALES}, {"dtype": 6, **SCALES, "K": 131071, "M": 1},
    {"M": 0, "x": None, "wg": None, "wu": None, "out": None}, {"M": 1, "N": 1, "K": 1, "workspace": None, "workspace_bytes": 0},
])
def test_valid_forward_arguments(lib, kw):
    assert lib.mhc_gated_validate_fwd(*fwd_args(**kw)) == MHC_SUCCESS, lib.mhc_gated_last_error_message()


@pytest.mark.parametrize("kw", [
    {"M": -1}, {"M": 1 << 31}, {"N": 0}, {"N": 1 << 30}, {"K": 0}, {"K": (1 << 21) + 1}, {"dtype": 0}, {"dtype": 5},
    {"dtype": 7}, {"act": -1}, {"act": 4}, {"x": None}, {"wg": None}, {"wu": None}, {"out": None}, {"wu": BASE + 2 * GAP + 1},
    {"out": BASE + 3 * GAP + 1}, {"bg": BASE + 8 * GAP + 1}, {"dtype": 3}, {"dtype": 3, **SCALES, "us": None},
    {"dtype": 4, **SCALES, "gs": None}, {"dtype": 6, **SCALES, "xs": BASE + 5 * GAP + 2}, {**SCALES}, {"us": BASE + 7 * GAP},
    {"dtype": 6, **SCALES, "K": 131072}, {"M": 1 << 30, "N": 1 << 29}, {"M": 64, "K": 4096, "workspace_bytes": 0},
    {"M": 64, "K": 4096, "workspace": None}, {"gate": BASE + 8 * GAP + 1},
])
def test_refused_forward_arguments(lib, kw):
    assert lib.mhc_gated_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_INVALID_VALUE
    assert lib.mhc_gated_last_error_message() != b""


@pytest.mark.parametrize("kw", [
    {"out": BASE}, {"out": BASE + 2 * GAP}, {"gate": BASE + 3 * GAP}, {"up": BASE + GAP}, {"bg": BASE + 3 * GAP},
    {"gate": BASE + 8 * GAP, "up": BASE + 8 * GAP}, {"dtype": 6, **SCALES, "us": BASE + 3 * GAP},
    {"M": 64, "K": 4096, "workspace": BASE + 2 * GAP},
])
def test_overlapping_forward_arguments(lib, kw):
    assert lib.mhc_gated_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_ALIASING


def test_launches(lib):
    from hyper_connection_residual_mhc_amd import gated as G
    for launch in ({"kernel": NARROW}, {"kernel": 6}, {"splits": 65}, {"kernel": ROWS, "splits": 2}):
        with pytest.raises(_lib.MhcError):
            G.mhc_gated_plan(8, 64, 64, 1, launch)
        with pytest.raises(ValueError):
            G.mhc_gated_fwd_workspace_bytes(8, 64, 64, 1, launch)
    with pytest.raises(_lib.MhcError):
        G.mhc_gated_plan(17, 64, 64, 1, {"kernel": ROWS})
    assert G.mhc_gated_plan(16, 4096, 4096, 1) == {"kernel": ROWS, "splits": 1}
    assert G.mhc_gated_plan(100, 8, 64, 1)["kernel"] not in (NARROW, ROWS)  # there is no narrow form
    assert G.mhc_gated_plan(4096, 8192, 4096, 1) == {"kernel": LARGE, "splits": 1}
    for kernel in (SMALL, MEDIUM, LARGE):
        p = G.mhc_gated_plan(100, 50, 4096, 1, {"kernel": kernel, "splits": 3})
        assert p == {"kernel": kernel, "splits": 3}
        assert G.mhc_gated_fwd_workspace_bytes(100, 50, 4096, 1, p) == -(-100 * 100 * 4 * 3 // 256) * 256


def bwd_args(**kw):
    a = dict(d=BASE, x=BASE + GAP, wg=BASE + 2 * GAP, wu=BASE + 3 * GAP, gate=BASE + 4 * GAP, up=BASE + 5 * GAP,
             gx=BASE + 6 * GAP, ggw=BASE + 7 * GAP, guw=BASE + 8 * GAP, ggb=BASE + 9 * GAP, gub=BASE + 10 * GAP,
             workspace=BASE + 11 * GAP, workspace_bytes=1 << 30, M=20, N=40, K=50, dtype=1, act=2)
    a.update(kw)
    return list(a.values())


def test_backward_arguments(lib):
    v = lib.mhc_gated_validate_bwd
    for kw in ({}, {"act": 0}, {"gx": None}, {"ggw": None, "guw": None}, {"ggb": None}, {"gub": None},
               {"gx": None, "ggw": None, "guw": None, "ggb": None, "gub": None}, {"N": 1 << 20, "M": 1},
               {"M": 0, "d": None, "x": None, "wg": None, "wu": None, "gate": None, "up": None, "workspace": None,
                "workspace_bytes": 0}):
        assert v(*bwd_args(**kw)) == MHC_SUCCESS, kw
    for kw in ({"gate": None}, {"up": None}, {"dtype": 3}, {"dtype": 6}, {"M": -1}, {"N": 0}, {"K": 0}, {"M": (1 << 21) + 1},
               {"N": (1 << 20) + 1}, {"act": 9}, {"x": None}, {"workspace_bytes": 100}, {"workspace": None}, {"ggw": None},
               {"guw": None}, {"workspace": BASE + 11 * GAP + 8}, {"guw": BASE + 8 * GAP + 1}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
    for kw in ({"gx": BASE}, {"gx": BASE + 7 * GAP}, {"gub": BASE + 5 * GAP}, {"workspace": BASE + GAP}, {"guw": BASE + 7 * GAP}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_ALIASING, kw
    assert lib.mhc_gated_bwd_workspace_bytes(0, 5, 5, 1) == 0
    assert lib.mhc_gated_bwd_workspace_bytes(5, 5, 5, 3) == -1


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import gated as G
    x, w = torch.zeros(2, 8, dtype=BF16), torch.zeros(4, 8, dtype=BF16)
    with pytest.raises(TypeError):
        G.gated(x, w, w)                                   # not on a GPU
    with pytest.raises(TypeError):
        G.gated(x.float(), w.float(), w.float())
    with pytest.raises(ValueError):
        G.gated(x[0], w, w)
    with pytest.raises(ValueError):
        G.gated(x, w, w, x_scales=torch.ones(2))


# ---------------------------------------------------------------------------
# Forward (GPU)
# ---------------------------------------------------------------------------

def make(kind, M, N, K, seed, bias=True):
    """Host operands and their fp64 values."""
    gen = torch.Generator().manual_seed(seed)
    t = F16 if kind == "f16" else BF16
    raw = [torch.randn(M, K, generator=gen), *(torch.randn(N, K, generator=gen) * K ** -0.5 for _ in range(2))]
    if kind in EIGHT:
        pairs = [quantise_int8(v) if kind == "int8" else R.quantise(v, kind) for v in raw]
        values = [R.dequantise(*p) for p in pairs]
    else:
        pairs = [(v.to(t), None) for v in raw]
        values = [R.d(v) for v, _ in pairs]
    bg, bu = ((R.normal(gen, N, dtype=t) for _ in range(2)) if bias else (None, None))
    ops = dict(x=pairs[0][0], gate_weight=pairs[1][0], up_weight=pairs[2][0], gate_bias=bg, up_bias=bu,
               x_scales=pairs[0][1], gate_scales=pairs[1][1], up_scales=pairs[2][1])
    return ops, values, t


def projection(xv, wv, b, kind):
    """(z, how far it may be off)."""
    K = xv.shape[1]
    z, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if kind == "int8":
        dz = z.abs() * 2 * STEP                            # the exact sum's rounding, the scales' product, the product with it
    else:
        dz = size * additions(K, 128 if kind in EIGHT else 32) * STEP
    if kind in ("row", "mx"):
        dz = dz + dropped(xv, wv)
    if kind == "row":
        dz = dz + size * 4 * STEP
    if b is not None:
        dz = dz + (size + b.abs()) * STEP
        z = z + b
    return z, dz


def check_forward(o, gate, up, ops, values, t, activation, kind):
    xv, wg, wu = values
    g, dg = projection(xv, wg, R.d(ops["gate_bias"]), kind)
    u, du = projection(xv, wu, R.d(ops["up_bias"]), kind)
    a, da = R.act(g, activation), act_error(g, dg, activation)
    want = a * u
    tol = u.abs() * da + a.abs() * du + da * du + want.abs() * STEP
    R.assert_within(o, want, tol + R.rounding(want.abs() + tol, t), "out")
    for got, z, dz, name in ((gate, g, dg, "gate"), (up, u, du, "up")):
        if got is not None:
            R.assert_within(got, z, dz + R.rounding(z.abs() + dz, t), name)


def run_forward(device, kind, M, N, K, seed, activation="silu", bias=True, launch=None, z=True,
                place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import gated as G
    ops, values, t = make(kind, M, N, K, seed, bias)
    up = {k: None if v is None else place(v, device) for k, v in ops.items()}
    out, gate, upv = (torch.empty(M, N, dtype=t, device=device) for _ in range(3))
    G.mhc_gated_fwd(up["x"], up["gate_weight"], up["up_weight"], out, gate_bias=up["gate_bias"], up_bias=up["up_bias"],
                    x_scales=up["x_scales"], gate_scales=up["gate_scales"], up_scales=up["up_scales"],
                    activation=activation, gate=gate if z else None, up=upv if z else None, launch=launch)
    torch.cuda.synchronize()
    check_forward(out, gate if z else None, upv if z else None, ops, values, t, activation, kind)
    return out


DEPTHS = [1, 7, 8, 16, 31, 33, 63, 64, 65, 127, 128, 129, 200, 256, 520, 1279, 2048]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx", "int8"])
@pytest.mark.parametrize("kernel", [ROWS, SMALL, MEDIUM, LARGE])
def test_forward_depths(device, kernel, kind):
    M, N = (5, 20) if kernel == ROWS else (70, 36) if kernel == SMALL else (140, 132)
    for k, K in enumerate(DEPTHS):
        say(f"gated {kind} kernel={kernel} K={K}")
        run_forward(device, kind, M, N, K, seed=k, launch={"kernel": kernel})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx", "int8"])
@pytest.mark.parametrize("kernel", [SMALL, MEDIUM, LARGE])
def test_forward_tiles(device, kernel, kind):
    """Rows and columns around the tiles' borders, and tiles in every place of the grid."""
    bm, bn = {SMALL: (64, 32), MEDIUM: (128, 64), LARGE: (256, 128)}[kernel]
    for k, (M, N) in enumerate(((1, 1), (bm - 1, bn - 1), (bm, bn), (bm + 1, bn + 1), (bm + 17, 3 * bn - 9),
                                (5 * bm + 3, 2 * bn), (9 * bm, bn + 7))):
        say(f"gated {kind} kernel={kernel} M={M} N={N}")
        run_forward(device, kind, M, N, 256, seed=k, launch={"kernel": kernel, "splits": 1})


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ROWS, SMALL, MEDIUM, LARGE])
def test_forward_block_scales(device, kernel):
    """Scales that differ from block to block by up to 2^16, over one to nine passes of the tiles and in parts."""
    from hyper_connection_residual_mhc_amd import gated as G
    M, N = (7, 20) if kernel == ROWS else (300, 145)
    for passes in range(1, 10):
        for splits in (1,) if kernel == ROWS or passes < 4 else (1, 2):
            K = 128 * passes
            say(f"gated block scales kernel={kernel} K={K} splits={splits}")
            gen = torch.Generator().manual_seed(passes)
            codes = [torch.randn(r, K, generator=gen).to(torch.float8_e4m3fn) for r in (M, N, N)]
            scales = [torch.randint(119, 136, (r, K // 32), generator=gen, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                      for r in (M, N, N)]
            out, gate, up = (torch.empty(M, N, dtype=BF16, device=device) for _ in range(3))
            c, s = [v.to(device) for v in codes], [v.to(device) for v in scales]
            G.mhc_gated_fwd(*c, out, x_scales=s[0], gate_scales=s[1], up_scales=s[2], gate=gate, up=up, activation="none",
                            launch={"kernel": kernel, "splits": splits})
            torch.cuda.synchronize()
            check_forward(out, gate, up, dict(gate_bias=None, up_bias=None),
                          [R.dequantise(v, q) for v, q in zip(codes, scales)], BF16, "none", "mx")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx", "int8"])
def test_forward_rows(device, kind):
    """One to seventeen rows, odd widths."""
    for M in (1, 2, 8, 15, 16, 17):
        for N, K in ((1, 300), (7, 4100), (16, 640), (100, 64), (1001, 1279)):
            say(f"gated {kind} M={M} N={N} K={K}")
            run_forward(device, kind, M, N, K, seed=M + N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx", "int8"])
@pytest.mark.parametrize("splits", [2, 3, 64])
def test_forward_splits(device, splits, kind):
    for kernel, M, N in ((SMALL, 65, 70), (MEDIUM, 100, 68), (LARGE, 257, 150)):
        for K in (128, 1000, 2304):
            say(f"gated {kind} kernel={kernel} splits={splits} K={K}")
            run_forward(device, kind, M, N, K, seed=splits, launch={"kernel": kernel, "splits": splits})


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "int8"])
def test_forward_epilogues(device, kind, activation):
    for M, N in ((3, 50), (128, 128), (150, 200)):
        for bias in (False, True):
            for z in (False, True):
                run_forward(device, kind, M, N, 256, 11, activation, bias, z=z)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx", "int8"])
def test_forward_alignment_and_edges(device, kind):
    """Operands one element past alignment give the same bytes; nothing outside out, gate, up and the workspace is
    written."""
    from hyper_connection_residual_mhc_amd import gated as G
    for M, N, K in ((3, 40, 256), (70, 72, 256), (300, 264, 512), (129, 1001, 1279)):
        ops, _, t = make(kind, M, N, K, 5)
        at = {k: None if v is None else v.to(device) for k, v in ops.items()}
        want = G.gated(**at, activation="relu", return_z=True)
        moved = {k: None if v is None else R.shifted(v, device) for k, v in ops.items()}
        for p, q in zip(G.gated(**moved, activation="relu", return_z=True), want):
            assert R.same_bytes(p, q)
        for fill in (0xA5, 0x3C):
            outs = [R.Guarded((M, N), t, device, fill) for _ in range(3)]
            ws = R.Guarded((max(G.mhc_gated_fwd_workspace_bytes(M, N, K, ABI[kind]), 1),), torch.uint8, device, fill)
            G.mhc_gated_fwd(at["x"], at["gate_weight"], at["up_weight"], outs[0].t, gate_bias=at["gate_bias"],
                            up_bias=at["up_bias"], x_scales=at["x_scales"], gate_scales=at["gate_scales"],
                            up_scales=at["up_scales"], activation="relu", gate=outs[1].t, up=outs[2].t, workspace=ws.t)
            assert ws.untouched()
            for p, q in zip(outs, want):
                assert p.untouched() and R.same_bytes(p.t, q)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "row", "mx", "int8"])
@pytest.mark.parametrize("M,N,K", [(1100, 900, 1999), (2050, 700, 2024)])
def test_forward_rows_that_are_no_whole_pieces(device, kind, M, N, K):
    """Products long enough for their operands to be copied into whole rows first; fp64 on the GPU."""
    from hyper_connection_residual_mhc_amd import gated as G
    say(f"gated {kind} M={M} N={N} K={K}")
    ops, values, t = make(kind, M, N, K, seed=M)
    at = {k: None if v is None else v.to(device) for k, v in ops.items()}
    out, gate, up = (R.Guarded((M, N), t, device) for _ in range(3))
    ws = R.Guarded((G.mhc_gated_fwd_workspace_bytes(M, N, K, ABI[kind]),), torch.uint8, device, 0xFF)
    G.mhc_gated_fwd(at["x"], at["gate_weight"], at["up_weight"], out.t, gate_bias=at["gate_bias"], up_bias=at["up_bias"],
                    x_scales=at["x_scales"], gate_scales=at["gate_scales"], up_scales=at["up_scales"], activation="none",
                    gate=gate.t, up=up.t, workspace=ws.t)
    assert out.untouched() and ws.untouched() and gate.untouched() and up.untouched()
    x, wg, wu, bg, bu = (v.to(device) for v in (*values, R.d(ops["gate_bias"]), R.d(ops["up_bias"])))
    z, dz = [], []
    for w, b, got in ((wg, bg, gate), (wu, bu, up)):
        want, size = x @ w.t() + b, x.abs() @ w.abs().t() + b.abs()
        tol = size * (additions(K, 128 if kind in EIGHT else 32) + 6) * STEP
        if kind in ("row", "mx"):
            tol = tol + size * 7 * 2.0 ** -13              # at most the largest product of each 8, so at most their sum
        z.append(want)
        dz.append(tol)
        over = (got.t.double() - want).abs() - tol - (want.abs() + tol) * R.HALF_STEP[t] - R.HALF_TINY[t]
        assert float(over.max()) <= 0, int((over > 0).sum())
    want = z[0] * z[1]
    tol = z[1].abs() * dz[0] + z[0].abs() * dz[1] + dz[0] * dz[1] + want.abs() * STEP
    over = (out.t.double() - want).abs() - tol - (want.abs() + tol) * R.HALF_STEP[t] - R.HALF_TINY[t]
    assert float(over.max()) <= 0, int((over > 0).sum())


@pytest.mark.gpu
def test_rows_do_not_depend_on_the_batch(device):
    """With a named tile kernel and one part, and with integers whatever the launch."""
    from hyper_connection_residual_mhc_amd import gated as G
    for kind, launch in (("bf16", {"kernel": SMALL, "splits": 1}), ("bf16", {"kernel": LARGE, "splits": 1}), ("int8", None)):
        ops, *_ = make(kind, 300, 136, 1000, 6)
        at = {k: None if v is None else v.to(device) for k, v in ops.items()}

        def run(rows):
            out = torch.empty(len(rows), 136, dtype=BF16, device=device)
            xs = at["x_scales"]
            G.mhc_gated_fwd(at["x"][rows].contiguous(), at["gate_weight"], at["up_weight"], out, gate_bias=at["gate_bias"],
                            up_bias=at["up_bias"], x_scales=None if xs is None else xs[rows].contiguous(),
                            gate_scales=at["gate_scales"], up_scales=at["up_scales"], launch=launch)
            return out

        everything = run(list(range(300)))
        for rows in ([0], [299], [5, 150, 77], list(range(100, 229))):
            assert R.same_bytes(run(rows), everything[rows])


@pytest.mark.gpu
def test_forward_nothing_and_extremes(device):
    from hyper_connection_residual_mhc_amd import gated as G
    w = torch.ones(40, 64, dtype=BF16, device=device)
    o = G.gated(torch.empty(0, 64, dtype=BF16, device=device), w, w, return_z=True)
    assert o.out.shape == o.gate.shape == o.up.shape == (0, 40)
    for M in (4, 130):
        x = torch.ones(M, 64, dtype=BF16)
        x[1, 3], x[2, 5], x[3, 7] = float("inf"), float("nan"), float("-inf")
        for name in ("none", "relu", "silu", "gelu"):
            o = G.gated(x.to(device), w, w, activation=name).out.cpu()
            assert (o[1] == float("inf")).all() and torch.isnan(o[2]).all()
            assert (o[0] == 64.0 * 64).all() and torch.isfinite(o[4:]).all()
            # act(-inf) * -inf: none inf; relu and gelu 0 * -inf, silu NaN
            assert (o[3] == float("inf")).all() if name == "none" else torch.isnan(o[3]).all()


@pytest.mark.gpu
def test_forward_long_weights(device):
    """Weights past 2^32 bytes: the last rows of two of 4.3 GB."""
    from hyper_connection_residual_mhc_amd import gated as G
    K, N = 4096, (1 << 19) + 64
    gen = torch.Generator().manual_seed(1)
    ends = [R.normal(gen, 64, K, scale=K ** -0.5) for _ in range(2)]
    ws = []
    for e in ends:
        ws.append(torch.zeros(N, K, dtype=BF16, device=device))
        ws[-1][-64:] = e.to(device)
    for M in (2, 64):
        x = R.normal(gen, M, K)
        o = G.gated(x.to(device), *ws, activation="none").out
        (g, dg), (u, du) = (projection(R.d(x), R.d(e), None, "bf16") for e in ends)
        tol = u.abs() * dg + g.abs() * du + dg * du + (g * u).abs() * STEP
        R.assert_within(o[:, -64:], g * u, tol + R.rounding((g * u).abs() + tol, BF16), "last columns")
        assert not o[:, :-64].any()


# ---------------------------------------------------------------------------
# Backward (GPU)
# ---------------------------------------------------------------------------

def backward_tolerances(d, g, u, values, grads, activation, t):
    """How far each of the five gradients may be off, before its own rounding."""
    xv, wg, wu = values
    M, N = d.shape
    *_, dg, du = grads
    eg = (d * u).abs() * slope_error(g, activation) + dg.abs() * 3 * STEP
    eu = d.abs() * act_error(g, torch.zeros_like(g), activation) + du.abs() * 2 * STEP
    rg, ru = eg + R.rounding(dg.abs() + eg, t), eu + R.rounding(du.abs() + eu, t)
    ag, au = dg.abs() + rg, du.abs() + ru
    half = -(-N // 64) * 64
    tx = rg @ wg.abs() + ru @ wu.abs() + (ag @ wg.abs() + au @ wu.abs()) * additions(2 * half, 32) * STEP
    tg = rg.t() @ xv.abs() + (ag.t() @ xv.abs()) * additions(M, 32) * STEP
    tu = ru.t() @ xv.abs() + (au.t() @ xv.abs()) * additions(M, 32) * STEP
    rows = max(32, math.ceil(M / 256))
    long = (math.ceil(rows / 4) + 4 + math.ceil(M / 8)) * STEP
    return tx, tg, tu, eg.sum(0) + ag.sum(0) * long, eu.sum(0) + au.sum(0) * long


def check_backward(device, kind, M, N, K, activation, seed, bias=True, place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import gated as G
    ops, values, t = make(kind, M, N, K, seed, bias)
    gen = torch.Generator().manual_seed(seed + 1)
    d = R.normal(gen, M, N, dtype=t)
    _, g, u = gated(*values, R.d(ops["gate_bias"]), R.d(ops["up_bias"]), activation)
    g, u = g.to(t), u.to(t)
    got = G.gated_backward(*(place(v, device) for v in (d, ops["x"], ops["gate_weight"], ops["up_weight"], g, u)),
                           activation=activation, bias=bias)
    torch.cuda.synchronize()
    dv, gv, uv = R.d(d), R.d(g), R.d(u)
    want = gated_grads(dv, *values, gv, uv, activation)
    tols = backward_tolerances(dv, gv, uv, values, want, activation, t)
    names = ("grad_x", "grad_gate_weight", "grad_up_weight", "grad_gate_bias", "grad_up_bias")
    for p, q, tol, name in zip(got, want, tols, names):
        if p is None:
            assert not bias and name.endswith("bias")
            continue
        R.assert_within(p, q, tol + R.rounding(q.abs() + tol, t), name)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
def test_backward_sizes(device, kind, activation):
    for k, (M, N, K) in enumerate(((1, 1, 1), (1, 64, 40), (3, 7, 9), (16, 17, 33), (64, 64, 64), (65, 130, 31),
                                   (129, 100, 257), (300, 520, 200), (2, 1001, 1279), (700, 24, 600), (130, 192, 128))):
        say(f"gated backward {kind} {activation} M={M} N={N} K={K}")
        check_backward(device, kind, M, N, K, activation, seed=k, bias=k % 3 != 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3800, 1852, 3528), (2100, 1025, 1000), (130, 1024, 3000), (1500, 801, 1001),
                                   (1031, 640, 1024), (2801, 3701, 2525)])
@pytest.mark.parametrize("activation", ["none", "relu"])
def test_backward_large_tiles(device, M, N, K, activation):
    """Sizes at which the products take the large and the middling tiles, with ragged edges and with rows that are
    copied first; fp64 on the GPU."""
    from hyper_connection_residual_mhc_amd import gated as G
    say(f"gated backward M={M} N={N} K={K} {activation}")
    gen = torch.Generator(device=device).manual_seed(M)
    d, x, wg, wu, g, u = (torch.randn(s, device=device, generator=gen).to(BF16)
                          for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N)))
    got = G.gated_backward(d, x, wg, wu, g, u, bias=True, activation=activation)
    # relu and none are exact; the products of two bf16 values are exact in fp32 and round to 16 bits once, as here
    a = torch.where(g > 0, g, torch.zeros_like(g)) if activation == "relu" else g
    on = (g > 0).double() if activation == "relu" else torch.ones_like(g, dtype=torch.float64)
    fg, fu = d.double() * u.double() * on, d.double() * a.double()
    dg, du = fg.to(BF16).double(), fu.to(BF16).double()
    xv, wgv, wuv = x.double(), wg.double(), wu.double()
    half = -(-N // 64) * 64
    for p, want, size, length in (
            (got[0], dg @ wgv + du @ wuv, dg.abs() @ wgv.abs() + du.abs() @ wuv.abs(), 2 * half),
            (got[1], dg.t() @ xv, dg.abs().t() @ xv.abs(), M), (got[2], du.t() @ xv, du.abs().t() @ xv.abs(), M)):
        tol = size * additions(length, 32) * STEP
        tol = tol + (want.abs() + tol) * R.HALF_STEP[BF16] + R.HALF_TINY[BF16]
        over = (p.double() - want).abs() - tol
        assert float(over.max()) <= 0, int((over > 0).sum())
    for p, f in ((got[3], fg), (got[4], fu)):
        want = f.sum(0)
        tol = f.abs().sum(0) * (8 + 4 + math.ceil(M / 8)) * STEP
        assert float(((p.double() - want).abs() - tol - (want.abs() + tol) * R.HALF_STEP[BF16]).max()) <= 0


@pytest.mark.gpu
def test_backward_nothing(device):
    from hyper_connection_residual_mhc_amd import gated as G
    x, w = torch.empty(0, 24, dtype=BF16, device=device), torch.ones(40, 24, dtype=BF16, device=device)
    z = torch.empty(0, 40, dtype=BF16, device=device)
    outs = [R.Guarded(s, BF16, device) for s in ((40, 24), (40, 24), (40,), (40,))]
    G.mhc_gated_bwd(z, x, w, w, z, z, grad_x=torch.empty_like(x), grad_gate_weight=outs[0].t, grad_up_weight=outs[1].t,
                    grad_gate_bias=outs[2].t, grad_up_bias=outs[3].t)
    for o in outs:
        assert o.untouched() and not o.t.any()


@pytest.mark.gpu
def test_backward_alignment_and_edges(device):
    from hyper_connection_residual_mhc_amd import gated as G
    names = ("grad_x", "grad_gate_weight", "grad_up_weight", "grad_gate_bias", "grad_up_bias")
    for M, N, K in ((70, 72, 80), (33, 1001, 129)):
        a = check_backward(device, "bf16", M, N, K, "silu", seed=3)
        b = check_backward(device, "bf16", M, N, K, "silu", seed=3, place=R.shifted)
        for p, q in zip(a, b):
            assert R.same_bytes(p, q)
        gen = torch.Generator().manual_seed(1)
        args = [R.normal(gen, *s).to(device) for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N))]
        outs = [R.Guarded(s, BF16, device) for s in ((M, K), (N, K), (N, K), (N,), (N,))]
        ws = R.Guarded((G.mhc_gated_bwd_workspace_bytes(M, N, K, 1),), torch.uint8, device, 0xFF)
        G.mhc_gated_bwd(*args, **{n: o.t for n, o in zip(names, outs)}, workspace=ws.t)
        want = G.gated_backward(*args, bias=True)
        assert ws.untouched()
        for o, q in zip(outs, want):
            assert o.untouched() and R.same_bytes(o.t, q)
        # each launch's gradients alone
        for some in ((0,), (1, 2), (3,), (4,)):
            one = {names[i]: torch.empty_like(want[i]) for i in some}
            G.mhc_gated_bwd(*args, **one)
            for i in some:
                assert R.same_bytes(one[names[i]], want[i])


@pytest.mark.gpu
def test_autograd_streams_and_graphs(device):
    from hyper_connection_residual_mhc_amd import gated as G
    gen = torch.Generator().manual_seed(2)
    M, N, K = 150, 264, 320
    x, wg, wu, bg, bu, d = (R.normal(gen, *s).to(device) for s in ((M, K), (N, K), (N, K), (N,), (N,), (M, N)))

    def both(x):
        o = G.gated(x, wg, wu, bg, bu, activation="gelu", return_z=True)
        return (o.out, *G.gated_backward(d, x, wg, wu, o.gate, o.up, activation="gelu", bias=True))

    want = both(x)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, bg, bu)]
    out = G.gated_autograd(*leaves, activation="gelu")
    for p, q in zip((out, *torch.autograd.grad(out, leaves, d)), want):
        assert R.same_bytes(p, q)
    # one weight alone, without biases; a gradient that is no contiguous tensor
    out = G.gated_autograd(x, wg, leaves[2])
    o = G.gated(x, wg, wu, return_z=True)
    gu, = torch.autograd.grad(out, leaves[2], d.t().contiguous().t())
    assert R.same_bytes(gu, G.gated_backward(d, x, wg, wu, o.gate, o.up)[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bufs = [torch.empty_like(t) for t in (*want, out, out)]
    G.mhc_gated_fwd(x, wg, wu, bufs[0], gate_bias=bg, up_bias=bu, activation="gelu", gate=bufs[6], up=bufs[7], stream=side)
    G.mhc_gated_bwd(d, x, wg, wu, bufs[6], bufs[7], grad_x=bufs[1], grad_gate_weight=bufs[2], grad_up_weight=bufs[3],
                    grad_gate_bias=bufs[4], grad_up_bias=bufs[5], activation="gelu", stream=side)
    side.synchronize()
    for p, q in zip(bufs, want):
        assert R.same_bytes(p, q)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(buf)
        small = G.gated(buf[:4], wg, wu, bg).out
    for k in range(4):
        new = (x * (k + 1)).contiguous()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((*got, small), (*both(new), G.gated(new[:4], wg, wu, bg).out)):
            assert R.same_bytes(p, q), k
