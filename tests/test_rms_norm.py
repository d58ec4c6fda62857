"""The root-mean-square norm (include/mhc_rms_norm.h) against its fp64 form,
forward and backward, and the rules of the call.

Tolerances, derived from the kernels' arithmetic (u = 2^-24, half a step of
fp32). A row's sum of squares is a chain of at most 8 * ceil(H / (8 * threads))
fused steps in each thread, 6 tree steps and 7 joins of positive terms, so its
relative error is at most M u with M that count; rstd takes half of it and
four more roundings (mean, + eps, root, quotient); y two products and one
rounding to its type.
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

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def threads(H: int) -> int:
    return next((t for t in (64, 128, 256) if H <= 8 * t), 512)


def chain(H: int) -> int:
    """Roundings of a sum over a row, at most."""
    return 8 * math.ceil(H / (8 * threads(H))) + 6 + 7


def rstd_rel(H: int) -> float:
    return (chain(H) / 2 + 4) * R.U32


# ---------------------------------------------------------------------------
# The fp64 form itself (CPU)
# ---------------------------------------------------------------------------

def test_formula_gradients_are_the_differences_of_the_forward():
    gen = torch.Generator().manual_seed(3)
    T, H = 3, 7
    x = torch.randn(T, H, generator=gen, dtype=torch.float64)
    w = torch.randn(H, generator=gen, dtype=torch.float64)
    g = torch.randn(T, H, generator=gen, dtype=torch.float64)
    gs = torch.randn(T, H, generator=gen, dtype=torch.float64)

    def loss():
        return (R.norm(x, w, 0.01)[0] * g).sum() + (gs * x).sum()

    gx, gw = R.norm_grads(g, x, w, R.norm(x, w, 0.01)[1], gs)
    # central differences of step 1e-5: truncation 1e-10 of third derivatives of order 10
    assert torch.allclose(gx, R.differences(loss, x), rtol=0, atol=1e-7)
    assert torch.allclose(gw, R.differences(loss, w), rtol=0, atol=1e-7)


def test_mx_power_is_the_smallest_that_holds():
    amax = torch.tensor([448.0, 448.0001, 1.75, 1.7500001, 2.0, 0.0, 1e-45, 3e38, 1.0])
    p = R.mx_power(amax)
    a = amax.double()
    assert ((a <= 448 * 2.0 ** p.double()) | (p == 127)).all()
    assert ((a > 448 * 2.0 ** (p.double() - 1)) | (p == -127)).all()


# ---------------------------------------------------------------------------
# Host rules (CPU)
# ---------------------------------------------------------------------------

BASE = 1 << 36
GAP = 1 << 30


def fwd_args(**kw):
    a = dict(x=BASE, residual=None, pre=None, n=0, weight=BASE + GAP, weight_dtype=_lib.MHC_NORM_BF16,
             eps=1e-6, out=BASE + 2 * GAP, scales=None, stored=None, rstd=None, T=5, H=40,
             dtype=_lib.MHC_NORM_BF16, out_format=_lib.MHC_NORM_SAME)
    a.update(kw)
    return list(a.values())


@pytest.fixture(scope="module")
def lib(built_library):
    return _lib.norm_lib()


@pytest.mark.parametrize("kw", [
    {}, {"T": 0, "x": None, "out": None, "weight": None}, {"residual": BASE + 3 * GAP, "stored": BASE + 4 * GAP},
    {"pre": BASE + 3 * GAP, "n": 4, "stored": BASE + 4 * GAP, "rstd": BASE + 5 * GAP},
    {"out_format": 1, "scales": BASE + 3 * GAP}, {"out_format": 2, "scales": BASE + 3 * GAP + 1, "out": BASE + 2 * GAP + 1},
    {"weight_dtype": 0}, {"dtype": 0, "weight_dtype": 0}, {"dtype": 2, "weight_dtype": 2}, {"eps": 0.0}, {"H": 1},
])
def test_valid_forward_arguments(lib, kw):
    assert lib.mhc_rms_norm_validate_fwd(*fwd_args(**kw)) == MHC_SUCCESS


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"H": 0}, {"H": (1 << 26) + 1}, {"dtype": 3}, {"dtype": -1}, {"weight_dtype": 2}, {"out_format": 3},
    {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}, {"x": None}, {"weight": None}, {"out": None},
    {"x": BASE + 1}, {"out": BASE + 2 * GAP + 1}, {"weight_dtype": 0, "weight": BASE + GAP + 2},
    {"residual": BASE + 3 * GAP, "pre": BASE + 4 * GAP, "n": 4}, {"pre": BASE + 3 * GAP, "n": 3},
    {"pre": BASE + 3 * GAP, "n": 0}, {"n": 4}, {"pre": BASE + 3 * GAP, "n": 4, "dtype": 0, "weight_dtype": 0},
    {"stored": BASE + 4 * GAP}, {"scales": BASE + 3 * GAP}, {"out_format": 1}, {"out_format": 2},
    {"out_format": 1, "scales": BASE + 3 * GAP + 2}, {"rstd": BASE + 3 * GAP + 2}, {"T": 1 << 62},
])
def test_refused_forward_arguments(lib, kw):
    assert lib.mhc_rms_norm_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_INVALID_VALUE
    assert lib.mhc_rms_norm_last_error_message() != b""


@pytest.mark.parametrize("kw", [
    {"out": BASE}, {"out": BASE + 398}, {"out": BASE + GAP}, {"residual": BASE + 2 * GAP},
    {"residual": BASE + 3 * GAP, "stored": BASE}, {"residual": BASE + 3 * GAP, "stored": BASE + 3 * GAP},
    {"rstd": BASE}, {"out_format": 1, "scales": BASE + 2 * GAP}, {"pre": BASE + 2 * GAP, "n": 2},
])
def test_overlapping_forward_arguments(lib, kw):
    assert lib.mhc_rms_norm_validate_fwd(*fwd_args(**kw)) == MHC_ERROR_ALIASING


def bwd_args(**kw):
    a = dict(grad_y=BASE, stored=BASE + GAP, weight=BASE + 2 * GAP, weight_dtype=1, rstd=BASE + 3 * GAP,
             grad_stored=None, grad_x=BASE + 4 * GAP, grad_weight=BASE + 5 * GAP, workspace=BASE + 6 * GAP,
             workspace_bytes=5 * 40 * 4, T=5, H=40, dtype=1)
    a.update(kw)
    return list(a.values())


def test_backward_arguments(lib):
    v = lib.mhc_rms_norm_validate_bwd
    assert v(*bwd_args()) == MHC_SUCCESS
    assert v(*bwd_args(grad_stored=BASE + 7 * GAP)) == MHC_SUCCESS
    none = dict(T=0, grad_y=None, stored=None, weight=None, rstd=None, grad_x=None, workspace=None, workspace_bytes=0)
    assert v(*bwd_args(**none)) == MHC_SUCCESS
    assert v(*bwd_args(**none, grad_weight=None)) == MHC_ERROR_INVALID_VALUE
    for kw in ({"workspace_bytes": 5 * 40 * 4 - 1}, {"workspace": None}, {"rstd": None}, {"grad_weight": None},
               {"grad_x": None}, {"T": -1}, {"H": 0}, {"dtype": 7}, {"weight_dtype": 2}, {"grad_weight": BASE + 5 * GAP + 2}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
    for kw in ({"grad_x": BASE}, {"grad_x": BASE + GAP}, {"workspace": BASE}, {"grad_weight": BASE + 6 * GAP},
               {"grad_stored": BASE + 4 * GAP}):
        assert v(*bwd_args(**kw)) == MHC_ERROR_ALIASING, kw


def test_workspace_bytes(lib):
    f = lib.mhc_rms_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(1, 64) == 256 and f(100, 64) == 25600
    assert f(1 << 20, 64) == f(1 << 21, 64) > 0
    assert f(10, 20000) == 80000 and f(33, 20000) == 160000 and f(-1, 64) == -1 and f(1, 0) == -1 and f(1, (1 << 26) + 1) == -1


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import norm
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        norm.rms_norm(x, torch.ones(8))                    # not on a GPU
    with pytest.raises(TypeError):
        norm.rms_norm(x.double(), torch.ones(8))
    with pytest.raises(ValueError):
        norm.rms_norm(x[0], torch.ones(8))
    with pytest.raises(ValueError):
        norm.rms_norm(torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.ones(8), pre=torch.ones(2, 3))


# ---------------------------------------------------------------------------
# Forward (GPU)
# ---------------------------------------------------------------------------

def make(T, H, dtype, source, seed, n=4, dev="cuda:0"):
    gen = torch.Generator().manual_seed(seed)
    shape = (T, n, H) if source == "streams" else (T, H)
    x = R.normal(gen, *shape, dtype=dtype)
    residual = R.normal(gen, T, H, dtype=dtype, scale=2.0) if source == "add" else None
    pre = torch.rand((T, n), generator=gen) if source == "streams" else None
    weight = 1 + R.normal(gen, H, dtype=torch.float32, scale=0.2)
    return x, residual, pre, weight


def want_stored(x, residual, pre):
    """The stored row in its storage type (fp32 operations, one rounding)."""
    if pre is not None:
        p = pre[:, :, None] * x.float()
        while p.shape[1] > 1:
            p = p[:, 0::2] + p[:, 1::2]
        return p[:, 0].to(x.dtype)
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def run(x, residual, pre, weight, dev, quant=None, place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import norm
    up = lambda t: None if t is None else place(t, dev)  # noqa: E731
    o = norm.rms_norm(up(x), up(weight), EPS, residual=up(residual), pre=up(pre), quant=quant, return_rstd=True)
    torch.cuda.synchronize()
    return o


def check_quantised(o, v, quant, rel):
    """q and scales against the fp64 normed rows v, whose fp32 values are within rel."""
    q = R.d(o.y)
    if quant == "row":
        scale = R.d(o.scales)
        amax = v.abs().amax(1)
        want = (amax / 448).clamp_min(2.0 ** -126)
        R.assert_within(o.scales, want, want * (rel + 2 * R.U32), "row scales")
        back, unit = q * scale[:, None], scale[:, None]
        rel = rel + 3 * R.U32
    else:
        amax = R.block_amax(v)
        p = o.scales.cpu().view(torch.uint8).to(torch.int64) - 127
        low, high = R.mx_power(amax * (1 - rel)), R.mx_power(amax * (1 + rel))
        assert ((p >= low) & (p <= high)).all(), "mx scales"
        unit = (2.0 ** p.double()).repeat_interleave(32, 1)[:, :v.shape[1]]
        back = q * unit
        rel = rel + R.U32
    tol = v.abs() * (rel + (1 + rel) * R.HALF_STEP[torch.float8_e4m3fn]) + unit * R.HALF_TINY[torch.float8_e4m3fn]
    R.assert_within(back, v, tol, f"{quant} values")


WIDTHS = [1, 7, 8, 31, 33, 96, 512, 520, 1023, 1279, 2048, 4096, 4104, 7168, 8200, 16384, 16385, 20008]


@pytest.mark.gpu
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("source", ["plain", "add", "streams"])
def test_forward_widths(device, H, source):
    T = 3
    say(f"norm forward {source} H={H}")
    for k, dtype in enumerate((torch.bfloat16,) if source == "streams" else tuple(TYPES.values())):
        for quant in (None, "row", "mx"):
            x, residual, pre, weight = make(T, H, dtype, source, seed=H + k, n=(2, 4, 8)[H % 3])
            weight = weight if H % 2 else weight.to(dtype)
            o = run(x, residual, pre, weight, device, quant)
            s = want_stored(x, residual, pre)
            if source == "plain":
                assert o.stored is None
            else:
                assert R.same_bytes(o.stored, s), "stored"
            v, rstd = R.norm(R.d(s), R.d(weight), EPS)
            R.assert_within(o.rstd, rstd, rstd * rstd_rel(H), "rstd")
            rel = rstd_rel(H) + 2 * R.U32
            if quant is None:
                R.assert_within(o.y, v, v.abs() * rel + R.rounding(v * (1 + rel), dtype), "y")
            else:
                check_quantised(o, v, quant, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 2, 257, 1000])
def test_forward_batches_and_row_bytes(device, T):
    """Any T; a row's bytes do not depend on T or its place."""
    from hyper_connection_residual_mhc_amd import norm
    H = 1288
    x, residual, _, weight = make(max(T, 1), H, torch.bfloat16, "add", seed=5)
    x, residual, weight = x[:T].to(device), residual[:T].to(device), weight.to(device)
    for quant in (None, "row", "mx"):
        o = norm.rms_norm(x, weight, EPS, residual=residual, quant=quant, return_rstd=True)
        for t in {0, T // 2, T - 1} if T else ():
            one = norm.rms_norm(x[t:t + 1], weight, EPS, residual=residual[t:t + 1], quant=quant, return_rstd=True)
            for a, b in zip(o, one):
                assert a is None or R.same_bytes(a[t:t + 1], b)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "row", "mx"])
@pytest.mark.parametrize("H", [1279, 4096, 16400])
def test_forward_alignment_and_edges(device, quant, H):
    """Buffers one element past alignment give the same bytes; nothing outside an output is written."""
    from hyper_connection_residual_mhc_amd import norm
    T = 5
    x, residual, _, weight = make(T, H, torch.bfloat16, "add", seed=6)
    o = run(x, residual, None, weight, device, quant)
    m = run(x, residual, None, weight, device, quant, place=R.shifted)
    for a, b in zip(o, m):
        assert a is None or R.same_bytes(a, b)
    for fill in (0xA5, 0x3C):
        y = R.Guarded((T, H), o.y.dtype, device, fill)
        stored = R.Guarded((T, H), torch.bfloat16, device, fill)
        rstd = R.Guarded((T,), torch.float32, device, fill)
        scales = None if quant is None else R.Guarded(tuple(o.scales.shape), o.scales.dtype, device, fill)
        norm.mhc_rms_norm_fwd(x.to(device), weight.to(device), y.t, eps=EPS, residual=residual.to(device),
                              stored=stored.t, rstd=rstd.t, scales=None if scales is None else scales.t, quant=quant)
        for got, want in zip((y, scales, stored, rstd), o):
            if got is not None:
                assert got.untouched() and R.same_bytes(got.t, want)


@pytest.mark.gpu
def test_forward_streams_are_the_collapse(device):
    from hyper_connection_residual_mhc_amd import norm, ops
    for n in (2, 4, 8):
        x, _, pre, weight = make(9, 1279, torch.bfloat16, "streams", seed=n, n=n)
        x, pre, weight = x.to(device), pre.to(device), weight.to(device)
        fused = norm.rms_norm(x, weight, EPS, pre=pre)
        row = ops.h_aggregate(x, pre)
        assert R.same_bytes(fused.stored, row)
        assert R.same_bytes(fused.y, norm.rms_norm(row, weight, EPS).y)


@pytest.mark.gpu
def test_forward_extremes(device):
    """Zero rows, subnormals, infinities and NaN stay in their rows and give what the formulas give."""
    from hyper_connection_residual_mhc_amd import norm
    H = 96
    x = torch.ones(6, H)
    x[0] = 0
    x[1] = 1e-20
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4] = 0
    x[4, 64:] = 1e4
    w = torch.ones(H)
    o = norm.rms_norm(x.to(device), w.to(device), EPS)
    y = o.y.cpu()
    assert (y[0] == 0).all()
    assert (y[2, :5] == 0).all() and torch.isnan(y[2, 5])
    assert torch.isnan(y[3]).all()
    assert torch.allclose(y[5], torch.ones(H) / (1 + EPS) ** 0.5, rtol=1e-6)
    q = norm.rms_norm(x.to(device), w.to(device), EPS, quant="mx")
    codes = q.scales.cpu().view(torch.uint8)
    assert (codes[0] == 0).all() and (q.y[0].float() == 0).all()
    assert codes[4, 0] == 0 and codes[4, 2] > 0
    assert torch.isnan(q.y[3].float()).all()
    r = norm.rms_norm(x.to(device), w.to(device), EPS, quant="row")
    assert float(r.scales[0]) == 2.0 ** -126 and (r.y[0].float() == 0).all()
    big = torch.full((1, H), 3e38).to(device)
    huge = norm.rms_norm(torch.ones(1, H, device=device), big[0], EPS, quant="mx")
    assert (huge.scales.cpu().view(torch.uint8) == 127 + 120).all()   # 448 * 2^120 holds the largest fp32
    assert torch.isfinite(huge.y.float()).all()
    # eps = 0 with a zero row: 1 / 0 times 0 is a NaN, as the formula says; the other rows are not touched by it
    z = norm.rms_norm(x.to(device), w.to(device), 0.0).y.cpu()
    assert torch.isnan(z[0]).all() and torch.isfinite(z[5]).all()


@pytest.mark.gpu
def test_mx_scale_at_the_border(device):
    """Blocks whose largest value is exactly 448 * 2^k, and one step beyond, in fp32 with unit rows."""
    from hyper_connection_residual_mhc_amd import norm
    H = 64
    x = torch.ones(1, H)
    w = torch.full((H,), 1e-3)
    w[3], w[40] = 1.75, torch.nextafter(torch.tensor(1.75), torch.tensor(2.0))
    q = norm.rms_norm(x.to(device), w.to(device), 0.0, quant="mx")   # rstd is exactly 1
    codes = q.scales.cpu().view(torch.uint8)[0].tolist()
    assert codes == [127 - 8, 127 - 7]
    assert float(q.y[0, 3].float()) == 448.0 and float(q.y[0, 40].float()) == 224.0


# ---------------------------------------------------------------------------
# Backward (GPU)
# ---------------------------------------------------------------------------

def check_backward(device, T, H, dtype, with_stored, seed, place=lambda t, dev: t.to(dev)):
    from hyper_connection_residual_mhc_amd import norm
    gen = torch.Generator().manual_seed(seed)
    s = R.normal(gen, T, H, dtype=dtype)
    g = R.normal(gen, T, H, dtype=dtype, scale=0.5)
    w = 1 + R.normal(gen, H, dtype=torch.float32, scale=0.2)
    w = w if seed % 2 else w.to(dtype)
    gs = R.normal(gen, T, H, dtype=dtype) if with_stored else None
    rstd = (1 / torch.sqrt((s.double() ** 2).mean(1) + EPS)).float()
    up = lambda t: None if t is None else place(t, device)  # noqa: E731
    gx, gw = norm.rms_norm_backward(up(g), up(s), up(w), up(rstd), grad_stored=up(gs))
    torch.cuda.synchronize()
    r = R.d(rstd)
    want_x, want_w = R.norm_grads(R.d(g), R.d(s), R.d(w), r, R.d(gs))
    u = (R.d(g) * R.d(w)).abs()
    sa = R.d(s).abs()
    # dot: one rounding in u, chain(H) in the sum; c: three more; the row: two products, one difference, one sum
    dot = (u * sa).mean(1, keepdim=True) * r[:, None] ** 2
    tol = r[:, None] * (5 * u + (chain(H) + 8) * sa * dot) * R.U32 + want_x.abs() * R.U32
    R.assert_within(gx, want_x, tol + R.rounding(want_x.abs() + tol, dtype), "grad_x")
    # rows: a product and a fused step each, the block's chain, then the parts of the blocks
    blocks = min(T, 512) if H <= 16384 else 1
    steps = 1 + math.ceil(T / max(blocks, 1)) + math.ceil(blocks / 4) + 3
    R.assert_within(gw, want_w, (R.d(g) * R.d(s) * r[:, None]).abs().sum(0) * steps * R.U32 + 2.0 ** -140, "grad_weight")
    return gx, gw


@pytest.mark.gpu
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(device, H):
    say(f"norm backward H={H}")
    for k, dtype in enumerate(TYPES.values()):
        check_backward(device, 3, H, dtype, with_stored=(H + k) % 2 == 0, seed=H + k)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 511, 513, 1500])
def test_backward_batches(device, T):
    check_backward(device, T, 264, torch.bfloat16, True, seed=T)
    check_backward(device, T, 129, torch.float32, False, seed=T + 1)


@pytest.mark.gpu
def test_longest_row(device):
    from hyper_connection_residual_mhc_amd import norm
    H = _lib.MHC_MAX_H
    say(f"norm forward and backward H={H}")
    gen = torch.Generator().manual_seed(3)
    s, g = R.normal(gen, 1, H), R.normal(gen, 1, H, scale=0.5)
    w = torch.ones(H, device=device)
    out = norm.rms_norm(s.to(device), w, EPS, return_rstd=True)
    sd = s.to(device).double()
    want = sd / torch.sqrt((sd ** 2).mean() + EPS)
    # the sum's order: 512 threads, a chain of chunks each, then trees
    tol = want.abs() * (H / 512 + 32) * R.U32
    assert bool(((out.y.double() - want).abs() <= tol + R.rounding(want.abs() + tol, torch.bfloat16)).all())
    gx, gw = norm.rms_norm_backward(g.to(device), s.to(device), w, out.rstd)
    exact = g.to(device).double()[0] * sd[0] * out.rstd.double()
    # a product and a fused step, and zeros added
    assert bool(((gw.double() - exact).abs() <= exact.abs() * 4 * R.U32 + 2.0 ** -140).all())
    assert bool(torch.isfinite(gx).all())


@pytest.mark.gpu
def test_backward_alignment_and_edges(device):
    from hyper_connection_residual_mhc_amd import norm
    a = check_backward(device, 6, 1279, torch.float16, True, seed=9)
    b = check_backward(device, 6, 1279, torch.float16, True, seed=9, place=R.shifted)
    assert R.same_bytes(a[0], b[0]) and R.same_bytes(a[1], b[1])
    gen = torch.Generator().manual_seed(1)
    s, g = R.normal(gen, 6, 520).to(device), R.normal(gen, 6, 520).to(device)
    w, r = torch.ones(520, device=device), torch.ones(6, device=device)
    gx, gw = R.Guarded((6, 520), torch.bfloat16, device), R.Guarded((520,), torch.float32, device)
    need = norm.mhc_rms_norm_bwd_workspace_bytes(6, 520)
    ws = R.Guarded((need,), torch.uint8, device)
    norm.mhc_rms_norm_bwd(g, s, w, r, gx.t, gw.t, workspace=ws.t)
    want = norm.rms_norm_backward(g, s, w, r)
    assert gx.untouched() and gw.untouched() and ws.untouched()
    assert R.same_bytes(gx.t, want[0]) and R.same_bytes(gw.t, want[1])


@pytest.mark.gpu
def test_autograd_runs_the_kernels(device):
    from hyper_connection_residual_mhc_amd import norm, ops
    x, residual, _, weight = (t if t is None else t.to(device) for t in make(7, 320, torch.bfloat16, "add", seed=2))
    gen = torch.Generator().manual_seed(4)
    g, gs = R.normal(gen, 7, 320).to(device), R.normal(gen, 7, 320).to(device)
    leaves = [t.clone().requires_grad_() for t in (x, residual, weight)]
    y, stored = norm.rms_norm_autograd(leaves[0], leaves[2], EPS, residual=leaves[1])
    got = torch.autograd.grad((y, stored), leaves, (g, gs))
    o = norm.rms_norm(x, weight, EPS, residual=residual, return_rstd=True)
    gx, gw = norm.rms_norm_backward(g, o.stored, weight, o.rstd, grad_stored=gs)
    assert R.same_bytes(y, o.y) and R.same_bytes(got[0], gx) and R.same_bytes(got[1], gx) and R.same_bytes(got[2], gw)
    # through the collapse, with only y used
    st, _, pre, weight = (t if t is None else t.to(device) for t in make(7, 320, torch.bfloat16, "streams", seed=3))
    leaves = [t.clone().requires_grad_() for t in (st, pre, weight.bfloat16())]
    y, stored = norm.rms_norm_autograd(leaves[0], leaves[2], EPS, pre=leaves[1])
    got = torch.autograd.grad(y, leaves, g)
    o = norm.rms_norm(st, weight.bfloat16(), EPS, pre=pre, return_rstd=True)
    gx, gw = norm.rms_norm_backward(g, o.stored, weight.bfloat16(), o.rstd)
    gst, gpre = ops.h_aggregate_backward(st, pre, gx)
    assert R.same_bytes(got[0], gst) and R.same_bytes(got[1], gpre) and R.same_bytes(got[2], gw.bfloat16())
    # only the stored row used, and x alone
    y, stored = norm.rms_norm_autograd(leaves[0], leaves[2], EPS, pre=leaves[1])
    got = torch.autograd.grad(stored, leaves[:2], g)
    gst, gpre = ops.h_aggregate_backward(st, pre, g)
    assert R.same_bytes(got[0], gst) and R.same_bytes(got[1], gpre)
    leaf = x.clone().requires_grad_()
    y, none = norm.rms_norm_autograd(leaf, weight, EPS)
    assert none is None
    y.sum().backward()
    assert leaf.grad.shape == x.shape


@pytest.mark.gpu
def test_streams_and_graphs(device):
    """Another stream than the current one, and a captured call replayed on new inputs."""
    from hyper_connection_residual_mhc_amd import norm
    T, H = 33, 2056
    x, residual, _, weight = (t if t is None else t.to(device) for t in make(T, H, torch.bfloat16, "add", seed=8))
    gen = torch.Generator().manual_seed(4)
    g = R.normal(gen, T, H).to(device)

    def both(x):
        o = norm.rms_norm(x, weight, EPS, residual=residual, quant=None, return_rstd=True)
        q = norm.rms_norm(x, weight, EPS, residual=residual, quant="mx")
        return (o.y, o.stored, q.y, q.scales, *norm.rms_norm_backward(g, o.stored, weight, o.rstd, grad_stored=g))

    want = both(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, stored, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=device)
    gx, gw = torch.empty_like(x), torch.empty(H, device=device)
    side.wait_stream(torch.cuda.current_stream())
    norm.mhc_rms_norm_fwd(x, weight, y, eps=EPS, residual=residual, stored=stored, rstd=rstd, stream=side)
    norm.mhc_rms_norm_bwd(g, stored, weight, rstd, gx, gw, grad_stored=g, stream=side)
    side.synchronize()
    for a, b in zip((y, stored, gx, gw), (want[0], want[1], want[4], want[5])):
        assert R.same_bytes(a, b)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(buf)
    for k in range(4):
        new = (x * (k + 1)).contiguous()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, both(new)):
            assert R.same_bytes(a, b), k
