"""The cross entropy of a large vocabulary (include/mhc_cross_entropy.h) against
its fp64 form, forward and gradients, and the rules of the calls.

Tolerances. A logit is a sum as in test_linear.py, off by at most dz. lse moves
by at most the mean of dz under the softmax. An exponential of a difference d is
off by |d| 4 u (its rounding, the product with log2 e and that constant's; u =
2^-24) and 4 u of the instruction; under the weight exp(d) of its term |d| 4 u is
at most 2 u, so each of the steps that a term goes through (in its group of 64, in
the joins of the groups of a thread, in the halving over at most 1024 threads)
costs at most 8 u of the sum, which is what lse sees. The logarithm and the
additions cost 4 u of their values.
A probability p made again from z and lse is off by dz + dlse + (|z - lse| + 2) 4 u
of itself; one that was held in fp16 under its group's maximum also by half a step
of fp16, or next to zero by half of fp16's smallest number over 2^15; what is below
2^-126 may count as 0. G is rounded (in fp16 after scaling its
largest share to 2^14 at least), and the products over it see that in full.
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
from test_linear import LARGE, MEDIUM, NARROW, ROWS, SMALL, STEP, additions

BF16, F16 = torch.bfloat16, torch.float16
TYPES = {"bf16": BF16, "f16": F16}
U = R.U32
GROUP = {ROWS: 8, SMALL: 32, MEDIUM: 64, LARGE: 64}
IGNORE = -100


def shares(targets, grad_loss, reduction, ignore):
    """s [M], fp64."""
    on = targets != ignore
    s = torch.ones(targets.shape, dtype=torch.float64, device=targets.device)
    if grad_loss is not None:
        s = s * grad_loss.double()
    if reduction == "mean":
        s = s / on.sum()
    return torch.where(on, s, torch.zeros_like(s))


def forward(x, w, targets, reduction, ignore):
    """(loss, lse, z, each row's loss), all fp64."""
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    on = targets != ignore
    each = torch.where(on, lse - z.gather(1, targets.clamp(0, w.shape[0] - 1)[:, None])[:, 0], torch.zeros_like(lse))
    loss = each if reduction == "none" else each.sum() if reduction == "sum" else each.sum() / on.sum()
    return loss, lse, z, each


def gradients(x, w, z, lse, targets, s, grad_lse=None):
    """(grad_x, grad_weight, G, p), all fp64."""
    p = torch.exp(z - lse[:, None])
    a = s if grad_lse is None else s + grad_lse
    g = p * a[:, None]
    rows = torch.arange(len(targets), device=z.device)
    g[rows, targets.clamp(0, w.shape[0] - 1)] -= s
    return g @ w, g.t() @ x, g, p


def errors(x, w, z, lse, V, K):
    """(dz [M, V], dlse [M])."""
    dz = (x.abs() @ w.abs().t()) * additions(K, 32) * STEP
    p = torch.exp(z - lse[:, None])
    steps = 16 + 4 + math.ceil(V / 8 / 64) + 10            # at least 64 threads to a row
    dlse = (p * dz).sum(1) + steps * 8 * U + lse.abs() * 4 * U + math.log(V + 1) * 4 * U
    return dz, dlse


# ---------------------------------------------------------------------------
# The fp64 form itself, and host rules (CPU)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_formula_gradients_are_the_differences_of_the_forward(reduction):
    gen = torch.Generator().manual_seed(5)
    M, V, K = 4, 6, 3
    x, w, e = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((M, K), (V, K), (M,)))
    g = torch.randn((M,) if reduction == "none" else (), generator=gen, dtype=torch.float64)
    targets = torch.tensor([2, IGNORE, 0, 5])

    def loss():
        out, lse, *_ = forward(x, w, targets, reduction, IGNORE)
        return (out * g).sum() + (lse * e).sum()

    _, lse, z, _ = forward(x, w, targets, reduction, IGNORE)
    gx, gw, *_ = gradients(x, w, z, lse, targets, shares(targets, g, reduction, IGNORE), e)
    for leaf, grad in ((x, gx), (w, gw)):
        assert torch.allclose(grad, R.differences(loss, leaf), rtol=0, atol=1e-7)


def test_formula_is_torch_s(built_library):
    gen = torch.Generator().manual_seed(6)
    x, w = torch.randn(9, 5, generator=gen, dtype=torch.float64), torch.randn(7, 5, generator=gen, dtype=torch.float64)
    targets = torch.tensor([0, 6, 3, IGNORE, 2, 2, IGNORE, 5, 1])
    for reduction in ("none", "sum", "mean"):
        want = torch.nn.functional.cross_entropy(x @ w.t(), targets, ignore_index=IGNORE, reduction=reduction)
        assert torch.allclose(forward(x, w, targets, reduction, IGNORE)[0], want, rtol=1e-12)


BASE = 1 << 40
GAP = 1 << 34


@pytest.fixture(scope="module")
def lib(built_library):
    return _lib.cross_entropy_lib()


def fwd_args(**kw):
    a = dict(x=BASE, w=BASE + GAP, targets=BASE + 2 * GAP, loss=BASE + 3 * GAP, lse=BASE + 4 * GAP, ws=BASE + 5 * GAP,
             ws_bytes=1 << 33, M=20, V=40, K=50, dtype=1, reduction=2, launch=None)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(x=BASE, w=BASE + GAP, targets=BASE + 2 * GAP, lse=BASE + 3 * GAP, g=BASE + 4 * GAP, gl=BASE + 5 * GAP,
             gx=BASE + 6 * GAP, gw=BASE + 7 * GAP, ws=BASE + 8 * GAP, ws_bytes=1 << 33, M=20, V=40, K=50, dtype=1,
             reduction=2, launch=None)
    a.update(kw)
    return list(a.values())


def grads_args(**kw):
    a = dict(x=BASE, w=BASE + GAP, targets=BASE + 2 * GAP, g=BASE + 3 * GAP, loss=BASE + 4 * GAP, lse=BASE + 5 * GAP,
             gx=BASE + 6 * GAP, gw=BASE + 7 * GAP, ws=BASE + 8 * GAP, ws_bytes=1 << 33, M=20, V=40, K=50, dtype=1,
             reduction=2, launch=None)
    a.update(kw)
    return list(a.values())


def launch(kernel, splits=0):
    from hyper_connection_residual_mhc_amd.linear import _launch_arg
    return _launch_arg({"kernel": kernel, "splits": splits})


CALLS = {"fwd": fwd_args, "bwd": bwd_args, "grads": grads_args}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_valid_arguments(lib, call):
    v, args = getattr(lib, f"mhc_cross_entropy_validate_{call}"), CALLS[call]
    for kw in ({}, {"dtype": 2}, {"reduction": 0}, {"reduction": 1}, {"x": BASE + 2, "w": BASE + GAP + 2}, {"V": 1 << 21, "K": 8},
               {"V": 1, "K": 1, "M": 1}, {"launch": launch(LARGE)}, {"launch": launch(0, 1)}, {"K": 1 << 21, "V": 8, "M": 1}):
        assert v(*args(**kw)) == MHC_SUCCESS, (kw, lib.mhc_cross_entropy_last_error_message())
    none = {"M": 0, "x": None, "targets": None, "lse": None, "ws": None, "ws_bytes": 0}
    assert v(*args(**none)) == MHC_SUCCESS
    if call != "bwd":
        assert v(*args(**none, reduction=0, loss=None)) == MHC_SUCCESS
        assert v(*args(launch=launch(ROWS), M=16)) == MHC_SUCCESS
    if call != "fwd":
        for kw in ({"g": None}, {"gx": None}, {"gw": None}, {"gx": None, "gw": None}):
            assert v(*args(**kw)) == MHC_SUCCESS, kw


@pytest.mark.parametrize("call", sorted(CALLS))
def test_refused_arguments(lib, call):
    v, args = getattr(lib, f"mhc_cross_entropy_validate_{call}"), CALLS[call]
    bad = [{"M": -1}, {"M": 1 << 31}, {"V": 0}, {"V": (1 << 21) + 1}, {"K": 0}, {"K": (1 << 21) + 1}, {"dtype": 0}, {"dtype": 3},
           {"dtype": 6}, {"reduction": -1}, {"reduction": 3}, {"x": None}, {"w": None}, {"targets": None}, {"lse": None},
           {"x": BASE + 1}, {"targets": BASE + 2 * GAP + 4}, {"ws": None}, {"ws": BASE + 8 * GAP + 8}, {"ws_bytes": 16},
           {"launch": launch(NARROW)}, {"launch": launch(SMALL, 2)}, {"launch": launch(6)}, {"launch": launch(ROWS)}]
    bad += [{"loss": None}, {"loss": BASE + 3 * GAP + 2}] if call != "bwd" else [{"launch": launch(ROWS), "M": 16}]
    bad += [{"gx": BASE + 6 * GAP + 1}, {"g": BASE + 3 * GAP + 1}] if call != "fwd" else []
    for kw in bad:
        assert v(*args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
        assert lib.mhc_cross_entropy_last_error_message() != b""
    over = [{"ws": BASE}, {"ws": BASE + 2 * GAP}]
    over += [{"loss": BASE + GAP}] if call != "bwd" else [{"gx": BASE + 3 * GAP}]
    over += [{"gx": BASE}, {"gw": BASE + 6 * GAP}] if call != "fwd" else [{"lse": BASE + 3 * GAP}]
    for kw in over:
        assert v(*args(**kw)) == MHC_ERROR_ALIASING, kw


def test_workspaces_hold_a_chunk(built_library):
    """The values that are kept of the logits never pass a chunk's bytes."""
    from hyper_connection_residual_mhc_amd import loss
    for M in (1, 4096, 8192, 100000, 1 << 20):
        for V in (256, 50000, 131072, 1 << 21):
            K = 64
            held = loss.mhc_cross_entropy_workspace_bytes("bwd", M, V, K, 1) - 12 * M
            others = V * K * 4 + 32 * 128 * 4 * 256 * 256 + 4096     # sums of grad_weight, split sums
            assert held <= _lib.MHC_CROSS_ENTROPY_CHUNK_BYTES + others, (M, V)
    with pytest.raises(ValueError):
        loss.mhc_cross_entropy_workspace_bytes("bwd", 4, 0, 8, 1)
    with pytest.raises(ValueError):
        loss.mhc_cross_entropy_workspace_bytes("both", 4, 8, 8, 1)


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import loss
    x, w, t = torch.zeros(2, 8, dtype=BF16), torch.zeros(4, 8, dtype=BF16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        loss.linear_cross_entropy(x, w, t)                 # not on a GPU
    with pytest.raises(TypeError):
        loss.linear_cross_entropy(x.float(), w.float(), t)
    with pytest.raises(ValueError):
        loss.linear_cross_entropy(x[0], w, t)
    with pytest.raises(ValueError):
        loss.linear_cross_entropy(x, w, t, reduction="median")


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def make(kind, M, V, K, seed, scale=2.0, ignored=0.2, ignore=IGNORE):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    w = R.normal(gen, V, K, dtype=t, scale=scale * K ** -0.5)
    targets = torch.randint(V, (M,), generator=gen)
    x = (torch.randn(M, K, generator=gen) + 2 * torch.rand(M, 1, generator=gen) * w[targets].float()).to(t)
    drop = torch.rand(M, generator=gen) < ignored
    return x, w, torch.where(drop, torch.full_like(targets, ignore), targets)


def check_loss(got, lse, x, w, targets, reduction, ignore):
    """Against fp64 on the inputs' device."""
    (M, K), V = x.shape, w.shape[0]
    want, wl, z, each = forward(x, w, targets, reduction, ignore)
    dz, dlse = errors(x, w, z, wl, V, K)
    R.assert_within(lse, wl.cpu(), dlse.cpu(), "lse")
    at = targets.clamp(0, V - 1)[:, None]
    de = torch.where(targets != ignore, dlse + dz.gather(1, at)[:, 0] + (wl.abs() + z.gather(1, at)[:, 0].abs()) * 2 * U,
                     torch.zeros_like(dlse))
    if reduction == "none":
        R.assert_within(got, each.cpu(), de.cpu(), "loss")
        return z, wl, dz, dlse
    tol = de.sum() + (each.abs() + de).sum() * (math.ceil(M / 1024) + 20) * STEP
    if reduction == "mean":
        tol = tol / (targets != ignore).sum() + want.abs() * STEP
    R.assert_within(got, want.cpu(), tol.cpu(), "loss")
    return z, wl, dz, dlse


def check_grads(gx, gw, x, w, targets, s, z, lse, dz, dlse, t, held, group=64, grad_lse=None, pieces=1):
    V = w.shape[0]
    wx, ww, g, p = gradients(x, w, z, lse, targets, s, grad_lse)
    a = (s if grad_lse is None else s + grad_lse).abs()
    rel = dz + dlse[:, None] + ((z - lse[:, None]).abs() + 2) * 4 * U
    dp = p * rel + 2.0 ** -126
    if held:
        top = torch.nn.functional.pad(p, (0, -V % group)).view(len(p), -1, group).amax(2).repeat_interleave(group, 1)[:, :V]
        dp = dp + p * (1 + rel) * R.HALF_STEP[F16] + top * R.HALF_TINY[F16] * 2.0 ** -14
        dp = dp + p * ((top.clamp_min(1e-300).log()).abs() + 2) * 4 * U
    largest = torch.maximum(a, s.abs()).max()
    dg = a[:, None] * dp + (g.abs() + a[:, None] * p) * 4 * U
    dg = dg + (g.abs() + dg) * R.HALF_STEP[t] + R.HALF_TINY[t] * (largest * 2.0 ** -14 if t == F16 else 1.0)
    dg = torch.where((a == 0)[:, None] & (s == 0)[:, None], torch.zeros_like(dg), dg)
    ag = g.abs() + dg
    for got, want, tol, long, name in (
            (gx, wx, dg @ w.abs() + ag @ w.abs() * (additions(V, 32) + 2 * pieces) * STEP, V, "grad_x"),
            (gw, ww, dg.t() @ x.abs() + ag.t() @ x.abs() * (additions(len(x), 32) + 2 * pieces) * STEP, len(x), "grad_weight")):
        if got is not None:
            tol = tol + R.rounding(want.abs() + tol, t)
            R.assert_within(got, want.cpu(), tol.cpu(), name)


def run(device, kind, M, V, K, seed, reduction="mean", ignore=IGNORE, kernel=0, scale=2.0, ignored=0.2, weighted=True,
        place=lambda t, dev: t.to(dev)):
    """All three calls against fp64 (on the GPU), and the two ways to the loss against each other."""
    from hyper_connection_residual_mhc_amd import loss as C
    t = TYPES[kind]
    x, w, targets = make(kind, M, V, K, seed, scale, ignored, ignore)
    gen = torch.Generator().manual_seed(seed + 1)
    g = torch.randn((M,) if reduction == "none" else (), generator=gen).to(device) if weighted else None
    x, w, targets = place(x, device), place(w, device), targets.to(device)
    how = dict(ignore_index=ignore, reduction=reduction)
    named = {"kernel": kernel} if kernel else None
    value = torch.empty((M,) if reduction == "none" else (), device=device)
    lse = torch.empty(M, device=device)
    C.mhc_cross_entropy_fwd(x, w, targets, value, lse, launch=named, **how)
    xv, wv = x.double(), w.double()
    group = GROUP[kernel or (ROWS if M <= 16 else SMALL)]
    z, wl, dz, dlse = check_loss(value, lse, xv, wv, targets, reduction, ignore)
    s = shares(targets, g, reduction, ignore)
    # in one call: the same loss, bit for bit
    value2, lse2, gx, gw = torch.empty_like(value), torch.empty_like(lse), torch.empty_like(x), torch.empty_like(w)
    C.mhc_cross_entropy_grads(x, w, targets, value2, lse2, g, grad_x=gx, grad_weight=gw, launch=named, **how)
    assert R.same_bytes(value, value2) and R.same_bytes(lse, lse2)
    check_grads(gx, gw, xv, wv, targets, s, z, wl, dz, dlse, t, True, group)
    # from lse, with a gradient of lse as well
    e = torch.randn(M, generator=gen).to(device) * (float(s.abs().max()) + 1e-3)
    bx, bw = torch.empty_like(x), torch.empty_like(w)
    for ge in (None, e):
        C.mhc_cross_entropy_bwd(x, w, targets, lse, g, grad_lse=ge, grad_x=bx, grad_weight=bw,
                                launch=named if kernel != ROWS else None, **how)
        check_grads(bx, bw, xv, wv, targets, s, z, wl, dz, dlse, t, False, grad_lse=None if ge is None else ge.double())
    return value, lse, gx, gw, bx, bw


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_sizes(device, kind, reduction):
    for k, (M, V, K) in enumerate(((1, 1, 1), (1, 7, 9), (3, 33, 64), (16, 100, 40), (17, 64, 33), (65, 130, 31), (129, 257, 100),
                                   (5, 5000, 72), (2, 4099, 129), (300, 520, 200), (40, 1001, 1279))):
        say(f"cross entropy {kind} {reduction} M={M} V={V} K={K}")
        run(device, kind, M, V, K, seed=k, reduction=reduction)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("kernel", [ROWS, SMALL, MEDIUM, LARGE])
def test_kernels(device, kernel, kind):
    """Rows and columns around the tiles' and the groups' borders on every kernel of the logits."""
    bm, bn = {ROWS: (16, 16), SMALL: (64, 64), MEDIUM: (128, 128), LARGE: (256, 256)}[kernel]
    sizes = ((1, 1), (bm, bn), (bm - 1, bn - 1), (bm - 1, 3 * bn - 9), (bm // 2, bn + 1))
    sizes += ((3, 2100), (16, 4099)) if kernel == ROWS else ((bm + 1, bn + 7), (3 * bm + 5, bn // 2 + 3), (2 * bm, 2 * bn + 33))
    for k, (M, V) in enumerate(sizes):
        say(f"cross entropy {kind} kernel={kernel} M={M} V={V}")
        run(device, kind, M, V, 192, seed=k, kernel=kernel, reduction=("none", "mean", "sum")[k % 3])


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ROWS, SMALL, MEDIUM, LARGE])
def test_depths(device, kernel):
    M, V = (9, 50) if kernel == ROWS else (70, 140)
    for k, K in enumerate((1, 7, 8, 31, 33, 63, 64, 65, 128, 129, 520, 1279)):
        say(f"cross entropy kernel={kernel} K={K}")
        run(device, "bf16", M, V, K, seed=k, kernel=kernel, weighted=k % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_steep_and_flat_rows(device, kind):
    """Logits from nearly equal to hundreds apart: probabilities down to 0 and losses of hundreds."""
    for scale in (1e-3, 1.0, 40.0):
        for reduction in ("none", "mean"):
            say(f"cross entropy {kind} scale={scale}")
            run(device, kind, 70, 300, 128, seed=3, scale=scale, reduction=reduction)


@pytest.mark.gpu
def test_small_shares_in_fp16(device):
    """A mean over many rows of a flat distribution: shares of 2^-11 and probabilities of 2^-12, whose product is no
    normal number of fp16, come through the weight's gradient of a summed loss scaled up."""
    from hyper_connection_residual_mhc_amd import loss as C
    M, V, K = 2048, 4096, 64
    x, w, targets = (t.to(device) for t in make("f16", M, V, K, 9, scale=0.1, ignored=0.0))
    xv, wv = x.double(), w.double()
    _, lse, z, _ = forward(xv, wv, targets, "mean", IGNORE)
    dz, dlse = errors(xv, wv, z, lse, V, K)
    g = torch.tensor(4096.0, device=device)                # a loss scale
    o = C.linear_cross_entropy_grads(x, w, targets, g)
    check_grads(o.grad_x, o.grad_weight, xv, wv, targets, shares(targets, g, "mean", IGNORE), z, lse, dz, dlse, F16, True, 64)
    gx, gw = C.linear_cross_entropy_backward(x, w, targets, o.lse, g)
    check_grads(gx, gw, xv, wv, targets, shares(targets, g, "mean", IGNORE), z, lse, dz, dlse, F16, False)
    rel = float((o.grad_weight.double() - gradients(xv, wv, z, lse, targets, shares(targets, g, "mean", IGNORE))[1]).norm()
                / gradients(xv, wv, z, lse, targets, shares(targets, g, "mean", IGNORE))[1].norm())
    assert rel < 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("M,V,K", [(1000, 3000, 1024), (2100, 5000, 512), (1500, 2001, 1001), (700, 10007, 320)])
def test_large_tiles(device, M, V, K):
    """Sizes at which the products take the large and the middling tiles, with ragged edges and with rows that are
    copied first."""
    say(f"cross entropy M={M} V={V} K={K}")
    run(device, "bf16", M, V, K, seed=M)


@pytest.mark.gpu
def test_chunks_of_rows_and_pieces_of_the_vocabulary(device):
    """The largest vocabulary: rows go by the 256, and the weight's gradient is the chunks' sum. Then a weight past 2^31
    bytes, whose gradient of x is summed in pieces."""
    from hyper_connection_residual_mhc_amd import loss as C
    for M, V, K, kind in ((300, 1 << 21, 16, "bf16"), (17, 1 << 21, 600, "bf16")):
        say(f"cross entropy M={M} V={V} K={K}")
        gen = torch.Generator(device=device).manual_seed(M)
        w = (torch.randn(V, K, device=device, generator=gen) * K ** -0.5).to(BF16)
        x = torch.randn(M, K, device=device, generator=gen).to(BF16)
        targets = torch.randint(V, (M,), device=device, generator=gen)
        targets[M // 2], targets[0], targets[-1] = IGNORE, V - 1, 0
        o = C.linear_cross_entropy_grads(x, w, targets)
        f = C.linear_cross_entropy(x, w, targets)
        assert R.same_bytes(o.loss, f.loss) and R.same_bytes(o.lse, f.lse)
        xv, wv = x.double(), w.double()
        z, lse, dz, dlse = check_loss(f.loss, f.lse, xv, wv, targets, "mean", IGNORE)
        s = shares(targets, None, "mean", IGNORE)
        args = (xv, wv, targets, s, z, lse, dz, dlse, BF16)
        check_grads(o.grad_x, o.grad_weight, *args, True, 64, pieces=2)
        check_grads(*C.linear_cross_entropy_backward(x, w, targets, f.lse), *args, False, pieces=2)
        del z, dz, args, xv, wv


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 70])
def test_ignored_rows_and_targets_outside(device, M):
    from hyper_connection_residual_mhc_amd import loss as C
    V, K = 77, 40
    x, w, targets = (t.to(device) for t in make("bf16", M, V, K, 1, ignored=0.0))
    # an index of the vocabulary may be the ignored one
    run(device, "bf16", M, V, K, 2, ignore=5)
    none = torch.full_like(targets, IGNORE)
    for reduction, want in (("none", 0.0), ("sum", 0.0), ("mean", math.nan)):
        o = C.linear_cross_entropy_grads(x, w, none, reduction=reduction)
        assert torch.equal(torch.nan_to_num(o.loss, nan=-1.0), torch.full_like(o.loss, -1.0 if math.isnan(want) else 0.0))
        assert torch.isfinite(o.lse).all() and not o.grad_x.any() and not o.grad_weight.any()
        gx, gw = C.linear_cross_entropy_backward(x, w, none, o.lse, reduction=reduction)
        assert not gx.any() and not gw.any()
    # ignored rows give nothing whatever their logits are; x's own infinities stay out of grad_x
    wild = x.clone()
    wild[2] = math.nan
    hide = targets.clone()
    hide[2] = IGNORE
    o = C.linear_cross_entropy_grads(wild, w, hide, reduction="none")
    keep = [m for m in range(M) if m != 2]
    assert o.loss[2] == 0 and torch.isfinite(o.loss).all() and not o.grad_x[2].any()
    alone = C.linear_cross_entropy_grads(x, w, hide, reduction="none")
    assert R.same_bytes(o.grad_x[keep], alone.grad_x[keep])
    # a target outside is NaN in its own row and in sums over rows, and nothing is read for it
    for bad in (V, -1, 1 << 40, -(1 << 62)):
        t = targets.clone()
        t[1] = bad
        o = C.linear_cross_entropy_grads(x, w, t, reduction="none")
        assert torch.isnan(o.loss[1]) and torch.isnan(o.grad_x[1]).all() and torch.isnan(o.grad_weight).all()
        rest = [m for m in range(M) if m != 1]
        assert torch.isfinite(o.loss[rest]).all() and torch.isfinite(o.grad_x[rest]).all() and torch.isfinite(o.lse).all()
        assert torch.isnan(C.linear_cross_entropy(x, w, t).loss)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [6, 70])
def test_infinite_logits(device, M):
    from hyper_connection_residual_mhc_amd import loss as C
    V, K = 150, 8
    x, w = torch.zeros(M, K, dtype=BF16), torch.zeros(V, K, dtype=BF16)
    w[0, 0], w[149, 0], w[3, 1], w[:, 2] = 3e38, 3e38, -3e38, -3e38
    x[0, 0] = 3e38                                         # two logits are inf
    x[1, 1] = 3e38                                         # one is -inf
    x[2, 2] = 3e38                                         # all are -inf
    x[3, 4] = math.nan
    targets = torch.full((M,), 3)
    targets[0] = 149
    o = C.linear_cross_entropy(x.to(device), w.to(device), targets.to(device), reduction="none")
    lse, loss = o.lse.cpu(), o.loss.cpu()
    assert lse[0] == math.inf and lse[2] == -math.inf and torch.isnan(lse[3])
    assert abs(float(lse[1]) - math.log(149)) < 1e-5 and loss[1] == math.inf
    assert torch.isnan(loss[0]) and torch.isnan(loss[2]) and torch.isnan(loss[3])
    assert torch.allclose(lse[4:], torch.full_like(lse[4:], math.log(150)), atol=1e-5)
    g = C.linear_cross_entropy_grads(x.to(device), w.to(device), targets.to(device), torch.ones(M, device=device), reduction="none")
    assert R.same_bytes(g.lse, o.lse) and torch.isfinite(g.grad_x[4:]).all()
    # the row whose target has probability 0: its share is taken off there, and nothing is NaN
    assert torch.isfinite(g.grad_x[1, 3:]).all()


@pytest.mark.gpu
def test_nothing(device):
    from hyper_connection_residual_mhc_amd import loss as C
    x, w = torch.empty(0, 24, dtype=BF16, device=device), torch.ones(40, 24, dtype=BF16, device=device)
    t = torch.empty(0, dtype=torch.int64, device=device)
    assert C.linear_cross_entropy(x, w, t, reduction="none").loss.shape == (0,)
    assert float(C.linear_cross_entropy(x, w, t, reduction="sum").loss) == 0
    assert math.isnan(float(C.linear_cross_entropy(x, w, t).loss))
    gw = R.Guarded((40, 24), BF16, device)
    C.mhc_cross_entropy_grads(x, w, t, torch.empty((), device=device), torch.empty(0, device=device), grad_weight=gw.t)
    assert gw.untouched() and not gw.t.any()
    gw.t.fill_(1)
    C.mhc_cross_entropy_bwd(x, w, t, torch.empty(0, device=device), grad_weight=gw.t)
    assert gw.untouched() and not gw.t.any()


@pytest.mark.gpu
def test_alignment_and_edges(device):
    from hyper_connection_residual_mhc_amd import loss as C
    for M, V, K in ((5, 130, 64), (70, 72, 80), (33, 1001, 129), (300, 600, 264)):
        say(f"cross entropy edges M={M} V={V} K={K}")
        a = run(device, "bf16", M, V, K, seed=3, reduction="none")
        b = run(device, "bf16", M, V, K, seed=3, reduction="none", place=R.shifted)
        for p, q in zip(a, b):
            assert R.same_bytes(p, q)
        x, w, targets = (t.to(device) for t in make("bf16", M, V, K, 3))
        want = C.linear_cross_entropy_grads(x, w, targets)
        for fill in (0xA5, 0xFF):
            outs = [R.Guarded(s, t, device, fill) for s, t in (((), torch.float32), ((M,), torch.float32), ((M, K), BF16), ((V, K), BF16))]
            ws = R.Guarded((C.mhc_cross_entropy_workspace_bytes("grads", M, V, K, 1),), torch.uint8, device, fill)
            C.mhc_cross_entropy_grads(x, w, targets, outs[0].t, outs[1].t, grad_x=outs[2].t, grad_weight=outs[3].t, workspace=ws.t)
            assert ws.untouched()
            for o, q in zip(outs, want):
                assert o.untouched() and R.same_bytes(o.t, q)
            outs = [R.Guarded(s, BF16, device, fill) for s in ((M, K), (V, K))]
            ws = R.Guarded((C.mhc_cross_entropy_workspace_bytes("bwd", M, V, K, 1),), torch.uint8, device, fill)
            C.mhc_cross_entropy_bwd(x, w, targets, want.lse, grad_x=outs[0].t, grad_weight=outs[1].t, workspace=ws.t)
            assert ws.untouched() and all(o.untouched() for o in outs)
            for o, q in zip(outs, C.linear_cross_entropy_backward(x, w, targets, want.lse)):
                assert R.same_bytes(o.t, q)
            value, lse = R.Guarded((), torch.float32, device, fill), R.Guarded((M,), torch.float32, device, fill)
            ws = R.Guarded((C.mhc_cross_entropy_workspace_bytes("fwd", M, V, K, 1),), torch.uint8, device, fill)
            C.mhc_cross_entropy_fwd(x, w, targets, value.t, lse.t, workspace=ws.t)
            assert ws.untouched() and value.untouched() and lse.untouched()
            assert R.same_bytes(value.t, want.loss) and R.same_bytes(lse.t, want.lse)
        # each gradient alone
        one = torch.empty_like(x)
        C.mhc_cross_entropy_grads(x, w, targets, torch.empty_like(want.loss), torch.empty_like(want.lse), grad_x=one)
        assert R.same_bytes(one, want.grad_x)
        one = torch.empty_like(w)
        C.mhc_cross_entropy_grads(x, w, targets, torch.empty_like(want.loss), torch.empty_like(want.lse), grad_weight=one)
        assert R.same_bytes(one, want.grad_weight)


@pytest.mark.gpu
def test_autograd_streams_and_graphs(device):
    from hyper_connection_residual_mhc_amd import loss as C
    M, V, K = 150, 520, 320
    x, w, targets = (t.to(device) for t in make("bf16", M, V, K, 2))
    for reduction in ("none", "mean"):
        g = torch.rand((M,) if reduction == "none" else (), device=device)
        e = torch.rand(M, device=device)
        leaves = [t.clone().requires_grad_() for t in (x, w)]
        value, lse = C.linear_cross_entropy_autograd(*leaves, targets, reduction=reduction)
        plain = C.linear_cross_entropy(x, w, targets, reduction=reduction)
        assert R.same_bytes(value, plain.loss) and R.same_bytes(lse, plain.lse)
        for weights, ge in (((g, None), None), ((g, e), e)):
            outs = (value,) if weights[1] is None else (value, lse)
            got = torch.autograd.grad(outs, leaves, [v for v in weights if v is not None], retain_graph=True)
            want = C.linear_cross_entropy_backward(x, w, targets, lse.detach(), g, grad_lse=ge, reduction=reduction)
            for p, q in zip(got, want):
                assert R.same_bytes(p, q)
        # lse alone
        got = torch.autograd.grad(lse, leaves, e)
        zero = torch.zeros_like(g)
        for p, q in zip(got, C.linear_cross_entropy_backward(x, w, targets, lse.detach(), zero, grad_lse=e, reduction=reduction)):
            assert R.same_bytes(p, q)
    want = C.linear_cross_entropy_grads(x, w, targets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bufs = [torch.empty_like(t) for t in want]
    C.mhc_cross_entropy_grads(x, w, targets, bufs[0], bufs[1], grad_x=bufs[2], grad_weight=bufs[3], stream=side)
    side.synchronize()
    for p, q in zip(bufs, want):
        assert R.same_bytes(p, q)
    buf, at = x.clone(), targets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*C.linear_cross_entropy_grads(buf, w, at), *C.linear_cross_entropy(buf[:4], w, at[:4], reduction="none"))
        got += C.linear_cross_entropy_backward(buf, w, at, got[1])
    for k in range(4):
        new = (x * (k + 1)).contiguous()
        buf.copy_(new)
        at.copy_(targets.roll(k))
        graph.replay()
        torch.cuda.synchronize()
        now = targets.roll(k)
        want = (*C.linear_cross_entropy_grads(new, w, now), *C.linear_cross_entropy(new[:4], w, now[:4], reduction="none"))
        want += C.linear_cross_entropy_backward(new, w, now, want[1])
        for p, q in zip(got, want):
            assert R.same_bytes(p, q), k
