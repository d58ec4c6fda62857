"""The cross entropy (include/mhc_cross_entropy.h) where logits or gradients leave the
ordinary: infinite logits, finite ones so large that fp32 holds them in steps of 2 or
more, shares whose sum is what has to fit 16 bits.

Inputs are made so that every logit is exact in fp32 (products and their partial sums
are), so a probability is off by what its exponentials, sums and roundings cost alone:
`REL` for the chain of the forward's sums (see test_cross_entropy.py: fewer than 64 steps
of 8 u), half a step of fp16 where it was held there, then half a step of G's type and
of the gradient's. Where the formula gives NaN or an infinity, so does the kernel.
"""

from __future__ import annotations

import math

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from hyper_connection_residual_mhc_amd import _lib
from test_linear import LARGE, MEDIUM, ROWS, SMALL, STEP, additions

BF16, F16 = torch.bfloat16, torch.float16
SHORT = _lib.MHC_LINEAR_SHORT
TYPES = {"bf16": BF16, "f16": F16}
REL = 64 * 8 * R.U32
IGNORE = -100


def product(a, b):
    """a @ b by single products, so that 0 times an infinity is there as NaN."""
    return (a[:, :, None] * b[None]).sum(1)


def fp32(v):
    """fp64 values whose overflows are fp32's."""
    return torch.where(v.abs() > torch.finfo(torch.float32).max, torch.sign(v) * math.inf, v)


def formula(x, w, targets, s, e=None):
    """(lse, each row's loss, G, a p), fp64, of logits as fp32 has them."""
    z = product(x.double(), w.double().t())
    z = fp32(z)
    # from the largest on, since 64 bits hold 2.55e38 in steps of 2^75
    top = z.amax(1, keepdim=True)
    d = torch.where((z == top) & torch.isfinite(z), torch.zeros_like(z), z - top)
    some = torch.where(torch.isinf(top), torch.zeros_like(top), torch.log(torch.exp(d).sum(1, keepdim=True)))
    lse = (top + some)[:, 0]
    rows = torch.arange(len(x))
    each = torch.where(targets != IGNORE, some[:, 0] - (z - top)[rows, targets.clamp(0)], torch.zeros_like(lse))
    each = fp32(torch.where(torch.isinf(lse) & (targets != IGNORE), lse - z[rows, targets.clamp(0)], each))
    a = s if e is None else s + e
    ap = a[:, None] * torch.exp(d - some)
    g = ap.clone()
    g[rows, targets.clamp(0)] -= s
    g[(a == 0) & (s == 0)] = 0
    return lse, each, g, ap


def check(got, x, w, g, ap, t, held, a_most):
    """(grad_x, grad_weight) against G's products."""
    xv, wv = x.double(), w.double()
    rel = REL + (R.HALF_STEP[F16] if held else 0)
    # fp16 shares are scaled to 2^13 at least, so that next to zero G is off by half of its smallest number over that
    dg = ap.abs() * rel + (g.abs() + ap.abs() * rel) * R.HALF_STEP[t] + R.HALF_TINY[t] * (a_most * 2.0 ** -13 if t == F16 else 1)
    dg = torch.nan_to_num(dg)
    if held:
        dg = dg + ap.nan_to_num().abs().amax(1, keepdim=True) * 2.0 ** -40
    clean = lambda v: torch.nan_to_num(v, posinf=0.0, neginf=0.0)  # noqa: E731
    for name, out, want, left, right, dl in (
            ("grad_x", got[0], product(g, wv), g, wv, dg), ("grad_weight", got[1], product(g.t(), xv), g.t(), xv, dg.t())):
        size = clean(left).abs() @ clean(right).abs()
        tol = dl @ clean(right).abs() + size * additions(left.shape[1], 32) * STEP
        # half a step past the type's largest number (3.39e38 in bf16) a value is an infinity
        past = want.abs() >= torch.finfo(t).max * (1 + torch.finfo(t).eps / 4)
        want = torch.where(past, torch.sign(want) * math.inf, want)
        # terms that together pass fp32's largest number have partial sums that may, whatever they come to: 1.33 p 3e38 over
        # all other columns is 3.9e38, which the target's column takes back
        any_value = (size > torch.finfo(torch.float32).max) & torch.isfinite(want)
        out = torch.where(any_value, want, out.double().cpu())
        R.assert_within(out, want, tol + R.rounding(clean(want).abs() + tol, t), name)


def calls(device, x, w, targets, s, kernel, lse=None):
    """The loss and its gradients in one call, and the gradients from lse (the forward's unless given)."""
    from hyper_connection_residual_mhc_amd import loss as C
    x, w, targets, s = x.to(device), w.to(device), targets.to(device), s.float().to(device)
    value, made = torch.empty(len(x), device=device), torch.empty(len(x), device=device)
    gx, gw, bx, bw = torch.empty_like(x), torch.empty_like(w), torch.empty_like(x), torch.empty_like(w)
    launch = {"kernel": kernel} if kernel else None
    C.mhc_cross_entropy_grads(x, w, targets, value, made, s, grad_x=gx, grad_weight=gw, reduction="none", launch=launch)
    C.mhc_cross_entropy_bwd(x, w, targets, made if lse is None else lse.to(device), s, grad_x=bx, grad_weight=bw, reduction="none",
                            launch=None if kernel == ROWS else launch)
    torch.cuda.synchronize()
    return value, made, (gx, gw), (bx, bw)


KERNELS = [ROWS, SHORT, SMALL, MEDIUM, LARGE]


# ---------------------------------------------------------------------------
# Infinite logits
# ---------------------------------------------------------------------------

def infinite(kind, case, M, V):
    """x, W, targets, s. `above`: two logits of row 0 are inf, its target one of them; of row 1 the target alone; of row 2
    one that is not its target; a row that counts for nothing has some as well. `below`: all of row 0 is -inf, of row 1
    its target alone. `nan`: row 0; one logit of row 1 is inf, all others are NaN."""
    x, w = torch.zeros(M, 8, dtype=TYPES[kind]), torch.zeros(V, 8, dtype=TYPES[kind])
    x[:, 3] = torch.arange(M) % 3 - 1.0
    w[:, 3] = torch.arange(V) % 5 * 0.5
    targets = torch.arange(M) % V
    s = torch.linspace(0.5, 1.5, M, dtype=torch.float64)
    s[::2] *= -1
    # bf16 overflows in the product; fp16 has infinities in x, times values that are not 0
    high = 3e38 if kind == "bf16" else 1.0
    if case == "above" and kind == "bf16":
        w[[1, V - 1], 0], x[0, 0] = high, high
        w[4, 1], x[1, 1], x[2, 1], x[M - 1, 1] = high, high, high, high
        targets[0], targets[1], targets[2], targets[M - 1] = V - 1, 4, 3, IGNORE
    elif case == "above":
        # an infinity in W meets every row: +inf in rows 0, 1 and the last, -inf in the others
        w[4, 0] = math.inf
        x[:, 0] = -1
        x[[0, 1, M - 1], 0] = 1
        targets[0], targets[1], targets[M - 1] = 4, 2, IGNORE
    elif case == "below":
        w[:, 2], x[0, 2] = (-high, high) if kind == "bf16" else (1.0, -math.inf)
        if kind == "bf16":
            w[5, 1], x[1, 1] = -high, high
            targets[1] = 5
    else:
        x[0, 5], x[1, 5], w[3, 5] = math.nan, math.inf, 1.0
    return x, w, targets, s


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", ["above", "below", "nan"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinite_logits_have_the_formula_s_gradients(device, kind, case, kernel):
    """NaN where z - lse has no value, in G's own places and in both calls alike; a row that counts for nothing stays 0."""
    for M, V in ((7, 12), (7, 150)) if kernel == ROWS else ((70, 150), (40, 300)):
        say(f"infinite logits {kind} {case} kernel={kernel} M={M} V={V}")
        x, w, targets, s = infinite(kind, case, M, V)
        s = torch.where(targets == IGNORE, torch.zeros_like(s), s)
        lse, each, g, ap = formula(x, w, targets, s)
        value, made, one, two = calls(device, x, w, targets, s, kernel)
        R.assert_within(made, lse, lse.abs().nan_to_num(posinf=0) * 4 * R.U32 + REL, "lse")
        R.assert_within(value, each, each.abs().nan_to_num(posinf=0) * 4 * R.U32 + REL, "loss")
        assert torch.isnan(g).any()
        check(one, x, w, g, ap, w.dtype, True, 1.5)
        check(two, x, w, g, ap, w.dtype, False, 1.5)


# ---------------------------------------------------------------------------
# Finite logits of any size
# ---------------------------------------------------------------------------

def large(kind, k, sign, M, V):
    """Logits of 2^(24 + k) to 2^(25 + k), another in each row, and within a row apart by multiples of their own step."""
    x, w = torch.zeros(M, 8, dtype=TYPES[kind]), torch.zeros(V, 8, dtype=TYPES[kind])
    x[:, 0], w[:, 0] = (128.0 + torch.arange(M) * 37 % 128) * 32, sign * 2.0 ** (12 + k)
    x[:, 3], w[:, 3] = 2.0 ** (1 + k), -(torch.arange(V) * 7 % 13).float()
    targets = torch.arange(M) * 11 % V
    s = torch.linspace(0.5, 1.5, M, dtype=torch.float64)
    s[::2] *= -1
    return x, w, targets, s


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_large_logits(device, kind, kernel):
    """A row's probabilities are those of its differences, which are exact however large the logits are."""
    M, V = (16, 150) if kernel == ROWS else (100, 300)
    for k in range(4):
        for sign in (1, -1):
            say(f"large logits {kind} kernel={kernel} k={k} sign={sign}")
            x, w, targets, s = large(kind, k, sign, M, V)
            assert float(product(x.double(), w.double().t()).abs().max()) < 2.0 ** (26 + k)
            lse, each, g, ap = formula(x, w, targets, s)
            value, made, one, _ = calls(device, x, w, targets, s, kernel)
            R.assert_within(made, lse, lse.abs() * 2 * R.U32 + REL, "lse")
            R.assert_within(value, each, each.abs() * 4 * R.U32 + REL, "loss")
            check(one, x, w, g, ap, w.dtype, True, 1.5)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_logits_whose_product_with_log2_e_has_no_place_in_fp32(device, kernel):
    M, V = (7, 150) if kernel == ROWS else (70, 150)
    say(f"logits of 2.55e38 kernel={kernel}")
    x, w = torch.zeros(M, 8, dtype=BF16), torch.zeros(V, 8, dtype=BF16)
    x[::2, 0], x[1::2, 0] = 2.0 ** 64, -2.0 ** 64
    w[::3, 0], w[1::5, 0] = 1.5 * 2.0 ** 63, -1.5 * 2.0 ** 63
    targets, s = torch.arange(M) * 3 % V, torch.linspace(0.5, 1.5, M, dtype=torch.float64)
    lse, each, g, ap = formula(x, w, targets, s)
    assert torch.isfinite(lse).all() and float(lse.max()) > 2.5e38
    value, made, one, two = calls(device, x, w, targets, s, kernel)
    R.assert_within(made, lse, lse.abs() * 2 * R.U32 + REL, "lse")
    R.assert_within(value, each, each.abs() * 4 * R.U32 + REL, "loss")
    check(one, x, w, g, ap, BF16, True, 1.5)


# ---------------------------------------------------------------------------
# Shares
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -13, 512.0])
def test_a_target_s_two_shares_of_opposite_signs(device, kind, factor):
    """At its target a row's G is a p - s with a = s + grad_lse: as large as both together where they differ in sign."""
    from hyper_connection_residual_mhc_amd import loss as C
    M, V, t = 40, 150, TYPES[kind]
    x, w = torch.zeros(M, M + 1, dtype=t), torch.zeros(V, M + 1, dtype=t)
    targets = torch.arange(M) * 11 % V
    rows = torch.arange(M)
    x[rows, rows], w[targets, rows] = 8.0, 8.0             # each target's probability is nearly 1
    x[:, M], w[:, M] = rows % 3 - 1.0, torch.arange(V) % 5 * 0.25
    for s0, e0 in ((-1.9999, 3.9998), (1.9999, -3.9998), (1.0, -1.0), (0.0, 1.9999)):
        say(f"shares {kind} s={s0 * factor} grad_lse={e0 * factor}")
        s = (torch.linspace(0.25, 1.0, M) * s0 * factor).float()
        e = (torch.linspace(0.25, 1.0, M) * e0 * factor).float()
        lse, _, g, ap = formula(x, w, targets, s.double(), e.double())
        gx, gw = torch.empty_like(x, device=device), torch.empty_like(w, device=device)
        C.mhc_cross_entropy_bwd(x.to(device), w.to(device), targets.to(device), lse.float().to(device), s.to(device),
                                grad_lse=e.to(device), grad_x=gx, grad_weight=gw, reduction="none")
        torch.cuda.synchronize()
        check((gx, gw), x, w, g, ap, t, False, 4 * factor)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS[1:])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_no_probability_passes_1(device, kind, kernel):
    """From lse, which is rounded: below the largest logit by up to half its step, where exp(z - lse) would be e^(1/2) and
    more, which in fp16's scale is an infinity."""
    M, V = 100, 300
    for k in range(4):
        say(f"large logits from lse {kind} kernel={kernel} k={k}")
        x, w, targets, s = large(kind, k, 1, M, V)
        w[1:, 3] -= 13.0                                   # one logit is ahead of all others
        z = product(x.double(), w.double().t())
        for lse in (torch.logsumexp(z, 1).float(), z.amax(1).float() - 2.0 ** (1 + k)):
            ap = s[:, None] * torch.exp((z - lse.double()[:, None]).clamp(max=0.0))
            g = ap.clone()
            g[torch.arange(M), targets] -= s
            *_, two = calls(device, x, w, targets, s, kernel, lse)
            check(two, x, w, g, ap, w.dtype, False, 1.5)


# ---------------------------------------------------------------------------
# Rows that are no whole pieces
# ---------------------------------------------------------------------------

def test_the_loss_of_few_rows_copies_no_weight(built_library):
    """The loss alone, a few rows, K no multiple of 8: its workspace is that of a K that is one."""
    from hyper_connection_residual_mhc_amd import loss as C
    for M, V, K in ((1, 131072, 8191), (2, 131072, 8191), (8, 65536, 7161), (16, 65536, 7167), (17, 65536, 7167), (300, 131072, 4095)):
        odd = C.mhc_cross_entropy_workspace_bytes("fwd", M, V, K, 1)
        assert odd == C.mhc_cross_entropy_workspace_bytes("fwd", M, V, -(-K // 8) * 8, 1), (M, V, K)
        assert odd < V * K * 2 // 32
    # with gradients, and of many rows, the copies pay
    assert C.mhc_cross_entropy_workspace_bytes("grads", 16, 65536, 7167, 1) > 65536 * 7168 * 2
    assert C.mhc_cross_entropy_workspace_bytes("fwd", 1024, 65536, 7167, 1) > 65536 * 7168 * 2


def test_workspaces_are_what_the_header_says(built_library):
    """One chunk of G, and from the second on the weight's gradient in fp32 as well, however many rows."""
    from hyper_connection_residual_mhc_amd import loss as C
    V, K, gib = 131072, 4096, 2.0 ** 30
    of = {M: [C.mhc_cross_entropy_workspace_bytes(call, M, V, K, 1) / gib for call in ("fwd", "bwd", "grads")]
          for M in (4096, 4097, 8192, 65536, 1 << 20)}
    assert of[4096] == pytest.approx([0.0625, 1.0, 1.0625], abs=0.001)
    assert of[4097][2] == pytest.approx(2.74, abs=0.01)
    for M in (8192, 65536, 1 << 20):
        assert of[M][0] < 0.07 and 3.0 <= of[M][1] < 3.1 and 3.0 < of[M][2] < 3.1


@pytest.mark.gpu
@pytest.mark.parametrize("M,V,K", [(8, 100000, 2047), (16, 50000, 2047), (130, 20000, 1023), (600, 12000, 1023)])
def test_the_loss_alone_and_with_gradients_agree(device, M, V, K):
    """Bit for bit, also where W is copied for the gradients and not for the loss alone."""
    from hyper_connection_residual_mhc_amd import loss as C
    from test_cross_entropy import check_loss
    assert C.mhc_cross_entropy_workspace_bytes("grads", M, V, K, 1) > V * (K + 1) * 2
    say(f"cross entropy of rows that are no whole pieces M={M} V={V} K={K}")
    gen = torch.Generator(device=device).manual_seed(M)
    x, w = (torch.randn(r, K, device=device, generator=gen) for r in (M, V))
    x, w, targets = x.to(BF16), (w * 2 * K ** -0.5).to(BF16), torch.randint(V, (M,), device=device, generator=gen)
    f, o = C.linear_cross_entropy(x, w, targets), C.linear_cross_entropy_grads(x, w, targets)
    assert R.same_bytes(f.loss, o.loss) and R.same_bytes(f.lse, o.lse)
    check_loss(f.loss, f.lse, x.double(), w.double(), targets, "mean", IGNORE)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_the_factor_of_all_rows_is_not_in_g_s_rounding(device, kind, reduction):
    """256 equal logits: p = 2^-8 and p - 1 = -255/256 are numbers of 8 bits, so that G without its rows' factor is exact,
    and the gradients are off by their sums and their own rounding alone, whatever 1 / C or grad_loss are."""
    from hyper_connection_residual_mhc_amd import loss as C
    t, M, V, K = TYPES[kind], 130, 256, 72
    gen = torch.Generator().manual_seed(7)
    targets = torch.arange(M) * 11 % V
    targets[M - 10:] = IGNORE                              # C = 120: 1 / C is 0.0034 off in bf16
    rows = torch.arange(M)
    on = (targets != IGNORE).double()
    for factor in (None, 1.0 / 3.0, -120.0 / 3870.0):
        for x, w in ((torch.zeros(M, K, dtype=t), R.normal(gen, V, K, dtype=t)), (R.normal(gen, M, K, dtype=t), torch.zeros(V, K, dtype=t))):
            say(f"common factor {kind} {reduction} {factor}")
            g = None if factor is None else torch.tensor(factor, device=device)
            s = on * (1.0 if factor is None else float(g.cpu().double()))
            s = s / on.sum() if reduction == "mean" else s
            G = s[:, None].repeat(1, V) / V
            G[rows, targets.clamp(0)] -= s
            o = C.linear_cross_entropy_grads(x.to(device), w.to(device), targets.to(device), g, reduction=reduction)
            two = C.linear_cross_entropy_backward(x.to(device), w.to(device), targets.to(device), o.lse, g, reduction=reduction)
            xv, wv = x.double(), w.double()
            for got in ((o.grad_x, o.grad_weight), two):
                for p, want, size, long in ((got[0], G @ wv, G.abs() @ wv.abs(), V), (got[1], G.t() @ xv, G.t().abs() @ xv.abs(), M)):
                    tol = size * (additions(long, 32) + 4) * STEP
                    R.assert_within(p, want, tol + R.rounding(want.abs() + tol, t), "gradient")


@pytest.mark.gpu
def test_a_mean_of_large_rows_has_sums_of_its_own_size(device):
    """Rows of 2^126 with one target: their mean is finite where their sum is not, and the products sum it as a mean."""
    from hyper_connection_residual_mhc_amd import loss as C
    M, V, K = 70, 40, 16
    x, w = torch.zeros(M, K, dtype=BF16), torch.zeros(V, K, dtype=BF16)
    x[:, 3] = 2.0 ** 126
    targets = torch.full((M,), 5)
    o = C.linear_cross_entropy_grads(x.to(device), w.to(device), targets.to(device))
    gx, gw = C.linear_cross_entropy_backward(x.to(device), w.to(device), targets.to(device), o.lse)
    want = torch.zeros(V, K, dtype=torch.float64)
    want[:, 3] = 2.0 ** 126 / V
    want[5, 3] -= 2.0 ** 126
    # p and p - 1 are rounded to bf16 each, then the mean itself
    tol = want.abs() * (2 * R.HALF_STEP[BF16] + REL)
    for got in (o.grad_weight, gw):
        R.assert_within(got, want, tol, "grad_weight")
    assert not o.grad_x.any() and not gx.any()
