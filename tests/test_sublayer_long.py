"""The sublayer's operators at sizes where their kernels loop: blocks that take
several rows, launches with fewer blocks than pieces of work, sums in many
parts, calls that read past the cache, operands that are copied first.

Tolerances as in the operators' own tests (u = 2^-24); what an operator gives
row by row is compared byte for byte with the same rows in small calls."""

from __future__ import annotations

import math

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from hyper_connection_residual_mhc_amd import _lib

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
STEP = 2.0 ** -23
ABI = {"bf16": 1, "f16": 2, "row": 3, "mx": 4}
LARGE = 5
BLOCKS = 1 << 20                       # of a launch, at most


def raw(t: torch.Tensor) -> torch.Tensor:
    return t.contiguous().view(torch.uint8)


def same(a: torch.Tensor, b: torch.Tensor) -> bool:
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(raw(a), raw(b))


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def parts_and_rows(T: int, H: int) -> tuple[int, int]:
    """(parts of the weight gradient's sum, rows in each) by the workspace that the call asks for."""
    need = _lib.norm_lib().mhc_rms_norm_bwd_workspace_bytes(T, H)
    assert need % (4 * H) == 0
    parts = need // (4 * H)
    return parts, math.ceil(T / parts)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,dtype,least_rows,least_parts", [
    (5200, 264, BF16, 6, 1024), (3100, 520, F32, 4, 1024), (2000, 2056, F16, 4, 512), (1500, 7168, BF16, 6, 256),
    (1031, 8192, F32, 5, 256), (100, 8200, BF16, 25, 4), (65, 8200, F32, 22, 3), (70, 16384, F16, 24, 3),
    (101, 16385, BF16, 26, 4),
])
def test_norm_backward_over_many_rows(device, T, H, dtype, least_rows, least_parts):
    """Blocks with three and more rows, and weight gradients of many parts."""
    from hyper_connection_residual_mhc_amd import norm
    say(f"norm backward T={T} H={H} {dtype}")
    parts, rows = parts_and_rows(T, H)
    assert parts >= least_parts and rows >= min(least_rows, 3)
    gen = torch.Generator(device=device).manual_seed(T)
    r = lambda *s: torch.randn(s, device=device, generator=gen)  # noqa: E731
    s, g, gs = r(T, H).to(dtype), (0.5 * r(T, H)).to(dtype), r(T, H).to(dtype)
    w = (1 + 0.2 * r(H)).to(dtype if T % 2 else F32)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    gx, gw = norm.rms_norm_backward(g, s, w, rstd, grad_stored=gs)
    sd, gd, wd, rd = s.double(), g.double(), w.double(), rstd.double()
    want_x, want_w = R.norm_grads(gd, sd, wd, rd, gs.double())
    u = (gd * wd).abs()
    # a row's sum: 8 fused steps for each chunk of a thread, trees and joins (at most 31 and 7 more)
    length = 8 * math.ceil(H / 512 / 8) + 38
    dot = (u * sd.abs()).mean(1, keepdim=True) * rd[:, None] ** 2
    tol = rd[:, None] * (5 * u + (length + 8) * sd.abs() * dot) * R.U32 + want_x.abs() * R.U32
    tol = tol + (want_x.abs() + tol) * R.HALF_STEP[dtype] + R.HALF_TINY[dtype]
    assert float(((gx.double() - want_x).abs() - tol).max()) <= 0
    # a column: a product, a fused step for each row of a part (32 at least are planned for long rows), and the parts:
    # every 64th in turn, then 8 and 8
    steps = 1 + max(rows, 32) + math.ceil(parts / 64) + 16
    tol = (gd * sd * rd[:, None]).abs().sum(0) * steps * R.U32 + 2.0 ** -140
    assert float(((gw.double() - want_w).abs() - tol).max()) <= 0
    # a row's bytes do not depend on the batch
    for t in (0, T // 2, T - 1):
        one = norm.rms_norm_backward(g[t:t + 1], s[t:t + 1], w, rstd[t:t + 1], grad_stored=gs[t:t + 1])[0]
        assert same(one, gx[t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("source", ["plain", "streams"])
@pytest.mark.parametrize("H", [8, 520])
def test_norm_forward_of_more_rows_than_blocks(device, H, source):
    from hyper_connection_residual_mhc_amd import norm
    T, base, n = BLOCKS + 37, 997, 2
    say(f"norm forward T={T} H={H} {source}")
    gen = torch.Generator(device=device).manual_seed(H)
    shape = (base, n, H) if source == "streams" else (base, H)
    x = torch.randn(shape, device=device, generator=gen).to(BF16)
    pre = torch.rand((base, n), device=device, generator=gen) if source == "streams" else None
    w = torch.rand(H, device=device, generator=gen) + 0.5
    rows = torch.arange(T, device=device) % base
    for quant in (None, "row", "mx"):
        few = norm.rms_norm(x, w, pre=pre, quant=quant, return_rstd=True)
        many = norm.rms_norm(x[rows], w, pre=None if pre is None else pre[rows], quant=quant, return_rstd=True)
        for a, b in zip(few, many):
            if a is not None:
                assert torch.equal(raw(a).view(base, -1)[rows], raw(b).view(T, -1)), quant


# ---------------------------------------------------------------------------
# Write-back
# ---------------------------------------------------------------------------

def make_post(T, n, H, device, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, device=device, generator=gen)  # noqa: E731
    return (r(T, n, H).to(BF16), r(T, n, H).to(BF16), torch.softmax(r(T, n, n), 2), 2 * torch.sigmoid(r(T, n)),
            r(T, H).to(BF16))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 4, 8])
@pytest.mark.parametrize("H", [500, 1031, 2056, 7175])
def test_write_back_past_the_cache(device, n, H):
    """Calls that read over 256 MiB read in another way; the bytes are those of small calls, which are compared with
    fp64 in the operator's own tests."""
    from hyper_connection_residual_mhc_amd import post
    T = (256 << 20) // (2 * H * (n + 1)) + 5
    say(f"write-back T={T} n={n} H={H}")
    g, *rest = make_post(T, n, H, device, H + n)
    out = post.post_update(*rest)
    grads = post.post_update_backward(g, *rest)
    step = T // 3 + 1
    assert step * H * 2 * (2 * n + 1) < 256 << 20 < T * H * 2 * (n + 1)
    for t in range(0, T, step):
        part = [x[t:t + step] for x in rest]
        assert same(post.post_update(*part), out[t:t + step])
        for a, b in zip(post.post_update_backward(g[t:t + step], *part), grads):
            assert same(a, b[t:t + step])


@pytest.mark.gpu
def test_write_back_of_more_tokens_than_blocks(device):
    from hyper_connection_residual_mhc_amd import post
    T, base, n, H = BLOCKS + 37, 997, 2, 8
    g, *rest = make_post(base, n, H, device, 3)
    rows = torch.arange(T, device=device) % base
    few = (post.post_update(*rest), *post.post_update_backward(g, *rest))
    many_rest = [x[rows] for x in rest]
    many = (post.post_update(*many_rest), *post.post_update_backward(g[rows], *many_rest))
    for a, b in zip(few, many):
        assert torch.equal(raw(a).view(base, -1)[rows], raw(b).view(T, -1))


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------

def additions(K: int, wide: int) -> int:
    """Additions that a term of a sum over K goes through, at most."""
    return wide + math.ceil(K / wide) + 64 + 16


def within(got, want, size, length, kind, t, more=0.0):
    tol = size * (additions(length, 128 if kind in ("row", "mx") else 32) + 6) * STEP + more
    if kind in ("row", "mx"):
        tol = tol + size * 7 * 2.0 ** -13                  # at most the largest product of each 8, so at most their sum
    tol = tol + (want.abs() + tol) * R.HALF_STEP[t] + R.HALF_TINY[t]
    over = (got.double() - want).abs() - tol
    assert float(over.max()) <= 0, int((over > 0).sum())


def padded(kind: str, M: int, N: int, K: int) -> int:
    """Bytes of the workspace that hold copies of the operands in whole rows."""
    whole = {"bf16": 8, "f16": 8, "row": 16, "mx": 128}[kind]
    size = 1 if kind in ("row", "mx") else 2
    ld = -(-K // whole) * whole * size
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    return up(M * ld) + up(N * ld) + (up(M * ld // 32) + up(N * ld // 32) if kind == "mx" else 0)


# past the border in terms, in rows and in columns: odd rows and columns, last pieces of 1 to 31 elements
COPIED = [(513, 8191, 1593), (6501, 512, 2047), (2050, 1700, 1999), (1601, 1503, 2721)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
def test_which_operands_are_copied(built_library, kind):
    """The workspace holds the copies at exactly the sizes past the border, and the split sums beside them."""
    from hyper_connection_residual_mhc_amd import linear as L

    def copies(M, N, K):
        splits = L.mhc_linear_plan(M, N, K, ABI[kind])["splits"]
        sums = -(-M * N * 4 * splits // 256) * 256 if splits > 1 else 0
        return L.mhc_linear_fwd_workspace_bytes(M, N, K, ABI[kind]) - sums

    for M, N, K in COPIED:
        assert copies(M, N, K) == padded(kind, M, N, K), (M, N, K)
    # rows of whole pieces: for block scales those are 128 elements
    assert copies(2050, 1700, 2048) == 0
    assert copies(2050, 1700, 2080) == (padded(kind, 2050, 1700, 2080) if kind == "mx" else 0)
    # fewer than 512 rows or columns, and fewer terms than 3 * 2^31
    for M, N, K in ((511, 16383, 1593), (16383, 511, 1593), (1100, 1300, 1593), (2050, 700, 1999)):
        assert copies(M, N, K) == 0, (M, N, K)
    assert 2048 * 1537 * 2047 > 3 << 31 > 2048 * 1536 * 2047
    assert copies(2048, 1537, 2047) > 0 and copies(2048, 1536, 2047) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
@pytest.mark.parametrize("M,N,K", COPIED)
def test_product_of_copied_operands(device, kind, M, N, K):
    """fp64 on the GPU; nothing outside out and the workspace is written, and with a named launch of one part a row's
    bytes are those of a call of few rows, whose operands are not copied."""
    from hyper_connection_residual_mhc_amd import linear as L
    say(f"copied operands {kind} M={M} N={N} K={K}")
    gen = torch.Generator().manual_seed(M)
    x, w = torch.randn(M, K, generator=gen), torch.randn(N, K, generator=gen) * K ** -0.5
    xs = ws = None
    t = F16 if kind == "f16" else BF16
    if kind in ("row", "mx"):
        (x, xs), (w, ws) = R.quantise(x, kind), R.quantise(w, kind)
        xv, wv = R.dequantise(x, xs).to(device), R.dequantise(w, ws).to(device)
        xs, ws = xs.to(device), ws.to(device)
    else:
        x, w = x.to(t), w.to(t)
        xv, wv = x.to(device).double(), w.to(device).double()
    x, w = x.to(device), w.to(device)
    out = R.Guarded((M, N), t, device)
    space = R.Guarded((L.mhc_linear_fwd_workspace_bytes(M, N, K, ABI[kind]),), torch.uint8, device, 0xFF)
    L.mhc_linear_fwd(x, w, out.t, x_scales=xs, weight_scales=ws, workspace=space.t)
    assert out.untouched() and space.untouched()
    within(out.t, xv @ wv.t(), xv.abs() @ wv.abs().t(), K, kind, t)
    launch = {"kernel": LARGE, "splits": 1}
    everything = torch.empty(M, N, dtype=t, device=device)
    L.mhc_linear_fwd(x, w, everything, x_scales=xs, weight_scales=ws, launch=launch)
    few = torch.empty(3, N, dtype=t, device=device)
    at = M - 3
    L.mhc_linear_fwd(x[at:], w, few, x_scales=None if xs is None else xs[at:], weight_scales=ws, launch=launch)
    assert same(few, everything[at:])


@pytest.mark.gpu
def test_join_of_more_results_than_threads(device):
    from hyper_connection_residual_mhc_amd import linear as L
    M, N, K = 3001, 3005, 512
    assert M * -(-N // 8) > 16384 * 64
    gen = torch.Generator(device=device).manual_seed(1)
    x, w = (torch.randn(s, device=device, generator=gen).to(BF16) for s in ((M, K), (N, K)))
    out = torch.empty(M, N, dtype=BF16, device=device)
    L.mhc_linear_fwd(x, w, out, launch={"kernel": LARGE, "splits": 3})
    within(out, x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t(), K, "bf16", BF16)


@pytest.mark.gpu
def test_zeros_of_more_elements_than_threads(device):
    from hyper_connection_residual_mhc_amd import linear as L
    N, K = 1101, 1003
    assert N * K > 4096 * 256
    x, g = torch.empty(0, K, dtype=BF16, device=device), torch.empty(0, N, dtype=BF16, device=device)
    gw = R.Guarded((N, K), BF16, device)
    L.mhc_linear_bwd(g, x, torch.ones(N, K, dtype=BF16, device=device), grad_weight=gw.t)
    assert gw.untouched() and not raw(gw.t).any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 16, 300, 2048])
def test_backward_of_few_columns_and_long_rows(device, kind, M):
    """The coefficients' product: 24 columns from 28672 values."""
    from hyper_connection_residual_mhc_amd import linear as L
    N, K, t = 24, 28672, BF16 if kind == "bf16" else F16
    say(f"backward {kind} M={M} N={N} K={K}")
    gen = torch.Generator(device=device).manual_seed(M)
    g, x, w = (torch.randn(s, device=device, generator=gen).to(t) for s in ((M, N), (M, K), (N, K)))
    gx, gw, gb = L.linear_backward(g, x, w, bias=True)
    gd, xd, wd = g.double(), x.double(), w.double()
    within(gx, gd @ wd, gd.abs() @ wd.abs(), N, kind, t)
    within(gw, gd.t() @ xd, gd.abs().t() @ xd.abs(), M, kind, t)
    within(gb, gd.sum(0), gd.abs().sum(0), M, kind, t)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [1, 2, 3, 4, LARGE])
@pytest.mark.parametrize("K", [256, 640, 200])
def test_scales_that_are_no_numbers(device, kernel, K):
    """A block scale of 255, which the norm writes for a block with an infinity, makes its row of x (its column, for a
    weight's) NaN and leaves the others alone."""
    from hyper_connection_residual_mhc_amd import linear as L
    M, N = (9, 40) if kernel == 1 else (70, 72)
    say(f"NaN scales kernel={kernel} K={K}")
    gen = torch.Generator().manual_seed(K)
    x, w = (torch.randn(r, K, generator=gen).to(E4M3).to(device) for r in (M, N))
    plain = [torch.full((r, -(-K // 32)), 127, dtype=torch.uint8, device=device) for r in (M, N)]
    marked = [s.clone() for s in plain]
    marked[0][4, -1] = 255
    marked[1][30, 1] = 255
    outs = []
    for xs, ws in (plain, marked):
        out = torch.empty(M, N, dtype=BF16, device=device)
        L.mhc_linear_fwd(x, w, out, x_scales=xs.view(torch.float8_e8m0fnu), weight_scales=ws.view(torch.float8_e8m0fnu),
                         launch={"kernel": kernel, "splits": 1})
        outs.append(out)
    rows, columns = torch.arange(M, device=device) != 4, torch.arange(N, device=device) != 30
    assert torch.isnan(outs[1][4]).all() and torch.isnan(outs[1][:, 30]).all()
    assert same(outs[0][rows][:, columns], outs[1][rows][:, columns])
