"""The write-back into the residual streams (include/mhc_post.h) against its
fp64 form, forward and backward, and the rules of the call.

Tolerances (u = 2^-24): a forward element is one product and n fused steps, so
at most (n + 1) u of the sum of its terms' magnitudes, then one rounding to
bf16; a gradient over the streams likewise. A sum over h is a chain of at most
8 * ceil(H / (8 * threads)) fused steps, 6 tree steps and 3 joins.
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

BF16 = torch.bfloat16
WIDTHS = [1, 7, 8, 33, 511, 512, 513, 1024, 1279, 2048, 2056, 4096, 7168, 20001]


def chain(H: int) -> int:
    threads = next((t for t in (64, 128) if H <= 8 * t), 256)
    return 8 * math.ceil(H / (8 * threads)) + 6 + 3


def make(T, n, H, seed):
    gen = torch.Generator().manual_seed(seed)
    comb = torch.softmax(torch.randn(T, n, n, generator=gen), 2)
    gate = 2 * torch.sigmoid(torch.randn(T, n, generator=gen))
    return (R.normal(gen, T, n, H, scale=0.5), R.normal(gen, T, n, H), comb, gate, R.normal(gen, T, H))


def check_forward(out, r, comb, gate, y):
    n = r.shape[1]
    want = R.post(*map(R.d, (r, comb, gate, y)))
    size = R.post(*(R.d(t).abs() for t in (r, comb, gate, y)))
    tol = size * (n + 1) * R.U32
    R.assert_within(out, want, tol + R.rounding(want.abs() + tol, BF16), "out")


def check_backward(grads, g, r, comb, gate, y):
    n, H = r.shape[1:]
    want = R.post_grads(*map(R.d, (g, r, comb, gate, y)))
    size = R.post_grads(*(R.d(t).abs() for t in (g, r, comb, gate, y)))
    for k, name in enumerate(("grad_residual", "grad_comb", "grad_post", "grad_y")):
        if name in ("grad_comb", "grad_post"):
            R.assert_within(grads[k], want[k], size[k] * chain(H) * R.U32 + 2.0 ** -140, name)
        else:
            tol = size[k] * n * R.U32
            R.assert_within(grads[k], want[k], tol + R.rounding(want[k].abs() + tol, BF16), name)


def test_formula_gradients_are_the_differences_of_the_forward():
    gen = torch.Generator().manual_seed(3)
    T, n, H = 2, 4, 5
    leaves = [torch.randn(s, generator=gen, dtype=torch.float64) for s in ((T, n, H), (T, n, n), (T, n), (T, H))]
    g = torch.randn(T, n, H, generator=gen, dtype=torch.float64)
    grads = R.post_grads(g, *leaves)
    for leaf, grad in zip(leaves, grads):
        # the forward is linear in each leaf: only rounding of the differences is left
        assert torch.allclose(grad, R.differences(lambda: (R.post(*leaves) * g).sum(), leaf), rtol=0, atol=1e-8)


BASE = 1 << 36
GAP = 1 << 30


@pytest.fixture(scope="module")
def lib(built_library):
    return _lib.post_lib()


def fwd_args(**kw):
    a = dict(residual=BASE, comb=BASE + GAP, post=BASE + 2 * GAP, y=BASE + 3 * GAP, out=BASE + 4 * GAP, T=5, n=4, H=40)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(grad_out=BASE, residual=BASE + GAP, comb=BASE + 2 * GAP, post=BASE + 3 * GAP, y=BASE + 4 * GAP,
             grad_residual=BASE + 5 * GAP, grad_comb=BASE + 6 * GAP, grad_post=BASE + 7 * GAP, grad_y=BASE + 8 * GAP,
             T=5, n=4, H=40)
    a.update(kw)
    return list(a.values())


def test_arguments(lib):
    f, b = lib.mhc_post_validate_fwd, lib.mhc_post_validate_bwd
    for n in (2, 4, 8):
        assert f(*fwd_args(n=n)) == MHC_SUCCESS and b(*bwd_args(n=n)) == MHC_SUCCESS
    none = {k: None for k in ("residual", "comb", "post", "y")}
    assert f(*fwd_args(T=0, out=None, **none)) == MHC_SUCCESS
    for kw in ({"n": 3}, {"n": 0}, {"T": -1}, {"H": 0}, {"H": (1 << 26) + 1}, {"T": 1 << 60}, {"residual": None},
               {"comb": None}, {"y": BASE + 3 * GAP + 1}, {"comb": BASE + GAP + 2}):
        assert f(*fwd_args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
        assert lib.mhc_post_last_error_message() != b""
        if "residual" not in kw:
            assert b(*bwd_args(**kw)) == MHC_ERROR_INVALID_VALUE, kw
    for name in ("grad_out", "residual", "grad_residual", "grad_comb", "grad_post", "grad_y"):
        assert b(*bwd_args(**{name: None})) == MHC_ERROR_INVALID_VALUE
    for kw in ({"out": BASE}, {"out": BASE + 1598}, {"out": BASE + GAP}, {"out": BASE + 3 * GAP}):
        assert f(*fwd_args(**kw)) == MHC_ERROR_ALIASING, kw
    for kw in ({"grad_residual": BASE}, {"grad_y": BASE + 5 * GAP}, {"grad_comb": BASE + 7 * GAP}):
        assert b(*bwd_args(**kw)) == MHC_ERROR_ALIASING, kw


def test_python_refusals(built_library):
    from hyper_connection_residual_mhc_amd import post
    _, r, comb, gate, y = make(2, 4, 8, 0)
    with pytest.raises(TypeError):
        post.post_update(r, comb, gate, y)                 # not on a GPU
    with pytest.raises(ValueError):
        post.post_update(r[:, :3], comb, gate, y)


@pytest.mark.gpu
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("n", [2, 4, 8])
def test_widths(device, n, H):
    from hyper_connection_residual_mhc_amd import post
    say(f"write-back n={n} H={H}")
    host = make(3, n, H, seed=H + n)
    g, *rest = (t.to(device) for t in host)
    out = post.post_update(*rest)
    grads = post.post_update_backward(g, *rest)
    torch.cuda.synchronize()
    check_forward(out, *host[1:])
    check_backward(grads, *host)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 2, 300, 1025])
def test_batches_and_row_bytes(device, T):
    from hyper_connection_residual_mhc_amd import post
    host = tuple(t[:T] for t in make(max(T, 1), 4, 520, seed=T))
    g, *rest = (t.to(device) for t in host)
    out, grads = post.post_update(*rest), post.post_update_backward(g, *rest)
    check_forward(out, *host[1:])
    check_backward(grads, *host)
    for t in {0, T // 2, T - 1} if T else ():
        one = [x[t:t + 1] for x in rest]
        assert R.same_bytes(out[t:t + 1], post.post_update(*one))
        for a, b in zip(grads, post.post_update_backward(g[t:t + 1], *one)):
            assert R.same_bytes(a[t:t + 1], b)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1279, 2056])
def test_alignment_and_edges(device, H):
    from hyper_connection_residual_mhc_amd import post
    T, n = 5, 4
    host = make(T, n, H, seed=H)
    g, *rest = (t.to(device) for t in host)
    out, grads = post.post_update(*rest), post.post_update_backward(g, *rest)
    moved = [R.shifted(t, device) for t in host]
    assert R.same_bytes(out, post.post_update(*moved[1:]))
    for a, b in zip(grads, post.post_update_backward(*moved)):
        assert R.same_bytes(a, b)
    for fill in (0xA5, 0x3C):
        o = R.Guarded((T, n, H), BF16, device, fill)
        b = [R.Guarded(tuple(t.shape), t.dtype, device, fill) for t in grads]
        post.mhc_post_fwd(*rest, o.t)
        post.mhc_post_bwd(g, *rest, *(x.t for x in b))
        assert o.untouched() and R.same_bytes(o.t, out)
        for x, want in zip(b, grads):
            assert x.untouched() and R.same_bytes(x.t, want)


@pytest.mark.gpu
def test_infinities_stay_in_their_token(device):
    from hyper_connection_residual_mhc_amd import post
    host = list(make(4, 4, 40, seed=1))
    host[1][1, 2, 3] = float("inf")
    host[4][2, 5] = float("nan")
    g, *rest = (t.to(device) for t in host)
    out, grads = post.post_update(*rest), post.post_update_backward(g, *rest)
    for t in (out, *grads):
        assert torch.isfinite(t[0].float()).all() and torch.isfinite(t[3].float()).all()
    assert torch.isinf(out[1, :, 3].float()).all() and torch.isfinite(out[1, :, :3].float()).all()
    assert torch.isnan(out[2, :, 5].float()).all() and torch.isnan(grads[2][2]).all()


@pytest.mark.gpu
def test_autograd_streams_and_graphs(device):
    from hyper_connection_residual_mhc_amd import post
    g, *rest = (t.to(device) for t in make(65, 4, 1288, seed=2))
    want = (post.post_update(*rest), *post.post_update_backward(g, *rest))
    leaves = [t.clone().requires_grad_() for t in rest]
    out = post.post_update_autograd(*leaves)
    got = (out, *torch.autograd.grad(out, leaves, g))
    for a, b in zip(got, want):
        assert R.same_bytes(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bufs = [torch.empty_like(t) for t in want]
    post.mhc_post_fwd(*rest, bufs[0], stream=side)
    post.mhc_post_bwd(g, *rest, *bufs[1:], stream=side)
    side.synchronize()
    for a, b in zip(bufs, want):
        assert R.same_bytes(a, b)
    y = rest[3].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (post.post_update(*rest[:3], y), *post.post_update_backward(g, *rest[:3], y))
    for k in range(4):
        y.copy_(rest[3] * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        new = [*rest[:3], (rest[3] * (k + 1)).contiguous()]
        for a, b in zip(got, (post.post_update(*new), *post.post_update_backward(g, *new))):
            assert R.same_bytes(a, b), k
