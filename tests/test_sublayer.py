"""The operators around a sublayer run together, as a model runs them: streams ->
collapse and norm -> product with activation -> product -> write-back, its
gradients through autograd, and the decoding form in 8 bits, each against the
same chain in plain PyTorch.

Tolerances are relative 2-norms. Every intermediate is rounded to bf16 (or
e4m3) once: a rounding is off by at most h = 2^-8 of each value (2^-4 in 8 bits), so by
at most h of the tensor's norm, and the chain below passes R such roundings one
after another, each carried on by operators whose gain the plain chain shares.
With independent roundings the result is off by about h sqrt(R / 3), and by h R in
the worst case; h R is what is allowed."""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
from gpu_util import say

BF16 = torch.bfloat16


def near(got: torch.Tensor, want: torch.Tensor, roundings: float, what: str) -> None:
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    off = float((got - want).norm() / want.norm())
    assert off <= roundings, f"{what}: {off:.3g} of the norm off, {roundings:.3g} allowed"


def make(T, n, H, F, seed, dev):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(s, generator=gen) * scale)  # noqa: E731
    return dict(streams=r(T, n, H).to(BF16).to(dev), pre=torch.sigmoid(r(T, n)).to(dev),
                comb=torch.softmax(r(T, n, n), 2).to(dev), gate=(2 * torch.sigmoid(r(T, n))).to(dev),
                norm=(1 + r(H, scale=0.1)).to(dev), w1=r(F, H, scale=H ** -0.5).to(BF16).to(dev),
                b1=r(F, scale=0.1).to(BF16).to(dev), w2=r(H, F, scale=F ** -0.5).to(BF16).to(dev))


def sublayer(p, act="gelu"):
    """Streams after one feed-forward sublayer, through the package's kernels."""
    from hyper_connection_residual_mhc_amd import linear, norm, post
    y, _ = norm.rms_norm_autograd(p["streams"], p["norm"], 1e-6, pre=p["pre"])
    h = linear.linear_autograd(y, p["w1"], p["b1"], activation=act)
    out = linear.linear_autograd(h, p["w2"])
    return post.post_update_autograd(p["streams"], p["comb"], p["gate"], out)


def plain(p, act="gelu"):
    """The same chain in fp64 PyTorch, without its roundings."""
    x = (p["pre"][:, :, None] * p["streams"]).sum(1)
    y, _ = R.norm(x, p["norm"], 1e-6)
    h, _ = R.linear(y, p["w1"], p["b1"], act)
    return R.post(p["streams"], p["comb"], p["gate"], h @ p["w2"].t())


def test_package_names():
    import hyper_connection_residual_mhc_amd as pkg
    from hyper_connection_residual_mhc_amd import linear, norm, post
    for module, names in ((norm, pkg._NORM_NAMES), (linear, pkg._LINEAR_NAMES), (post, pkg._POST_NAMES)):
        for name in names:
            assert getattr(pkg, name) is getattr(module, name)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,H,F", [(1, 4, 256, 512), (37, 2, 264, 520), (200, 4, 1288, 640), (130, 8, 129, 77)])
def test_training_step(device, T, n, H, F):
    say(f"sublayer T={T} n={n} H={H} F={F}")
    p = make(T, n, H, F, seed=T, dev=device)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(T, n, H, generator=gen).to(BF16).to(device)
    out = sublayer(leaves)
    grads = torch.autograd.grad(out, list(leaves.values()), g)
    exact = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    want = plain(exact)
    wants = torch.autograd.grad(want, list(exact.values()), g.cpu().double())
    # out: collapse, norm, hidden, product, write-back; a gradient passes those and their backward: gz, two products,
    # the norm's, the collapse's, and the sum of the streams' two gradients
    near(out, want, 5 * 2.0 ** -8, "out")
    for name, a, b in zip(leaves, grads, wants):
        assert a.dtype == p[name].dtype
        near(a, b, 12 * 2.0 ** -8, "gradient of " + name)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["row", "mx"])
@pytest.mark.parametrize("T", [1, 16, 100])
def test_decoding_step_in_8_bits(device, T, kind):
    """The norm's codes and scales go into the product as they are."""
    from hyper_connection_residual_mhc_amd import linear, norm, post
    n, H, F = 4, 512, 768
    p = make(T, n, H, F, seed=T + 5, dev=device)
    w1, s1 = (t.to(device) for t in R.quantise(p["w1"].float().cpu(), kind))
    o = norm.rms_norm(p["streams"], p["norm"], 1e-6, pre=p["pre"], quant=kind)
    h = linear.linear(o.y, w1, p["b1"], activation="silu", x_scales=o.scales, weight_scales=s1).out
    y = linear.linear(h, p["w2"]).out
    out = post.post_update(p["streams"], p["comb"], p["gate"], y)
    d = {k: v.cpu().double() for k, v in p.items()}
    x = (d["pre"][:, :, None] * d["streams"]).sum(1)
    yn, _ = R.norm(x, d["norm"], 1e-6)
    # the product alone on the codes' own values: hidden and its roundings only
    near(h, R.linear(R.dequantise(o.y, o.scales), R.dequantise(w1, s1), d["b1"], "silu")[0], 2 * 2.0 ** -8, "hidden")
    near(R.dequantise(o.y, o.scales), yn, 2.0 ** -4 + 2 * 2.0 ** -8, "codes")
    near(out, R.post(d["streams"], d["comb"], d["gate"], R.d(y)), 2.0 ** -8, "streams")
    # whole chain: the weight's and the activations' roundings to 8 bits, and the bf16 ones
    want = R.post(d["streams"], d["comb"], d["gate"], R.linear(yn, d["w1"], d["b1"], "silu")[0] @ d["w2"].t())
    near(out, want, 2 * 2.0 ** -4 + 5 * 2.0 ** -8, "chain")


@pytest.mark.gpu
def test_decoding_step_in_a_graph(device):
    """One captured decoding step, replayed on new streams, gives the eager bytes."""
    from hyper_connection_residual_mhc_amd import linear, norm, post
    T, n, H, F = 8, 4, 512, 640
    p = make(T, n, H, F, seed=3, dev=device)
    w1, s1 = (t.to(device) for t in R.quantise(p["w1"].float().cpu(), "mx"))

    def step(streams):
        o = norm.rms_norm(streams, p["norm"], 1e-6, pre=p["pre"], quant="mx")
        h = linear.linear(o.y, w1, p["b1"], activation="silu", x_scales=o.scales, weight_scales=s1).out
        return post.post_update(streams, p["comb"], p["gate"], linear.linear(h, p["w2"]).out)

    buf = p["streams"].clone()
    step(buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for k in range(4):
        new = (p["streams"] * (k + 0.5)).contiguous()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert R.same_bytes(got, step(new)), k


@pytest.mark.gpu
def test_workspaces_belong_to_the_stream_that_uses_them(device, monkeypatch):
    from hyper_connection_residual_mhc_amd import linear, norm
    side = torch.cuda.Stream()
    x, w = torch.randn(300, 4096, device=device).to(BF16), torch.randn(64, 4096, device=device).to(BF16)
    out, gw = torch.empty(300, 64, device=device, dtype=BF16), torch.empty_like(w)
    g, ones, dw = torch.randn_like(x), torch.ones(300, device=device), torch.empty(4096, device=device)
    gx = torch.empty_like(x)
    torch.cuda.synchronize()
    seen, empty = [], torch.empty

    def recording(*a, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", recording)
    linear.mhc_linear_fwd(x, w, out, launch={"kernel": 3, "splits": 4}, stream=side)
    linear.mhc_linear_bwd(out, x, w, grad_weight=gw, stream=side)
    norm.mhc_rms_norm_bwd(g, x, w[0], ones, gx, dw, stream=side)
    assert seen == [side] * 3
    seen.clear()
    linear.mhc_linear_fwd(x, w, out, launch={"kernel": 3, "splits": 4})
    assert seen == [torch.cuda.current_stream()]
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_second_derivatives_are_refused(device):
    from hyper_connection_residual_mhc_amd import linear, norm, post
    p = make(5, 4, 64, 32, 0, device)
    x = torch.randn(5, 64, device=device).to(BF16)
    for call, leaf in ((lambda t: norm.rms_norm_autograd(t, p["norm"])[0], x),
                       (lambda t: linear.linear_autograd(t, p["w1"], p["b1"], activation="silu"), x),
                       (lambda t: post.post_update_autograd(p["streams"], p["comb"], p["gate"], t), x)):
        t = leaf.clone().requires_grad_()
        first, = torch.autograd.grad(call(t).float().square().sum(), t, create_graph=True)
        with pytest.raises(RuntimeError):
            first.float().square().sum().backward()
