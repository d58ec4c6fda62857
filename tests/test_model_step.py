"""The operators of a model's step together, as a model runs them: streams ->
collapse and norm -> gated block -> product -> write-back -> collapse and norm ->
cross entropy of the vocabulary, with all gradients through autograd; the
decoding form in 8-bit integers; and the products' kernels against each other.

Tolerances are relative 2-norms, counted as in test_sublayer.py: h R for R
roundings one after another, h = 2^-8 in bf16. A code of 8-bit integers is off by
at most half a step of the row's largest value / 127; normal values of up to a
few thousand columns reach at most 4.5 times their root mean square, so that the
row is off by at most 4.5 / 254 < 2^-5 of its norm."""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from test_gated import quantise_int8
from test_sublayer import make, near

BF16 = torch.bfloat16
H16 = 2.0 ** -8


def make_model(T, n, H, F, V, seed, dev):
    p = make(T, n, H, F, seed, dev)
    gen = torch.Generator().manual_seed(seed + 100)
    r = lambda *s, scale=1.0: (torch.randn(s, generator=gen) * scale)  # noqa: E731
    del p["b1"]
    p |= dict(w3=r(F, H, scale=H ** -0.5).to(BF16).to(dev), pre_out=torch.sigmoid(r(T, n)).to(dev),
              norm_out=(1 + r(H, scale=0.1)).to(dev), head=r(V, H, scale=H ** -0.5).to(BF16).to(dev))
    targets = torch.randint(0, V, (T,), generator=gen)
    targets[::5] = -100  # tokens of a prompt
    return p, targets.to(dev)


def losses(p, targets, reduction):
    """Streams to losses through the package's kernels."""
    from hyper_connection_residual_mhc_amd import gated, linear, loss, norm, post
    y, _ = norm.rms_norm_autograd(p["streams"], p["norm"], 1e-6, pre=p["pre"])
    h = gated.gated_autograd(y, p["w1"], p["w3"])
    out = linear.linear_autograd(h, p["w2"])
    streams = post.post_update_autograd(p["streams"], p["comb"], p["gate"], out)
    last, _ = norm.rms_norm_autograd(streams, p["norm_out"], 1e-6, pre=p["pre_out"])
    return loss.linear_cross_entropy_autograd(last, p["head"], targets, reduction=reduction)[0]


def plain(p, targets, reduction):
    """The same chain in fp64 PyTorch, without its roundings."""
    y, _ = R.norm((p["pre"][:, :, None] * p["streams"]).sum(1), p["norm"], 1e-6)
    g = y @ p["w1"].t()
    h = g / (1 + torch.exp(-g)) * (y @ p["w3"].t())
    streams = R.post(p["streams"], p["comb"], p["gate"], h @ p["w2"].t())
    last, _ = R.norm((p["pre_out"][:, :, None] * streams).sum(1), p["norm_out"], 1e-6)
    return torch.nn.functional.cross_entropy(last @ p["head"].t(), targets, reduction=reduction)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,H,F,V", [(2, 4, 256, 512, 600), (37, 2, 264, 520, 1001), (200, 4, 1288, 640, 2056), (130, 8, 129, 77, 333)])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_training_step(device, T, n, H, F, V, reduction):
    say(f"step T={T} n={n} H={H} F={F} V={V} {reduction}")
    p, targets = make_model(T, n, H, F, V, T, device)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    g = torch.rand((T,) if reduction == "none" else (), generator=torch.Generator().manual_seed(1))
    value = losses(leaves, targets, reduction)
    grads = torch.autograd.grad(value, list(leaves.values()), g.to(device))
    exact = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    want = plain(exact, targets.cpu(), reduction)
    wants = torch.autograd.grad(want, list(exact.values()), g.double())
    # collapse, norm, gate and up, their product, the second product, write-back, collapse, norm
    near(value, want, 8 * H16, "loss")
    # and back: the shares of the gradient, x's gradient, the norm's, the write-back's, the product's, gate's and up's, x's again,
    # the norm's, and the sum of the streams' two
    for name, a, b in zip(leaves, grads, wants):
        assert a.dtype == p[name].dtype
        near(a, b, 17 * H16, "gradient of " + name)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F,V", [(37, 264, 520, 1001), (130, 1288, 640, 2056)])
def test_training_step_in_a_graph(device, T, H, F, V):
    say(f"captured step T={T} H={H} F={F} V={V}")
    p, targets = make_model(T, 4, H, F, V, T, device)

    def step(leaves, targets):
        value = losses(leaves, targets, "mean")
        return (value.detach(), *torch.autograd.grad(value, list(leaves.values())))

    held, at = {k: v.clone().requires_grad_() for k, v in p.items()}, targets.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held, at)                                     # no graph of these leaves is left when it returns
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held, at)
    for k in range(4):
        new = {n: (v * (1 + 0.25 * k)).contiguous() if n in ("streams", "w1", "head") else v for n, v in p.items()}
        with torch.no_grad():
            for n, v in held.items():
                v.copy_(new[n])
        at.copy_(targets.roll(k))
        graph.replay()
        torch.cuda.synchronize()
        want = step({n: v.clone().requires_grad_() for n, v in new.items()}, targets.roll(k))
        for a, b in zip(got, want):
            assert R.same_bytes(a, b), k


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 100])
def test_decoding_step_in_8_bit_integers(device, T):
    """The norm's codes and scales go into the gated block and the products as they are."""
    from hyper_connection_residual_mhc_amd import gated, linear, norm, post
    n, H, F, V = 4, 512, 768, 1000
    p, _ = make_model(T, n, H, F, V, T + 5, device)
    w1, w3, head = (tuple(t.to(device) for t in quantise_int8(p[k].float().cpu())) for k in ("w1", "w3", "head"))
    o = norm.rms_norm(p["streams"], p["norm"], 1e-6, pre=p["pre"], quant="int8")
    h = gated.gated(o.y, w1[0], w3[0], x_scales=o.scales, gate_scales=w1[1], up_scales=w3[1]).out
    streams = post.post_update(p["streams"], p["comb"], p["gate"], linear.linear(h, p["w2"]).out)
    last = norm.rms_norm(streams, p["norm_out"], 1e-6, pre=p["pre_out"], quant="int8")
    logits = linear.linear(last.y, head[0], x_scales=last.scales, weight_scales=head[1]).out
    d = {k: v.cpu().double() for k, v in p.items()}
    value = lambda codes, scales: codes.cpu().double() * scales.cpu().double()[:, None]  # noqa: E731
    # the block and the last product alone, on the codes' own values
    y, g = value(o.y, o.scales), None
    g = y @ value(*w1).t()
    near(h, g / (1 + torch.exp(-g)) * (y @ value(*w3).t()), 2 * H16, "hidden")
    near(logits, value(last.y, last.scales) @ value(*head).t(), H16, "logits")
    yn, _ = R.norm((d["pre"][:, :, None] * d["streams"]).sum(1), d["norm"], 1e-6)
    near(y, yn, 2.0 ** -5 + 2 * H16, "codes")
    # whole chain: two norms' and two weights' roundings to 8 bits, one weight of which stands beside another, and those to bf16
    g = yn @ d["w1"].t()
    s = R.post(d["streams"], d["comb"], d["gate"], (g / (1 + torch.exp(-g)) * (yn @ d["w3"].t())) @ d["w2"].t())
    want = R.norm((d["pre_out"][:, :, None] * s).sum(1), d["norm_out"], 1e-6)[0] @ d["head"].t()
    near(logits, want, 6 * 2.0 ** -5 + 9 * H16, "chain")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("M,N,K", [(256, 256, 64), (256, 512, 1), (300, 520, 40), (513, 257, 200), (1031, 770, 1288)])
def test_large_tiles_give_the_medium_tiles_bytes(device, kind, M, N, K):
    """Both add up an output in the same order, so a policy that chooses between them changes no byte."""
    from hyper_connection_residual_mhc_amd import gated, linear
    from hyper_connection_residual_mhc_amd._lib import MHC_LINEAR_LARGE, MHC_LINEAR_MEDIUM
    say(f"large and medium {kind} {M} x {N} x {K}")
    gen = torch.Generator().manual_seed(M + K)
    scales = {}
    if kind == "int8":
        (x, xs), (w, ws), (u, us) = (tuple(t.to(device) for t in quantise_int8(torch.randn(r, K, generator=gen))) for r in (M, N, N))
        one, both = dict(x_scales=xs, weight_scales=ws), dict(x_scales=xs, gate_scales=ws, up_scales=us)
    else:
        t = BF16 if kind == "bf16" else torch.float16
        x, w, u = (R.normal(gen, r, K, dtype=t).to(device) for r in (M, N, N))
        one, both = {}, {}
    kind_out = BF16 if kind == "int8" else x.dtype
    for make, args in ((linear.mhc_linear_fwd, (x, w)), (gated.mhc_gated_fwd, (x, w, u))):
        scales = one if len(args) == 2 else both
        outs = []
        for kernel in (MHC_LINEAR_LARGE, MHC_LINEAR_MEDIUM):
            out = torch.full((M, N), 7.0, dtype=kind_out, device=device)
            make(*args, out, launch={"kernel": kernel, "splits": 1}, **scales)
            outs.append(out)
        assert R.same_bytes(*outs)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,splits", [(4100, 4104, 40, 1), (4100, 4104, 104, 1), (1024, 1031, 4480, 33), (300, 520, 640, 7),
                                          (1024, 2050, 64, 1)])
def test_large_tiles_one_after_another(device, M, N, K, splits):
    """More tiles than blocks, of one and of two passes, and parts of the sum without any: the loads run ahead through all of them."""
    from hyper_connection_residual_mhc_amd import linear
    from hyper_connection_residual_mhc_amd._lib import MHC_LINEAR_LARGE, MHC_LINEAR_MEDIUM
    say(f"tiles in turn {M} x {N} x {K} in {splits}")
    gen = torch.Generator().manual_seed(M + K)
    x, w, b = (R.normal(gen, *s).to(device) for s in ((M, K), (N, K), (N,)))
    outs = []
    for kernel in (MHC_LINEAR_LARGE, MHC_LINEAR_MEDIUM):
        out = torch.full((M, N), 7.0, dtype=BF16, device=device)
        linear.mhc_linear_fwd(x, w, out, bias=b, launch={"kernel": kernel, "splits": splits})
        outs.append(out)
    assert R.same_bytes(*outs)
    near(outs[0][::37], x[::37].cpu().double() @ w.cpu().double().t() + b.cpu().double(), H16, "product")
