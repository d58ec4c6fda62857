"""Cases of the products around a hyper-connected sublayer's norm:

* gated: both projections of a gated feed-forward block, the activation and
  the product of the two in one call; 16-bit or e4m3 operands;
* loss: softmax cross entropy of a large vocabulary's logits x W^T, which are
  not kept, with its gradients;
* int8: matrix product of 8-bit integers with a scale for each token and each
  channel, alone or behind the norm that writes such rows.

A "train" case returns what the forward pass gives and the gradients. `own`
selects the package's kernels; otherwise `run` computes the plain form in fp32.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
I8_MAX = 127.0
IGNORED = -100
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"bf16": 2, "f16": 2, "row": 1, "mx": 1}


def listed():
    return [
        # One decoded token through a feed-forward block's two projections: both weights are streamed once.
        dict(name="gated 1 token", op="gated", type="bf16", rows=1, cols=16384, depth=4096, act="silu", bias=False,
             train=False),
        # A small decoding batch with 8-bit weights and activations.
        dict(name="gated 24 tokens mx", op="gated", type="mx", rows=24, cols=14336, depth=7168, act="silu", bias=False,
             train=False),
        # Training step at odd sizes in fp16, with biases.
        dict(name="gated odd train", op="gated", type="f16", rows=129, cols=1001, depth=1279, act="gelu", bias=True,
             train=True),
        # Training step of a wide model's feed-forward block.
        dict(name="gated train", op="gated", type="bf16", rows=4096, cols=14336, depth=4096, act="silu", bias=False,
             train=True),
        # Scoring a few tokens: the loss alone.
        dict(name="loss 8 tokens", op="loss", type="bf16", rows=8, cols=65536, depth=7168, reduction="none", ignored=0.0,
             train=False),
        # Training step with a weight for each token, some of them ignored, at odd sizes in fp16.
        dict(name="loss odd train", op="loss", type="f16", rows=129, cols=10007, depth=1279, reduction="none",
             ignored=0.2, train=True),
        # Training step of a model with a large vocabulary, the largest of all.
        dict(name="loss train", op="loss", type="bf16", rows=4096, cols=131072, depth=4096, reduction="mean",
             ignored=0.05, train=True),
        # One decoded token through an 8-bit projection back into the residual.
        dict(name="int8 1 token", op="int8", norm=False, rows=1, cols=4096, depth=7168, act="none", bias=False,
             residual=True),
        # A decoding batch: the norm writes the 8-bit rows that the projection reads.
        dict(name="int8 norm 32 tokens", op="int8", norm=True, rows=32, cols=7168, depth=4096, act="none", bias=True,
             residual=False),
        # Odd sizes.
        dict(name="int8 odd", op="int8", norm=False, rows=129, cols=1001, depth=1279, act="relu", bias=True,
             residual=True),
        # Prefill with an activation.
        dict(name="int8 prefill", op="int8", norm=False, rows=8192, cols=4096, depth=7168, act="silu", bias=True,
             residual=False),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """Widths over the whole range: most of them whole tiles, some multiples of 8, some odd."""
    v, kind = _log_int(rng, low, high), rng.random()
    step = 128 if kind < 0.5 and v >= 128 else 8 if kind < 0.75 else 1
    return max(low, v // step * step)


def _drawn(rng):
    op = rng.choice(("gated", "loss", "int8"))
    rows = _log_int(rng, 1, 8192)
    if op == "gated":
        kind = rng.choice(("bf16", "bf16", "f16", "row", "mx"))
        return dict(op=op, type=kind, rows=rows, cols=_width(rng, 8, 28672), depth=_width(rng, 64, 8192),
                    act=rng.choice(("none", "relu", "silu", "gelu")), bias=rng.random() < 0.5,
                    train=kind in TYPES and rng.random() < 0.6)
    if op == "loss":
        return dict(op=op, type=rng.choice(("bf16", "bf16", "f16")), rows=rows, cols=_width(rng, 256, 131072),
                    depth=_width(rng, 64, 8192), reduction=rng.choice(("none", "mean", "sum")),
                    ignored=rng.choice((0.0, 0.1, 0.5)), train=rng.random() < 0.6)
    return dict(op=op, norm=rng.random() < 0.4, rows=rows, cols=_width(rng, 8, 8192), depth=_width(rng, 64, 28672),
                act=rng.choice(("none", "relu", "silu", "gelu")), bias=rng.random() < 0.5, residual=rng.random() < 0.5)


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], {})
        m.update({k: max(m.get(k, 0), w[k]) for k in w})
    while True:
        c = _drawn(rng)
        w = work(c)
        if all(w[k] <= most[c["op"]][k] for k in w):
            return c


def work(case):
    """Each input read once and each output written once, and the operations of the definition."""
    c = case
    T, N, K = c["rows"], c["cols"], c["depth"]
    if c["op"] == "gated":
        e = BYTES[c["type"]]
        b = (T + 2 * N) * K * e + T * N * 2 + 4 * N * c["bias"]
        b += {"row": (T + 2 * N) * 4, "mx": (T + 2 * N) * -(-K // 32)}.get(c["type"], 0)
        if c["train"]:
            # the two values before the activation, the output's gradient, and the gradients
            b += T * N * 2 * 3 + (T + 2 * N) * K * e + 4 * N * c["bias"]
        return {"bytes": b, "flops": 4 * T * N * K * (3 if c["train"] else 1)}
    if c["op"] == "loss":
        b = (T + N) * K * 2 * (2 if c["train"] else 1) + T * (8 + 4 + (4 if c["reduction"] == "none" else 0))
        return {"bytes": b, "flops": 2 * T * N * K * (3 if c["train"] else 1)}
    b = (T + N) * K + (T + N) * 4 + T * N * 2 * (1 + c["residual"]) + N * 2 * c["bias"]
    if c["norm"]:
        b += T * K * (2 * 3 - 1) + K * 2
    return {"bytes": b, "flops": 2 * T * N * K}


def _mx(v):
    """v [R, C] in e4m3 with a power-of-two scale for each 32 columns: the smallest that keeps 448 unpassed."""
    R, C = v.shape
    blocks = torch.nn.functional.pad(v.double(), (0, -C % 32)).view(R, -1, 32)
    fraction, exponent = torch.frexp(blocks.abs().amax(2) / E4M3_MAX)
    power = torch.where(fraction == 0.5, exponent - 1, exponent).clamp(-127, 127)
    power = torch.where(fraction == 0, torch.full_like(power, -127), power)
    codes = torch.ldexp(blocks, -power[:, :, None]).view(R, -1)[:, :C].float().to(torch.float8_e4m3fn)
    return codes.contiguous(), (power + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _rows(v):
    """v [R, C] in e4m3 with one fp32 scale a row."""
    scale = (v.abs().amax(1) / E4M3_MAX).clamp_min(2.0 ** -126)
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def _int8(v):
    """v [R, C] in 8-bit integers with one fp32 scale a row."""
    scale = (v.abs().amax(1) / I8_MAX).clamp_min(2.0 ** -126)
    return (v / scale[:, None]).round().to(torch.int8), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, type=torch.bfloat16, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).to(type)

    T, N, K = c["rows"], c["cols"], c["depth"]
    f32 = torch.float32
    s = dict(case=c)
    if c["op"] == "gated":
        t = TYPES.get(c["type"], torch.bfloat16)
        quant = {"row": _rows, "mx": _mx}.get(c["type"], lambda v: (v.to(t), None))
        s["x"], s["x_scales"] = quant(normal(T, K, type=f32))
        s["gate_weight"], s["gate_scales"] = quant(normal(N, K, type=f32, scale=K ** -0.5))
        s["up_weight"], s["up_scales"] = quant(normal(N, K, type=f32, scale=K ** -0.5))
        s["gate_bias"] = normal(N, type=t, scale=0.1) if c["bias"] else None
        s["up_bias"] = normal(N, type=t, scale=0.1) if c["bias"] else None
        s["grad_out"] = normal(T, N, type=t, scale=0.1) if c["train"] else None
    elif c["op"] == "loss":
        t = TYPES[c["type"]]
        s["weight"] = normal(N, K, type=t, scale=2 * K ** -0.5)
        s["targets"] = torch.randint(N, (T,), device="cuda", generator=g)
        # rows lean to their targets by 0 to 12 logits, as a trained model's do
        lean = 3 * torch.rand((T, 1), device="cuda", generator=g)
        s["x"] = (normal(T, K, type=f32) + lean * s["weight"][s["targets"]].float()).to(t)
        drop = torch.rand((T,), device="cuda", generator=g) < c["ignored"]
        s["targets"] = torch.where(drop, torch.full_like(s["targets"], IGNORED), s["targets"])
        s["grad_loss"] = None
        if c["train"] and c["reduction"] == "none":
            s["grad_loss"] = torch.rand((T,), device="cuda", generator=g)
    else:
        s["weight"], s["weight_scales"] = _int8(normal(N, K, type=f32, scale=K ** -0.5))
        # a residual stream has columns of its own size
        x = normal(T, K, type=f32) * torch.exp(normal(K, type=f32, scale=0.5))
        if c["norm"]:
            s["x"] = x.to(torch.bfloat16)
            s["added"] = normal(T, K)
            s["norm_weight"] = (1 + normal(K, type=f32, scale=0.1)).to(torch.bfloat16)
        else:
            s["x"], s["x_scales"] = _int8(x)
        s["bias"] = normal(N, scale=0.1) if c["bias"] else None
        s["residual"] = normal(T, N) if c["residual"] else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gated": _own_gated, "loss": _own_loss, "int8": _own_int8}[op](state)
    return {"gated": _plain_gated, "loss": _plain_loss, "int8": _plain_int8}[op](state)


def _own_gated(s):
    from hyper_connection_residual_mhc_amd import gated
    c = s["case"]
    o = gated.gated(s["x"], s["gate_weight"], s["up_weight"], s["gate_bias"], s["up_bias"], activation=c["act"],
                    x_scales=s["x_scales"], gate_scales=s["gate_scales"], up_scales=s["up_scales"],
                    return_z=c["train"])
    got = {"out": o.out}
    if c["train"]:
        got["gate"], got["up"] = o.gate, o.up
        names = ("grad_x", "grad_gate_weight", "grad_up_weight", "grad_gate_bias", "grad_up_bias")
        got.update(zip(names, gated.gated_backward(s["grad_out"], s["x"], s["gate_weight"], s["up_weight"], o.gate,
                                                   o.up, activation=c["act"], bias=c["bias"])))
    return got


def _own_loss(s):
    from hyper_connection_residual_mhc_amd import loss
    c = s["case"]
    if not c["train"]:
        o = loss.linear_cross_entropy(s["x"], s["weight"], s["targets"], ignore_index=IGNORED,
                                      reduction=c["reduction"])
        return {"loss": o.loss, "lse": o.lse}
    o = loss.linear_cross_entropy_grads(s["x"], s["weight"], s["targets"], s["grad_loss"], ignore_index=IGNORED,
                                        reduction=c["reduction"])
    return {"loss": o.loss, "lse": o.lse, "grad_x": o.grad_x, "grad_weight": o.grad_weight}


def _own_int8(s):
    from hyper_connection_residual_mhc_amd import linear, norm
    c = s["case"]
    got = {}
    if c["norm"]:
        o = norm.rms_norm(s["x"], s["norm_weight"], EPS, residual=s["added"], quant="int8")
        x, x_scales = o.y, o.scales
        got["stored"], got["scales"] = o.stored, o.scales
    else:
        x, x_scales = s["x"], s["x_scales"]
    got["out"] = linear.linear(x, s["weight"], s["bias"], activation=c["act"], residual=s["residual"],
                               x_scales=x_scales, weight_scales=s["weight_scales"]).out
    return got


def _wide(q, scales):
    """The fp32 values that an operand of a product stands for."""
    if scales is None:
        return q.float()
    if scales.dtype == torch.float32:
        return q.float() * scales[:, None]
    return q.float() * scales.float().repeat_interleave(32, 1)[:, :q.shape[1]]


def _act(z, name):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z / (1 + torch.exp(-z)),
            "gelu": lambda: 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))}[name]()


def _act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _plain_gated(s):
    c = s["case"]
    t = TYPES.get(c["type"], torch.bfloat16)
    x, wg, wu = (_wide(s[k], s[q]) for k, q in (("x", "x_scales"), ("gate_weight", "gate_scales"),
                                                ("up_weight", "up_scales")))
    gate, up = x @ wg.t(), x @ wu.t()
    if c["bias"]:
        gate, up = gate + s["gate_bias"].float(), up + s["up_bias"].float()
    a = _act(gate, c["act"])
    got = {"out": (a * up).to(t)}
    if c["train"]:
        got["gate"], got["up"] = gate.to(t), up.to(t)
        g = s["grad_out"].float()
        g_gate, g_up = g * up * _act_slope(gate, c["act"]), g * a
        got["grad_x"] = (g_gate @ wg + g_up @ wu).to(t)
        got["grad_gate_weight"], got["grad_up_weight"] = (g_gate.t() @ x).to(t), (g_up.t() @ x).to(t)
        got["grad_gate_bias"] = g_gate.sum(0).to(t) if c["bias"] else None
        got["grad_up_bias"] = g_up.sum(0).to(t) if c["bias"] else None
    return got


def _plain_loss(s):
    c = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    counts = s["targets"] != IGNORED
    at = torch.where(counts, s["targets"], torch.zeros_like(s["targets"]))[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    each = torch.where(counts, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    got = {"lse": lse}
    if c["reduction"] == "none":
        got["loss"] = each
    else:
        got["loss"] = each.sum() / counts.sum() if c["reduction"] == "mean" else each.sum()
    if c["train"]:
        share = counts.float()
        if c["reduction"] == "none":
            share = share * s["grad_loss"]
        elif c["reduction"] == "mean":
            share = share / share.sum()
        # a row without a target that counts gives nothing, and 0 / 0 has no place in it
        share = torch.where(counts, share, torch.zeros_like(share))[:, None]
        p = p * (share / total)
        p.scatter_add_(1, at, -share)
        got["grad_x"], got["grad_weight"] = (p @ w).to(s["x"].dtype), (p.t() @ x).to(s["x"].dtype)
    return got


def _plain_int8(s):
    c = s["case"]
    got = {}
    if c["norm"]:
        got["stored"] = (s["x"].float() + s["added"].float()).to(torch.bfloat16)
        v = got["stored"].float()
        v = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * s["norm_weight"].float()
        x, x_scales = _int8(v)
        got["scales"] = x_scales
    else:
        x, x_scales = s["x"], s["x_scales"]
    z = (x.float() @ s["weight"].float().t()) * (x_scales[:, None] * s["weight_scales"])
    z = z + s["bias"].float() if c["bias"] else z
    out = _act(z, c["act"])
    got["out"] = (out + s["residual"].float() if c["residual"] else out).to(torch.bfloat16)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "loss": _exact_loss, "int8": _exact_int8}[case["op"]](s)


_ACTIVATIONS = {"none": lambda v: v * 1, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
                "gelu": torch.nn.functional.gelu}


def _value(q, scales):
    """What an operand stands for, in 64 bits."""
    v = q.double() if q.dtype != torch.float8_e4m3fn else q.float().double()
    if scales is None:
        return v
    each = q.shape[1] if scales.dim() == 1 else 32
    at = torch.arange(q.shape[1], device=q.device) // each
    return v * scales.float().double().view(q.shape[0], -1)[:, at]


def _exact_gated(s):
    """The definition in 64 bits; its gradients by differentiation from the two projections on."""
    c = s["case"]
    x = _value(s["x"], s["x_scales"])
    wg, wu = _value(s["gate_weight"], s["gate_scales"]), _value(s["up_weight"], s["up_scales"])
    # both projections as one, of the two weights above one another
    both = torch.mm(x, torch.cat((wg, wu)).t())
    if c["bias"]:
        both += torch.cat((s["gate_bias"], s["up_bias"])).double()
    both.requires_grad_()
    gate, up = both.chunk(2, 1)
    out = _ACTIVATIONS[c["act"]](gate) * up
    got = {"out": out.detach()}
    if c["train"]:
        got["gate"], got["up"] = gate.detach(), up.detach()
        g, = torch.autograd.grad(out, both, s["grad_out"].double())
        got["grad_x"] = torch.mm(g, torch.cat((wg, wu)))
        got["grad_gate_weight"], got["grad_up_weight"] = torch.mm(g.t(), x).chunk(2)
        bias = g.sum(0).chunk(2) if c["bias"] else (None, None)
        got["grad_gate_bias"], got["grad_up_bias"] = bias
    return got


def _exact_loss(s):
    """torch's cross entropy of the logits in 64 bits, its gradients by differentiation."""
    c = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    z = torch.mm(x, w.t()).requires_grad_(c["train"])
    got = {"lse": torch.logsumexp(z.detach(), 1)}
    loss = torch.nn.functional.cross_entropy(z, s["targets"], ignore_index=IGNORED, reduction=c["reduction"])
    got["loss"] = loss.detach()
    if c["train"]:
        upstream = s["grad_loss"].double() if c["reduction"] == "none" else torch.ones_like(loss)
        g, = torch.autograd.grad(loss, z, upstream)
        got["grad_x"], got["grad_weight"] = torch.mm(g, w), torch.mm(g.t(), x)
    return got


def _exact_int8(s):
    c = s["case"]
    got = {}
    if c["norm"]:
        got["stored"] = s["x"].double() + s["added"].double()
        # the norm is defined on the stored row, which has the type of x, and the product on its codes
        v = got["stored"].to(torch.bfloat16).double()
        v = v * torch.rsqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS) * s["norm_weight"].double()
        got["scales"] = v.abs().amax(1) / I8_MAX
        x = torch.round(v / got["scales"][:, None]) * got["scales"][:, None]
    else:
        x = _value(s["x"], s["x_scales"])
    z = torch.mm(x, _value(s["weight"], s["weight_scales"]).t())
    z = z + s["bias"].double() if c["bias"] else z
    out = _ACTIVATIONS[c["act"]](z)
    got["out"] = out + s["residual"].double() if c["residual"] else out
    return got
