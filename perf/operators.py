"""Cases of the operators around the collapse of a hyper-connected sublayer:

* norm: root-mean-square norm of x, of x + residual, or of the collapsed
  streams; output in the input's type or in 8 bits (e4m3) with scales;
* linear: matrix product with bias, activation and residual in its
  epilogue, 16-bit or e4m3 operands with the norm's scales;
* post: the write-back of a sublayer's output into the streams.

A "train" case is a forward pass and its backward pass. `own` selects the
package's kernels; otherwise `run` computes the plain form in fp32.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "row": 1, "mx": 1}


def listed():
    return [
        # One decoded token: the residual's addition, the norm and the 8-bit row that the next product reads.
        dict(name="norm 1 token to rows", op="norm", source="add", type="bf16", weight="bf16", n=1, rows=1, cols=4096,
             quant="row", train=False),
        # Prefill: the four streams are collapsed, normed and written in 8 bits with a scale for each 32 columns.
        dict(name="norm streams to mx", op="norm", source="streams", type="bf16", weight="bf16", n=4, rows=1024,
             cols=7168, quant="mx", train=False),
        # Training step of a wide model, the largest of its kind.
        dict(name="norm add train", op="norm", source="add", type="bf16", weight="f32", n=1, rows=4096, cols=7168,
             quant="none", train=True),
        # A ragged batch of odd width in fp16, forward and backward.
        dict(name="norm odd train", op="norm", source="plain", type="f16", weight="f16", n=1, rows=129, cols=1279,
             quant="none", train=True),
        # One decoded token through a projection back into the residual.
        dict(name="linear 1 token", op="linear", type="bf16", rows=1, cols=4096, depth=7168, act="none", bias=True,
             residual=True, train=False),
        # A small decoding batch with 8-bit weights and activations.
        dict(name="linear 16 tokens mx", op="linear", type="mx", rows=16, cols=7168, depth=4096, act="none", bias=False,
             residual=False, train=False),
        # The coefficient columns (pre, post and the 4 x 4 mixing logits) from the flattened streams: long and narrow.
        dict(name="linear coefficients", op="linear", type="bf16", rows=2048, cols=24, depth=28672, act="none",
             bias=True, residual=False, train=False),
        # Odd sizes in fp16, forward and backward.
        dict(name="linear odd train", op="linear", type="f16", rows=129, cols=1001, depth=1279, act="relu", bias=True,
             residual=True, train=True),
        # Prefill in 8 bits with an activation.
        dict(name="linear prefill mx", op="linear", type="mx", rows=8192, cols=4096, depth=7168, act="silu", bias=True,
             residual=False, train=False),
        # Training step of a projection with its activation, the largest of all.
        dict(name="linear train", op="linear", type="bf16", rows=4096, cols=7168, depth=4096, act="gelu", bias=True,
             residual=False, train=True),
        # A small decoding batch written back into its four streams.
        dict(name="post 8 tokens", op="post", n=4, rows=8, cols=4096, train=False),
        # Training step of the write-back.
        dict(name="post train", op="post", n=4, rows=4096, cols=7168, train=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """Widths over the whole range: most of them whole tiles, some multiples of 8, some odd."""
    v, kind = _log_int(rng, low, high), rng.random()
    step = 128 if kind < 0.5 and v >= 128 else 8 if kind < 0.75 else 1
    return max(low, v // step * step)


def _drawn(rng):
    op = rng.choice(("norm", "linear", "post"))
    if op == "norm":
        source = rng.choice(("plain", "add", "streams"))
        train = source != "streams" and rng.random() < 0.5
        kind = "bf16" if source == "streams" else rng.choice(("bf16", "bf16", "f16", "f32"))
        return dict(op=op, source=source, type=kind, weight=rng.choice((kind, "f32")),
                    n=rng.choice((2, 4, 8)) if source == "streams" else 1, rows=_log_int(rng, 1, 8192),
                    cols=_width(rng, 64, 16384), quant="none" if train else rng.choice(("none", "row", "mx")),
                    train=train)
    if op == "linear":
        kind = rng.choice(("bf16", "bf16", "f16", "row", "mx"))
        return dict(op=op, type=kind, rows=_log_int(rng, 1, 8192), cols=_width(rng, 8, 8192),
                    depth=_width(rng, 64, 28672), act=rng.choice(("none", "relu", "silu", "gelu")),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    train=kind in ("bf16", "f16") and rng.random() < 0.5)
    return dict(op=op, n=rng.choice((2, 4, 8)), rows=_log_int(rng, 1, 8192), cols=_width(rng, 64, 16384),
                train=rng.random() < 0.5)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most = {k: max(most.get(k, 0), w[k]) for k in w}
    while True:
        c = _drawn(rng)
        w = work(c)
        if all(w[k] <= most[k] for k in w):
            return c


def work(case):
    """Each input read once and each output written once, and the operations of the definition."""
    c = case
    T, H = c["rows"], c["cols"]
    if c["op"] == "norm":
        e, w, n, out = BYTES[c["type"]], BYTES[c["weight"]], c["n"], c["quant"]
        b = T * H * e * n + H * w + (T * n * 4 if c["source"] == "streams" else 0)
        b += T * H * e * (c["source"] == "add") + T * H * e * (c["source"] != "plain")
        b += {"none": T * H * e, "row": T * H + T * 4, "mx": T * H + T * -(-H // 32)}[out]
        if c["train"]:
            b += T * H * e * (2 + (c["source"] == "add")) + H * 4
        return {"bytes": b, "flops": T * H * (5 + 2 * n + (10 if c["train"] else 0))}
    if c["op"] == "linear":
        K, e = c["depth"], BYTES[c["type"]]
        b = (T + H) * K * e + T * H * 2 * (1 + c["residual"]) + H * 2 * c["bias"]
        b += {"row": (T + H) * 4, "mx": (T + H) * -(-K // 32)}.get(c["type"], 0)
        if c["train"]:
            b += T * H * 2 + (T + H) * K * e + H * 2 * c["bias"]
        return {"bytes": b, "flops": 2 * T * H * K * (3 if c["train"] else 1)}
    n = c["n"]
    b = T * H * 2 * (2 * n + 1) + T * n * (n + 1) * 4
    if c["train"]:
        b += T * H * 2 * (2 * n + 1) + T * n * (n + 1) * 4
    return {"bytes": b, "flops": T * H * 2 * n * (n + 1) * (3 if c["train"] else 1)}


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


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, type=torch.bfloat16, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).to(type)

    T, H = c["rows"], c["cols"]
    s = dict(case=c)
    if c["op"] == "norm":
        t = TYPES[c["type"]]
        s["weight"] = (1 + normal(H, type=torch.float32, scale=0.1)).to(TYPES[c["weight"]])
        # a residual stream has columns of its own size
        size = torch.exp(normal(H, type=torch.float32, scale=0.5))
        shape = (T, c["n"], H) if c["source"] == "streams" else (T, H)
        s["x"] = (normal(*shape, type=torch.float32) * size).to(t)
        s["pre"] = torch.rand((T, c["n"]), device="cuda", generator=g) if c["source"] == "streams" else None
        s["residual"] = (normal(T, H, type=torch.float32) * size).to(t) if c["source"] == "add" else None
        if c["train"]:
            s["grad_y"] = normal(T, H, type=t, scale=0.1)
            s["grad_stored"] = normal(T, H, type=t, scale=0.1) if c["source"] == "add" else None
    elif c["op"] == "linear":
        K = c["depth"]
        t = TYPES.get(c["type"], torch.bfloat16)
        quant = {"row": _rows, "mx": _mx}.get(c["type"], lambda v: (v.to(t), None))
        s["x"], s["x_scales"] = quant(normal(T, K, type=torch.float32))
        s["weight"], s["weight_scales"] = quant(normal(H, K, type=torch.float32, scale=K ** -0.5))
        s["bias"] = normal(H, type=t, scale=0.1) if c["bias"] else None
        s["residual"] = normal(T, H, type=t) if c["residual"] else None
        s["grad_out"] = normal(T, H, type=t, scale=0.1) if c["train"] else None
    else:
        n = c["n"]
        s["streams"] = normal(T, n, H)
        s["y"] = normal(T, H)
        # mixing rows sum to one, write-back gates are twice a sigmoid
        s["comb"] = torch.softmax(normal(T, n, n, type=torch.float32), 2)
        s["post"] = 2 * torch.sigmoid(normal(T, n, type=torch.float32))
        s["grad_out"] = normal(T, n, H, scale=0.1) if c["train"] else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "post": _own_post}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "post": _plain_post}[op](state)


def _own_norm(s):
    from hyper_connection_residual_mhc_amd import norm
    c = s["case"]
    o = norm.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], pre=s["pre"],
                      quant=None if c["quant"] == "none" else c["quant"], return_rstd=c["train"])
    got = {"y": o.y, "scales": o.scales, "stored": o.stored if c["source"] != "plain" else None}
    if c["train"]:
        stored = s["x"] if c["source"] == "plain" else o.stored
        got["grad_x"], got["grad_weight"] = norm.rms_norm_backward(
            s["grad_y"], stored, s["weight"], o.rstd, grad_stored=s["grad_stored"])
    return got


def _own_linear(s):
    from hyper_connection_residual_mhc_amd import linear
    c = s["case"]
    o = linear.linear(s["x"], s["weight"], s["bias"], activation=c["act"], residual=s["residual"],
                      x_scales=s["x_scales"], weight_scales=s["weight_scales"], return_z=c["train"])
    got = {"out": o.out}
    if c["train"]:
        got["grad_x"], got["grad_weight"], got["grad_bias"] = linear.linear_backward(
            s["grad_out"], s["x"], s["weight"], activation=c["act"], z=o.z, bias=c["bias"])
    return got


def _own_post(s):
    from hyper_connection_residual_mhc_amd import post
    got = {"out": post.post_update(s["streams"], s["comb"], s["post"], s["y"])}
    if s["case"]["train"]:
        names = ("grad_streams", "grad_comb", "grad_post", "grad_y")
        got.update(zip(names, post.post_update_backward(s["grad_out"], s["streams"], s["comb"], s["post"], s["y"])))
    return got


def _pairs(p):
    """Sum over dim 1 as the collapse defines it: adjacent pairs first."""
    return p.view(p.shape[0], -1, 2, p.shape[2]).sum(2)


def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    if c["source"] == "streams":
        x = s["pre"][:, :, None] * x
        x = _pairs(x) if c["n"] > 1 else x
        x = _pairs(x) if c["n"] > 2 else x
        x = _pairs(x) if c["n"] > 4 else x
        x = x[:, 0]
    elif c["source"] == "add":
        x = x + s["residual"].float()
    stored = x.to(t)
    x = stored.float()
    rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * w
    got = {"y": None, "scales": None, "stored": stored if c["source"] != "plain" else None}
    if c["quant"] == "none":
        got["y"] = y.to(t)
    else:
        got["y"], got["scales"] = (_rows if c["quant"] == "row" else _mx)(y)
    if c["train"]:
        u = s["grad_y"].float() * w
        grad = rstd * (u - x * ((u * x).mean(1, keepdim=True) * rstd.square()))
        got["grad_x"] = (grad + s["grad_stored"].float() if c["source"] == "add" else grad).to(t)
        got["grad_weight"] = (s["grad_y"].float() * x * rstd).sum(0)
    return got


def _wide(q, scales, type):
    """The fp32 values that an operand of the product stands for."""
    if scales is None:
        return q.float()
    if scales.dtype == torch.float32:
        return q.float() * scales[:, None]
    return q.float() * scales.float().repeat_interleave(32, 1)[:, :q.shape[1]]


def _act(z, name):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z / (1 + torch.exp(-z)),
            "gelu": lambda: 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))}[name]()


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _plain_linear(s):
    c = s["case"]
    t = TYPES.get(c["type"], torch.bfloat16)
    x, w = _wide(s["x"], s["x_scales"], t), _wide(s["weight"], s["weight_scales"], t)
    z = x @ w.t()
    z = z + s["bias"].float() if c["bias"] else z
    out = _act(z, c["act"])
    out = out + s["residual"].float() if c["residual"] else out
    got = {"out": out.to(t)}
    if c["train"]:
        g = s["grad_out"].float()
        g = g * _act_slope(z, c["act"]) if c["act"] != "none" else g
        got["grad_x"], got["grad_weight"] = (g @ w).to(t), (g.t() @ x).to(t)
        got["grad_bias"] = g.sum(0).to(t) if c["bias"] else None
    return got


def _plain_post(s):
    r, y = s["streams"].float(), s["y"].float()
    got = {"out": (torch.bmm(s["comb"], r) + s["post"][:, :, None] * y[:, None]).to(torch.bfloat16)}
    if s["case"]["train"]:
        g = s["grad_out"].float()
        got["grad_streams"] = torch.bmm(s["comb"].transpose(1, 2).contiguous(), g).to(torch.bfloat16)
        got["grad_comb"] = torch.bmm(g, r.transpose(1, 2).contiguous())
        got["grad_post"] = (g * y[:, None]).sum(2)
        got["grad_y"] = (s["post"][:, :, None] * g).sum(1).to(torch.bfloat16)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "post": _exact_post}[case["op"]](s)


def _exact_norm(s):
    """The definition in 64 bits, its gradients by differentiation of the definition."""
    c = s["case"]
    x = s["x"].double()
    if c["source"] == "streams":
        x = torch.einsum("tnh,tn->th", x, s["pre"].double())
    elif c["source"] == "add":
        x = x + s["residual"].double()
    stored = x
    # the norm is defined on the stored row, which has the type of x
    x = x.to(s["x"].dtype).double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    y = torch.nn.functional.normalize(x, dim=1, eps=0) * x.shape[1] ** 0.5
    # rms with eps: |x|^2 / (|x|^2 + H eps) takes the eps in
    square = x.square().sum(1, keepdim=True)
    y = y * torch.sqrt(square / (square + x.shape[1] * EPS)) * w
    got = {"y": y.detach(), "scales": None, "stored": stored if c["source"] != "plain" else None}
    if c["quant"] == "row":
        got["scales"] = y.detach().abs().amax(1) / E4M3_MAX
        got["y"] = y.detach() / got["scales"][:, None]
    elif c["quant"] == "mx":
        H = x.shape[1]
        v = torch.nn.functional.pad(y.detach(), (0, -H % 32)).view(y.shape[0], -1, 32)
        got["scales"] = torch.exp2(torch.ceil(torch.log2(v.abs().amax(2) / E4M3_MAX)))
        got["y"] = (v / got["scales"][:, :, None]).reshape(y.shape[0], -1)[:, :H]
    if c["train"]:
        gx, gw = torch.autograd.grad(y, (x, w), s["grad_y"].double())
        got["grad_x"] = gx + s["grad_stored"].double() if c["source"] == "add" else gx
        got["grad_weight"] = gw
    return got


def _exact_linear(s):
    c = s["case"]

    def value(q, scales):
        v = q.to(torch.float32).double()
        if scales is None:
            return v
        each = q.shape[1] if scales.dim() == 1 else 32
        at = torch.arange(q.shape[1], device=q.device) // each
        return v * scales.float().double().view(q.shape[0], -1)[:, at]

    x, w = value(s["x"], s["x_scales"]), value(s["weight"], s["weight_scales"])
    b = s["bias"].double() if c["bias"] else torch.zeros(c["cols"], dtype=torch.float64, device=x.device)
    z = torch.addmm(b, x, w.t()).requires_grad_()
    f = torch.nn.functional
    out = {"none": lambda v: v * 1, "relu": f.relu, "silu": f.silu, "gelu": f.gelu}[c["act"]](z)
    got = {"out": out.detach() + s["residual"].double() if c["residual"] else out.detach()}
    if c["train"]:
        g, = torch.autograd.grad(out, z, s["grad_out"].double())
        got["grad_x"], got["grad_weight"] = torch.mm(g, w), torch.mm(g.t(), x)
        got["grad_bias"] = g.sum(0) if c["bias"] else None
    return got


def _exact_post(s):
    leaves = [s[k].double().requires_grad_() for k in ("streams", "comb", "post", "y")]
    r, comb, post, y = leaves
    # the sublayer's output as one more stream, its gate as one more column of the mixing matrix
    out = torch.bmm(torch.cat((comb, post[:, :, None]), 2), torch.cat((r, y[:, None]), 1))
    got = {"out": out.detach()}
    if s["case"]["train"]:
        grads = torch.autograd.grad(out, leaves, s["grad_out"].double())
        got.update(zip(("grad_streams", "grad_comb", "grad_post", "grad_y"), grads))
    return got
