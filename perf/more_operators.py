"""Cases, plain forms and exact values of the operators of a dense gated sublayer, trained and served: its two
projections with activation and product in one call and their gradients, the norm and clipping of all gradients of a
step, and microscaled 4-bit floating point (OCP MX: E2M1 codes, one E8M0 scale for 32 of them) with its product.

`own = False` computes every operator from elementary torch operations in 32 bits (64 where long sums need them);
`own = True` calls the framework's entry points on the same data.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32  # elements that share a scale
CLIP_EPS = 1e-6


def listed():
    return [
        # one decoded token through the gate and up projections of a dense sublayer: latency and the weights' bytes
        {"name": "gated_token", "op": "gated", "rows": 1, "cols": 2560, "inner": 5120, "x": "bf16", "y": "bf16",
         "act": "silu", "bias": False, "pre": False, "pad": 0},
        # the same over a long prefill
        {"name": "gated_prefill", "op": "gated", "rows": 16384, "cols": 2560, "inner": 5120, "x": "bf16", "y": "bf16",
         "act": "silu", "bias": False, "pre": False, "pad": 0},
        # gradients of a small sublayer whose sizes no tile divides, half precision, rows in wider buffers
        {"name": "gated_back_odd", "op": "gated_back", "rows": 517, "cols": 1003, "inner": 777, "x": "f16", "y": "f16",
         "act": "gelu", "bias": True, "pad": 3},
        # training: gradients of both projections
        {"name": "gated_back_train", "op": "gated_back", "rows": 8192, "cols": 2560, "inner": 5120, "x": "bf16",
         "y": "bf16", "act": "silu", "bias": False, "pad": 0},
        # clipping the gradients of a few norms and biases alone, as when the rest is frozen
        {"name": "clip_few", "op": "clip", "tensors": 9, "total": 30011, "x": "f32", "y": "f32", "scale": 1.0},
        # clipping all gradients of a model at the end of a step: 16-bit matrices, 32-bit vectors, into the optimizer's
        # flat 32-bit buffer
        {"name": "clip_model", "op": "clip", "tensors": 197, "total": 600_000_000, "x": "mixed", "y": "f32",
         "scale": 0.125},
        # a small matrix of odd width to 4 bits and back
        {"name": "mx_values_odd", "op": "mx_values", "rows": 509, "cols": 1003, "x": "f16", "y": "f16", "pad": 5},
        # a prefill's activations to 4 bits and back
        {"name": "mx_values_prefill", "op": "mx_values", "rows": 16384, "cols": 5120, "x": "bf16", "y": "bf16",
         "pad": 0},
        # one token through a projection whose weights are held in 4 bits
        {"name": "mx_linear_token", "op": "mx_linear", "rows": 1, "cols": 2560, "inner": 5120, "x": "bf16", "y": "bf16",
         "four": False, "act": "silu", "residual": False, "pad": 0},
        # a decode batch through the down projection, 4-bit weights, onto the fp32 stream
        {"name": "mx_linear_batch", "op": "mx_linear", "rows": 64, "cols": 5120, "inner": 2560, "x": "bf16", "y": "f32",
         "four": False, "act": "none", "residual": True, "pad": 0},
        # activations quantised on the way, sizes that no tile or block of 32 divides
        {"name": "mx_linear_odd", "op": "mx_linear", "rows": 259, "cols": 1003, "inner": 777, "x": "f16", "y": "f16",
         "four": True, "act": "gelu", "residual": False, "pad": 3},
        # a prefill with weights and activations in 4 bits, activations quantised on the way
        {"name": "mx_linear_prefill", "op": "mx_linear", "rows": 16384, "cols": 5120, "inner": 2560, "x": "bf16",
         "y": "bf16", "four": True, "act": "none", "residual": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_back", "clip", "mx_values", "mx_linear", "mx_linear"])
    x = rng.choice(["bf16", "bf16", "f16"])
    if op == "clip":
        total = _log(rng, 1000, 500_000_000)
        x = rng.choice(["bf16", "f16", "f32", "mixed"])
        return {"op": op, "tensors": min(_log(rng, 1, 400), total // 16), "total": total, "x": x,
                "y": rng.choice(["f32", x if x != "mixed" else "f32"]), "scale": rng.choice([1.0, 0.125, 1 / 3])}
    pad = rng.choice([0, 0, 8, 3])
    if op == "mx_values":
        cols = _log(rng, 20, 8192)
        x = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": min(_log(rng, 1, 16384), 16384 * 5120 // cols), "cols": cols, "x": x,
                "y": rng.choice([x, "f32"]), "pad": pad}
    cols, inner = _log(rng, 100, 5120), _log(rng, 100, 5120)
    if rng.random() < 0.6:
        cols, inner = max(64, cols // 64 * 64), max(64, inner // 64 * 64)
    case = {"op": op, "rows": _log(rng, 1, 8192), "cols": cols, "inner": inner, "x": x, "y": rng.choice([x, x, "f32"]),
            "act": rng.choice(["none", "relu", "silu", "gelu"]), "pad": pad}
    if op == "mx_linear":
        case.update(four=rng.random() < 0.5, residual=rng.random() < 0.5)
    else:
        case.update(bias=rng.random() < 0.5, act=rng.choice(["relu", "silu", "silu", "gelu"]))
        if op == "gated":
            case["pre"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, shape, dtype, scale=1.0, pad=0):
    """Normal values; with pad > 0 a view of the first columns of a wider buffer."""
    t = torch.randn((*shape[:-1], shape[-1] + pad), generator=g, device="cuda", dtype=torch.float32) * scale
    return t.to(dtype)[..., : shape[-1]]


def _lengths(case):
    """Elements of each gradient: far apart, a few large matrices and many short vectors, none of them even sizes."""
    r = np.random.RandomState(case["tensors"])
    share = r.lognormal(0.0, 2.0, case["tensors"])
    n = np.maximum(1, np.floor(share / share.sum() * (case["total"] - case["tensors"]))).astype(int)
    n[int(np.argmax(n))] += case["total"] - int(n.sum())
    return [int(v) for v in n]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op == "clip":
        n = _lengths(case)
        # norms of 0.3 to 30 before the scale, so that most steps are clipped to 1 and some are not
        size = math.exp(torch.rand((), generator=g, device="cuda").item() * math.log(100.0)) * 0.3
        size /= math.sqrt(case["total"]) * case["scale"]
        kinds = [("f32" if m < 10000 else "bf16") if case["x"] == "mixed" else case["x"] for m in n]
        if case["x"] == "f16":  # such gradients are held times a loss scale
            s["scale"], size = case["scale"] / 256, size * 256
        s["grads"] = [(torch.randn(m, generator=g, device="cuda") * size).to(DT[k]) for m, k in zip(n, kinds)]
        s["flat"] = torch.zeros(case["total"], dtype=DT[case["y"]], device="cuda")
        s["outs"] = list(torch.split(s["flat"], n))
        s["max_norm"] = 1.0
        return s
    dt, p = DT[case["x"]], case["pad"]
    if op == "mx_values":
        T, H = case["rows"], case["cols"]
        # some channels of activations are far larger than the others
        wide = 1 + 15 * (torch.rand(H, generator=g, device="cuda") < 0.02)
        x = torch.randn((T, H + p), generator=g, device="cuda")
        s.update(xs=(x[:, :H] * wide).to(dt) if p == 0 else (x * torch.nn.functional.pad(wide, (0, p))).to(dt)[:, :H],
                 y_dtype=DT[case["y"]])
        return s
    M, N, Kd = case["rows"], case["cols"], case["inner"]
    yt = DT[case["y"]]
    s.update(xs=_randn(g, (M, Kd), dt, 1.0, p), y_dtype=yt)
    if op == "mx_linear":
        blocks = -(-Kd // BLOCK)
        # weights of a deviation of about inner^-1/2 as they are stored: codes two to a byte, low half first, scales
        # with an exponent's bias of 127
        codes = torch.randint(0, 256, (N, blocks * BLOCK // 2), generator=g, device="cuda", dtype=torch.uint8)
        codes.view(N, -1)[:, (Kd + 1) // 2:] = 0
        if Kd % 2:
            codes[:, Kd // 2] &= 15
        mid = 127 - int(round(0.5 * math.log2(Kd))) - 2
        scales = torch.randint(mid - 1, mid + 2, (N, blocks), generator=g, device="cuda").to(torch.uint8)
        s.update(codes=codes, scales=scales, bias=_randn(g, (N,), torch.float32, 0.1),
                 res=_randn(g, (M, N), yt, 1.0, p) if case["residual"] else None)
        s["keep"], s["add"] = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if case["residual"] else (1.0, 1.0)
        return s
    s.update(wg=_randn(g, (N, Kd), dt, Kd ** -0.5, p), wu=_randn(g, (N, Kd), dt, Kd ** -0.5, p))
    if op == "gated":
        s["bg"], s["bu"] = (_randn(g, (N,), torch.float32, 0.1) if case["bias"] else None for _ in range(2))
    else:
        s.update(dh=_randn(g, (M, N), yt, 1.0, p), zg=_randn(g, (M, N), dt, 1.0, p), zu=_randn(g, (M, N), dt, 1.0, p))
    return s


# --------------------------------------------------------------------------
# the plain forms, and the framework's calls
# --------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _gated(s):
    x = s["xs"].float()
    zg, zu = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if s["bias"]:
        zg, zu = zg + s["bg"], zu + s["bu"]
    h = (_act(zg, s["act"]) * zu).to(s["y_dtype"])
    return (h, zg.to(s["xs"].dtype), zu.to(s["xs"].dtype)) if s["pre"] else h


def _gated_back(s):
    dh, zg, zu, x, dt = s["dh"].float(), s["zg"].float(), s["zu"].float(), s["xs"].float(), s["xs"].dtype
    dg, du = dh * zu * _act_slope(zg, s["act"]), dh * _act(zg, s["act"])
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    out = dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    return (*out, dg.sum(0), du.sum(0)) if s["bias"] else out


def _clip(s):
    flat = torch.cat([t.reshape(-1).float() for t in s["grads"]])
    norm = s["scale"] * flat.square().sum(dtype=torch.float64).sqrt()
    factor = s["scale"] * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return (flat * factor.float()).to(s["flat"].dtype), norm.float()


def _four(x):
    """The values that x [M, K] has in microscaled 4 bits, in 32: each block of 32 shares the power of two that takes
    its largest magnitude into [4, 8); what is left goes to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6, ties to even."""
    M, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(M, -1, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    scale = torch.exp2(torch.clamp(torch.frexp(top)[1] - 3, min=-126, max=127).float())
    v = v / scale
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(a / step) * step, max=6.0) * scale
    return torch.copysign(q, v).view(M, -1)[:, :K]


def _weights(s):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    c = s["codes"].int()
    v = table[torch.stack([c & 15, c >> 4], 2)].view(c.shape[0], -1, BLOCK)
    return (v * torch.exp2(s["scales"].float() - 127)[:, :, None]).view(c.shape[0], -1)[:, : s["inner"]]


def _mx_values(s):
    return _four(s["xs"]).to(s["y_dtype"])


def _mx_linear(s):
    x = _four(s["xs"]) if s["four"] else s["xs"].float()
    y = s["add"] * _act(x @ _weights(s).t() + s["bias"], s["act"])
    if s["res"] is not None:
        y = s["keep"] * s["res"].float() + y
    return y.to(s["y_dtype"])


PLAIN = {"gated": _gated, "gated_back": _gated_back, "clip": _clip, "mx_values": _mx_values, "mx_linear": _mx_linear}


def _own(s):
    import grouped_top_routing_fp32_amd as fw
    op = s["op"]
    if op == "gated":
        return fw.beam_moe_gated_linear(s["xs"], s["wg"], s["wu"], s["bg"], s["bu"], act=s["act"],
                                        out_dtype=s["y_dtype"], want_pre=s["pre"])
    if op == "gated_back":
        out = fw.beam_moe_gated_linear_backward(s["dh"], s["xs"], s["wg"], s["wu"], s["zg"], s["zu"], act=s["act"],
                                                want_dbias=s["bias"])
        return out if s["bias"] else out[:3]
    if op == "clip":
        norm = fw.beam_moe_clip_grads(s["grads"], s["max_norm"], scale=s["scale"], eps=CLIP_EPS, out=s["outs"])
        return s["flat"], norm
    if op == "mx_values":
        q = fw.beam_moe_quantize_mxfp4(s["xs"])
        return fw.beam_moe_dequantize_mxfp4(q, s["cols"], out_dtype=s["y_dtype"])
    x = fw.beam_moe_quantize_mxfp4(s["xs"]) if s["four"] else s["xs"]
    return fw.beam_moe_linear_mxfp4(x, (s["codes"], s["scales"]), s["bias"], act=s["act"], residual=s["res"],
                                    keep=s["keep"], add=s["add"], out_dtype=s["y_dtype"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "clip":
        x = sum(m * SIZE[("f32" if m < 10000 else "bf16") if case["x"] == "mixed" else case["x"]]
                for m in _lengths(case))
        return {"bytes": x + case["total"] * SIZE[case["y"]] + 4, "flops": 3 * case["total"]}
    if op == "mx_values":  # the codes and scales are the point of it: written once and read once
        T, H = case["rows"], case["cols"]
        return {"bytes": T * H * (SIZE[case["x"]] + SIZE[case["y"]]) + 2 * T * (-(-H // BLOCK)) * 17,
                "flops": 6 * T * H}
    M, N, Kd, x, y = case["rows"], case["cols"], case["inner"], SIZE[case["x"]], SIZE[case["y"]]
    if op == "mx_linear":
        w = N * -(-Kd // BLOCK) * 17
        return {"bytes": M * Kd * x + w + 4 * N + M * N * y * (2 if case["residual"] else 1), "flops": 2 * M * N * Kd}
    if op == "gated":
        return {"bytes": (M * Kd + 2 * N * Kd) * x + M * N * (y + (2 * x if case["pre"] else 0))
                + (8 * N if case["bias"] else 0), "flops": 4 * M * N * Kd}
    return {"bytes": 2 * (M * Kd + 2 * N * Kd) * x + M * N * (y + 2 * x) + (8 * N if case["bias"] else 0),
            "flops": 8 * M * N * Kd}


def _nearest(x):
    """What quantisation to microscaled 4 bits makes of x, in 64 bits, by the borders between neighbouring values."""
    M, K = x.shape
    out = torch.zeros((M, -(-K // BLOCK) * BLOCK), dtype=torch.float64, device=x.device)
    out[:, :K] = x
    b = out.view(-1, BLOCK)
    top = b.abs().max(1).values
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -125)))
    e = e - (torch.exp2(e) > top).double() + (torch.exp2(e + 1) <= top).double()
    unit = torch.exp2(e.clamp_min(-124) - 2)[:, None]
    a = b.abs() / unit
    values = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    q = torch.zeros_like(a)
    for i, (lo, hi) in enumerate(zip(values, values[1:])):
        border = (lo + hi) / 2  # the upper of the two has an even code where i is odd
        q += (hi - lo) * ((a >= border) if i % 2 else (a > border))
    return (torch.sign(b) * q * unit).view(M, -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        sq = [float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]]
        norm = s["scale"] * math.sqrt(math.fsum(sq))
        factor = s["scale"] * min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        return torch.cat([t.double() * factor for t in s["grads"]]), torch.tensor(norm, dtype=torch.float64)
    x = s["xs"].double()
    if op == "mx_values":
        return _nearest(x)
    fn = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
          "gelu": torch.nn.functional.gelu}[case["act"]]
    if op == "mx_linear":
        N, Kd = case["cols"], case["inner"]
        size = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        c = torch.empty((N, 2 * s["codes"].shape[1]), dtype=torch.int64, device="cuda")
        c[:, 0::2], c[:, 1::2] = s["codes"] % 16, s["codes"] // 16
        w = size[c % 8] * (1 - 2 * (c // 8))
        w = w * torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, 1)
        z = torch.nn.functional.linear(_nearest(x) if case["four"] else x, w[:, :Kd].contiguous(), s["bias"].double())
        y = s["add"] * fn(z)
        return y if s["res"] is None else y + s["keep"] * s["res"].double()
    wg, wu = s["wg"].double(), s["wu"].double()
    if op == "gated":
        bg, bu = (s[k].double() if case["bias"] else None for k in ("bg", "bu"))
        zg, zu = torch.nn.functional.linear(x, wg, bg), torch.nn.functional.linear(x, wu, bu)
        h = fn(zg) * zu
        return (h, zg, zu) if case["pre"] else h
    zg, zu = (s[k].double().requires_grad_(True) for k in ("zg", "zu"))
    dg, du = torch.autograd.grad(fn(zg) * zu, (zg, zu), s["dh"].double())
    out = torch.matmul(dg, wg) + torch.matmul(du, wu), torch.matmul(x.t(), dg).t(), torch.matmul(x.t(), du).t()
    return (*out, dg.t().sum(1), du.t().sum(1)) if case["bias"] else out
