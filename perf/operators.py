"""Cases, plain forms and exact values of the operators around the block that a training step and the
dense sublayers need: layer norm, the router's balance loss and gradient, and a matrix product with
bias, activation and residual in its epilogue, each with its backward pass.

`own = False` computes every operator from elementary torch operations in 32 bits (64 where long sums
need them); `own = True` calls the framework's entry points on the same data.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
ALPHA = 1e-3
SCALING = 2.5


def listed():
    return [
        # the pre-norm of one decode step: an fp32 residual stream of 64 tokens to the bf16 input of a sublayer
        {"name": "norm_decode", "op": "norm", "rows": 64, "cols": 5120, "x": "f32", "y": "bf16", "pad": 0},
        # the same pre-norm over a long prefill or a training batch
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "cols": 5120, "x": "f32", "y": "bf16", "pad": 0},
        # a fine-tuning batch of odd width whose rows sit in a wider buffer, half precision
        {"name": "norm_back_odd", "op": "norm_back", "rows": 1021, "cols": 2561, "x": "f16", "y": "f16", "pad": 7},
        # training: gradient of the pre-norm on the fp32 stream, bf16 gradients from the sublayer
        {"name": "norm_back_train", "op": "norm_back", "rows": 8192, "cols": 5120, "x": "f32", "y": "bf16", "pad": 0},
        # watching the load of a decode batch: one sequence's worth of 64 tokens
        {"name": "balance_step", "op": "balance", "tokens": 64, "experts": 256, "topk": 8, "seqs": 1, "tail": 0},
        # a training batch of packed documents of very different lengths, padded at the end
        {"name": "balance_packed", "op": "balance", "tokens": 16384, "experts": 256, "topk": 8, "seqs": 37, "tail": 131},
        # the router's gradient for a small batch, weights and balance loss together
        {"name": "route_back_small", "op": "route_back", "tokens": 509, "experts": 256, "topk": 8, "seqs": 3, "tail": 0},
        # the router's gradient for a packed training batch
        {"name": "route_back_packed", "op": "route_back", "tokens": 16384, "experts": 256, "topk": 8, "seqs": 37,
         "tail": 131},
        # one token through a dense projection: latency and the weights' bytes
        {"name": "linear_token", "op": "linear", "rows": 1, "cols": 2560, "inner": 5120, "x": "bf16", "y": "bf16",
         "act": "silu", "residual": False, "pad": 0},
        # the down projection of a dense sublayer over a long prefill, added onto the fp32 stream
        {"name": "linear_prefill", "op": "linear", "rows": 16384, "cols": 5120, "inner": 2560, "x": "bf16", "y": "f32",
         "act": "none", "residual": True, "pad": 0},
        # gradients of a projection whose sizes no tile divides, half precision
        {"name": "linear_back_odd", "op": "linear_back", "rows": 517, "cols": 1003, "inner": 777, "x": "f16",
         "y": "f16", "act": "gelu", "residual": False, "pad": 0},
        # training: gradients of the up projection of a dense sublayer
        {"name": "linear_back_train", "op": "linear_back", "rows": 8192, "cols": 2560, "inner": 5120, "x": "bf16",
         "y": "bf16", "act": "silu", "residual": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "balance", "route_back", "linear", "linear_back"])
    if op in ("norm", "norm_back"):
        cols = _log(rng, 100, 8192)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = min(_log(rng, 1, 16384), 16384 * 5120 // cols)
        x = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": rows, "cols": cols, "x": x, "y": x if x == "f16" else rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, 0, 8, 5])}
    if op in ("balance", "route_back"):
        experts = rng.choice([16, 60, 64, 128, 200, 256, rng.randint(9, 256)])
        tokens = _log(rng, 1, 16384)
        tail = rng.choice([0, 0, rng.randint(0, tokens // 4)])
        return {"op": op, "tokens": tokens, "experts": experts, "topk": rng.randint(2, 8),
                "seqs": rng.choice([1, _log(rng, 1, 200)]), "tail": tail}
    cols, inner = _log(rng, 100, 5120), _log(rng, 100, 5120)
    if rng.random() < 0.6:
        cols, inner = max(64, cols // 64 * 64), max(64, inner // 64 * 64)
    x = rng.choice(["bf16", "bf16", "f16"])
    return {"op": op, "rows": _log(rng, 1, 8192), "cols": cols, "inner": inner, "x": x, "y": rng.choice([x, x, "f32"]),
            "act": rng.choice(["none", "relu", "silu", "gelu"]), "residual": rng.random() < 0.5,
            "pad": rng.choice([0, 0, 8, 3])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, shape, dtype, scale=1.0, pad=0):
    """Normal values; with pad > 0 a view of the first columns of a wider buffer."""
    t = torch.randn((*shape[:-1], shape[-1] + pad), generator=g, device="cuda", dtype=torch.float32) * scale
    return t.to(dtype)[..., : shape[-1]]


def _offsets(case, seed):
    """Starts of the packed sequences, [seqs + 1], the last one before the padding. From two sequences on
    the lengths are far apart, and one in eight is empty."""
    n, b = case["tokens"] - case["tail"], case["seqs"]
    if b == 1:
        return [0, n]
    r = np.random.RandomState(seed % (1 << 31))
    share = r.lognormal(0.0, 1.0, b) * (r.rand(b) >= 0.125)
    ends = np.floor(np.cumsum(share) / max(share.sum(), 1e-9) * n + 1e-6).astype(int)
    ends[-1] = n
    return [0] + [int(v) for v in ends]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op in ("norm", "norm_back"):
        T, H = case["rows"], case["cols"]
        size = torch.exp2(torch.arange(T, device="cuda") % 7 - 3.0)[:, None]
        x = torch.randn((T, H + case["pad"]), generator=g, device="cuda")
        x = ((x + 0.25) * size).to(DT[case["x"]])[:, :H]
        s.update(x=x, gamma=1 + _randn(g, (H,), torch.float32, 0.1), beta=_randn(g, (H,), torch.float32, 0.1))
        if op == "norm":
            s["y_dtype"] = DT[case["y"]]
        else:
            xd = x.double()
            mean, var = xd.mean(1), xd.var(1, unbiased=False)
            s.update(dy=_randn(g, (T, H), DT[case["y"]], 1.0, case["pad"]), mean=mean.float(),
                     rstd=(var + EPS).rsqrt().float())
    elif op in ("balance", "route_back"):
        T, E, K = case["tokens"], case["experts"], case["topk"]
        lean = torch.randn((E,), generator=g, device="cuda") * 0.7  # some experts are liked more than others
        scores = torch.sigmoid(torch.randn((T, E), generator=g, device="cuda") + lean)
        w, ids = torch.topk(scores, K, dim=1)
        off = _offsets(case, int(seed))
        s.update(scores=scores, ids=ids.to(torch.int32),
                 off=torch.tensor(off, dtype=torch.int32, device="cuda"))
        if op == "route_back":
            B = case["seqs"]
            seq = torch.bucketize(torch.arange(T, device="cuda"), s["off"][1:].long(), right=True)
            seen = torch.zeros((B + 1, E), dtype=torch.int64, device="cuda")
            seen.view(-1).index_add_(0, (seq[:, None] * E + ids).view(-1), torch.ones_like(ids).view(-1))
            s.update(dw=_randn(g, (T, K), torch.float32, 1e-2), counts=seen[:B].to(torch.int32).contiguous(),
                     dloss=torch.full((B,), 1.0 / B, device="cuda"))
    else:
        M, N, Kd, p = case["rows"], case["cols"], case["inner"], case["pad"]
        dt, yt = DT[case["x"]], DT[case["y"]]
        s.update(xs=_randn(g, (M, Kd), dt, 1.0, p), w=_randn(g, (N, Kd), dt, Kd ** -0.5, p), y_dtype=yt)
        # residual sublayers keep the stream with sqrt((k-1)/k) and add with sqrt(1/k); k = 3 here
        s["keep"], s["add"] = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if case["residual"] else (1.0, 1.0)
        if op == "linear":
            s["bias"] = _randn(g, (N,), torch.float32, 0.1)
            s["res"] = _randn(g, (M, N), yt, 1.0, p) if case["residual"] else None
        else:
            s["dy"] = _randn(g, (M, N), yt, 1.0, p)
            s["z"] = _randn(g, (M, N), dt, 1.0) if case["act"] != "none" else None
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
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    return (d * rstd[:, None] * s["gamma"] + s["beta"]).to(s["y_dtype"]), mean, rstd


def _norm_back(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    hat = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * hat).sum(0), dy.sum(0)


def _sequence_of(s):
    """The sequence of each token; seqs for the padding at the end."""
    at = torch.arange(s["tokens"], device="cuda")
    return torch.bucketize(at, s["off"][1:].long(), right=True)


def _balance(s):
    B, E, K = s["seqs"], s["experts"], s["topk"]
    at = torch.arange(B, device="cuda")[:, None]
    member = (_sequence_of(s) == at).double()  # [B, T]: which tokens are a sequence's
    total = member @ (s["scores"] / s["scores"].sum(1, keepdim=True)).double()
    picks = torch.zeros_like(s["scores"]).scatter_add_(1, s["ids"].long(), torch.ones_like(s["ids"]).float())
    counts = (member @ picks.double()).to(torch.int32)
    n = (s["off"][1:] - s["off"][:-1]).double()[:, None].clamp_min(1)
    prob = total / n
    loss = ALPHA * E * (counts / (K * n) * prob).sum(1)
    return loss.float(), counts, prob.float()


def _route_back(s):
    E, K, sc = s["experts"], s["topk"], s["scores"]
    ids = s["ids"].long()
    # the weights w = 2.5 s / sum(s) over the chosen experts
    chosen = sc.gather(1, ids)
    total = chosen.sum(1, keepdim=True)
    mean = (s["dw"] * chosen).sum(1, keepdim=True) / total
    ds = torch.zeros_like(sc).scatter_add_(1, ids, SCALING / total * (s["dw"] - mean))
    # the balance loss, through p = s / sum(s) over all experts; what a row shares drops out
    seq = _sequence_of(s)
    n = (s["off"][1:] - s["off"][:-1]).float()[:, None].clamp_min(1)
    c = s["dloss"][:, None] * ALPHA * (s["counts"] * E - K * n) / (K * n * n)
    c = torch.cat([c, torch.zeros_like(c[:1])])[seq]
    whole = sc.sum(1, keepdim=True)
    ds = ds + (c - (c * sc).sum(1, keepdim=True) / whole) / whole
    return ds * sc * (1 - sc)


def _linear(s):
    z = s["xs"].float() @ s["w"].float().t() + s["bias"]
    y = s["add"] * _act(z, s["act"])
    if s["res"] is not None:
        y = s["keep"] * s["res"].float() + y
    return y.to(s["y_dtype"])


def _linear_back(s):
    dz = s["add"] * s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    dx, dw = dz @ s["w"].float(), dz.t() @ s["xs"].float()
    return dx.to(s["xs"].dtype), dw.to(s["w"].dtype), dz.sum(0)


PLAIN = {"norm": _norm, "norm_back": _norm_back, "balance": _balance, "route_back": _route_back, "linear": _linear,
         "linear_back": _linear_back}


def _own(s):
    import grouped_top_routing_fp32_amd as fw
    op = s["op"]
    if op == "norm":
        return fw.beam_moe_layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS, out_dtype=s["y_dtype"])
    if op == "norm_back":
        return fw.beam_moe_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
    if op in ("balance", "route_back"):
        dims = fw.Dims(5120, 2560, s["experts"], 1, 1, s["topk"], SCALING)
        if op == "balance":
            return fw.beam_moe_balance_loss(dims, s["scores"], s["ids"], alpha=ALPHA, seq_offsets=s["off"])
        return fw.beam_moe_route_backward(dims, s["scores"], s["ids"], dw=s["dw"], dloss=s["dloss"],
                                          counts=s["counts"], alpha=ALPHA, seq_offsets=s["off"])
    if op == "linear":
        return fw.beam_moe_linear(s["xs"], s["w"], s["bias"], act=s["act"], residual=s["res"], keep=s["keep"],
                                  add=s["add"], out_dtype=s["y_dtype"])
    return fw.beam_moe_linear_backward(s["dy"], s["xs"], s["w"], s["z"], act=s["act"], add=s["add"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        T, H, x, y = case["rows"], case["cols"], SIZE[case["x"]], SIZE[case["y"]]
        if op == "norm":
            return {"bytes": T * H * (x + y) + 8 * H + 8 * T, "flops": 8 * T * H}
        return {"bytes": T * H * (2 * x + y) + 12 * H + 8 * T, "flops": 14 * T * H}
    if op in ("balance", "route_back"):
        T, E, K, B = case["tokens"], case["experts"], case["topk"], case["seqs"]
        n = T - case["tail"]
        if op == "balance":
            return {"bytes": n * (E + K) * 4 + B * (E * 8 + 8), "flops": 3 * n * E}
        return {"bytes": T * (2 * E + 2 * K) * 4 + B * (E * 4 + 8), "flops": 9 * T * E}
    M, N, Kd, x, y = case["rows"], case["cols"], case["inner"], SIZE[case["x"]], SIZE[case["y"]]
    if op == "linear":
        return {"bytes": (M * Kd + N * Kd) * x + N * 4 + M * N * y * (2 if case["residual"] else 1),
                "flops": 2 * M * N * Kd}
    z = M * N * x if case["act"] != "none" else 0
    return {"bytes": 2 * (M * Kd + N * Kd) * x + M * N * y + z + N * 4, "flops": 4 * M * N * Kd}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_back"):
        x = s["x"].double().requires_grad_(op == "norm_back")
        gamma, beta = (s[k].double().requires_grad_(op == "norm_back") for k in ("gamma", "beta"))
        y = torch.nn.functional.layer_norm(x, (case["cols"],), gamma, beta, EPS)
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            return y, mean, (var + EPS) ** -0.5
        return torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
    if op in ("balance", "route_back"):
        B, E, K = case["seqs"], case["experts"], case["topk"]
        # d stands for a change of the logits: ds/dlogit = s (1 - s)
        d = torch.zeros_like(s["scores"], dtype=torch.float64, requires_grad=True)
        sc = s["scores"].double()
        sc = sc + sc * (1 - sc) * d
        p = sc / sc.sum(1, keepdim=True)
        off = s["off"].tolist()
        loss, count, prob = [], [], []
        for a, b in zip(off[:-1], off[1:]):
            n = max(1, b - a)
            c = torch.bincount(s["ids"][a:b].reshape(-1).long(), minlength=E)
            m = p[a:b].sum(0) / n
            loss.append(ALPHA * ((E / (K * n)) * c.double() @ m))
            count.append(c)
            prob.append(m)
        if op == "balance":
            return torch.stack(loss).detach(), torch.stack(count), torch.stack(prob).detach()
        picked = sc.gather(1, s["ids"].long())
        w = SCALING * picked / picked.sum(1, keepdim=True)
        aim = (w * s["dw"].double()).sum() + (torch.stack(loss) * s["dloss"].double()).sum()
        return torch.autograd.grad(aim, d)[0]
    fn = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}
    x, w = s["xs"].double(), s["w"].double()
    if op == "linear":
        y = s["add"] * fn[case["act"]](torch.nn.functional.linear(x, w, s["bias"].double()))
        return y if s["res"] is None else y + s["keep"] * s["res"].double()
    dz = s["dy"].double() * s["add"]
    if s["z"] is not None:
        z = s["z"].double().requires_grad_(True)
        dz = torch.autograd.grad(fn[case["act"]](z), z, dz)[0]
    return torch.matmul(dz, w), torch.matmul(x.t(), dz).t(), dz.t().sum(1)
