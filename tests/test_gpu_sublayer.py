"""GPU parity of the operators around the block (layer norm, balance loss, the router's gradient,
linear) with their formulas in 64 bits.

Tolerances are bounds on the kernels' own roundings: u = 2^-24 is FP32's half step, a sum of
depth d is off by at most d u times the sum of magnitudes, and a result stored in type t by at
most half a step, finfo(t).eps / 2 of its value (plus half the least subnormal of fp16).
"""
import math

import pytest
import torch

from grouped_top_routing_fp32_amd import binding as fw
from grouped_top_routing_fp32_amd.synth import Dims

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _say(*what):
    print("\n[case]", *what, flush=True)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=F32, scale=1.0, pad=0):
    """Normal values; with pad, the first columns of a wider buffer whose rest is NaN."""
    t = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), device=DEV)
    t[..., : shape[-1]] = torch.randn(shape, generator=g, device=DEV) * scale
    return t.to(dtype)[..., : shape[-1]]


def _step(t):
    return torch.finfo(t.dtype).eps / 2


def _tiny(t):
    return 2.0 ** -25 if t.dtype == F16 else 0.0


def _near(got, want, bound, what=""):
    """|got - want| <= bound + the rounding to got's type, element by element."""
    torch.cuda.synchronize()
    want = want.double()
    # the value that is rounded is itself up to `bound` off
    tol = bound + _step(got) * (want.abs() + bound) + _tiny(got)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol.clamp_min(1e-300)).max()))


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def _norm_ref(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = ((d * d).mean(1) + eps) ** -0.5
    hat = d * rstd[:, None]
    y = hat * (gamma.double() if gamma is not None else 1.0) + (beta.double() if beta is not None else 0.0)
    return y, mean, rstd, hat


def _norm_check(x, gamma, beta, eps, out):
    """Mean: its wave's rest r / n is a sum of depth <= 64 of the differences to the wave's rounded mean.
    rstd: the sum of squares has depth <= 64, its square root half of that, and a few steps after it."""
    y, mean, rstd = out
    ry, rm, rr, hat = _norm_ref(x, gamma, beta, eps)
    std = 1 / rr
    _near(mean, rm, 64 * U * std, "mean")
    _near(rstd, rr, 40 * U * rr, "rstd")
    g = gamma.double().abs() if gamma is not None else 1.0
    _near(y, ry, U * (g * (64 + 48 * hat.abs()) + 4 * ry.abs()), "y")


NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (4, 100), (2, 512), (3, 520), (7, 1000), (9, 2561), (64, 5120), (130, 768),
               (2, 8192), (3, 8200), (2, 16384), (2, 16383), (5, 4097), (1030, 129)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xt,yt", [(F32, BF16), (BF16, BF16), (F16, F16), (BF16, F32), (F32, F32)])
def test_layer_norm(rows, cols, xt, yt):
    _say("layer_norm", rows, cols, xt, yt)
    g = _gen(rows * 7 + cols)
    for pad in (0, 8, 5):
        x = _randn(g, (rows, cols), xt, 2.0, pad)
        gamma, beta = 1 + _randn(g, (cols,), F32, 0.2), _randn(g, (cols,), F32, 0.5)
        _norm_check(x, gamma, beta, 1e-5, fw.beam_moe_layer_norm(x, gamma, beta, eps=1e-5, out_dtype=yt))
        _norm_check(x, None, None, 1e-5, fw.beam_moe_layer_norm(x, eps=1e-5, out_dtype=yt))


@pytest.mark.parametrize("cols", [96, 2561, 5120])
def test_layer_norm_far_mean_constant_rows_and_nan(cols):
    _say("layer_norm far mean", cols)
    g = _gen(cols)
    x = _randn(g, (6, cols)) + 1000.0
    x[1] = 3.0                                   # constant: variance 0
    x[4] = -1e4 + 0.01 * torch.randn((cols,), generator=g, device=DEV)
    y, mean, rstd = fw.beam_moe_layer_norm(x, eps=1e-5)
    ry, rm, rr, hat = _norm_ref(x, None, None, 1e-5)
    # the mean's rest is exact to 64 u of the spread, the stored mean to half a step
    _near(mean, rm, 64 * U / rr, "mean")
    _near(rstd, rr, 40 * U * rr, "rstd")
    _near(y, ry, U * (64 + 48 * hat.abs() + 4 * ry.abs()), "y")
    assert (y[1] == 0).all()
    x[2, cols // 2] = float("nan")
    x[5, 0] = float("inf")
    z, _, _ = fw.beam_moe_layer_norm(x, eps=1e-5)
    for r in (0, 1, 3, 4):
        assert torch.equal(z[r], y[r])
    assert z[2].isnan().all() and z[5].isnan().any()


@pytest.mark.parametrize("cols", [96, 2561, 5120, 16383])
def test_layer_norm_large_constant_rows(cols):
    """Equal columns of any size have variance 0, never a negative one.  A wave's mean P is off by e <= 64 u |x|,
    the rest D by 64 u e, so the variance comes out within 64 u e^2 and y within 64 u e rstd."""
    _say("layer_norm large constants", cols)
    g = _gen(cols)
    c = torch.rand((200,), generator=g, device=DEV) * 10.0 ** torch.linspace(0, 12, 200, device=DEV)
    y, mean, rstd = fw.beam_moe_layer_norm(c[:, None].expand(200, cols).contiguous(), eps=1e-5)
    e = 64 * U * c.double()
    assert y.isfinite().all() and rstd.isfinite().all()
    assert ((mean.double() - c.double()).abs() <= 64 * U * e + U * c.double()).all()
    assert (rstd.double() <= 1e-5 ** -0.5 * (1 + 8 * U)).all()
    assert (rstd.double() >= (1e-5 + 64 * U * e * e) ** -0.5 * (1 - 8 * U)).all()
    assert (y.double().abs() <= (64 * U * e * 1e-5 ** -0.5)[:, None]).all()


def test_layer_norm_zero_eps_and_padding_untouched():
    _say("layer_norm padding")
    g = _gen(3)
    buf = torch.full((9, 48), 7.0, device=DEV, dtype=BF16)
    x = _randn(g, (9, 40), BF16)
    out = fw.beam_moe_layer_norm(x, eps=0.0, out=buf[:, :40], want_stats=False)
    assert out[1] is None and out[2] is None
    ry, _, _, hat = _norm_ref(x, None, None, 0.0)
    _near(buf[:, :40], ry, U * (64 + 48 * hat.abs() + 4 * ry.abs()))
    assert (buf[:, 40:] == 7).all()
    y, mean, rstd = fw.beam_moe_layer_norm(x[:0])
    assert y.shape == (0, 40) and mean.numel() == 0 and rstd.numel() == 0


def test_layer_norm_offsets_past_32_bits():
    """Rows of a buffer so wide that the last ones start past 2^32 elements."""
    _say("layer_norm wide rows")
    g = _gen(12)
    rows, ld, cols = 66000, 65600, 72
    buf = torch.empty((rows, ld), dtype=BF16, device=DEV)
    x = buf[:, :cols]
    x.copy_(torch.randn((rows, cols), generator=g, device=DEV))
    y, mean, rstd = fw.beam_moe_layer_norm(x, out=buf[:, 128: 128 + cols])
    want = fw.beam_moe_layer_norm(x.contiguous())
    assert torch.equal(y, want[0]) and torch.equal(mean, want[1]) and torch.equal(rstd, want[2])
    a = fw.beam_moe_layer_norm_backward(y, x, mean, rstd)
    b = fw.beam_moe_layer_norm_backward(y.contiguous(), x.contiguous(), mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def _norm_back_ref(dy, x, mean, rstd, gamma):
    dy, x, rs = dy.double(), x.double(), rstd.double()[:, None]
    hat = (x - mean.double()[:, None]) * rs
    g = dy * (gamma.double() if gamma is not None else 1.0)
    c1, c2 = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    return rs * (g - c1 - hat * c2), (dy * hat).sum(0), dy.sum(0), hat, g


def _norm_back_check(dy, x, mean, rstd, gamma, out):
    """dx: two row sums of depth <= 64 of g and g xh, whose factors carry a few steps each.
    Column sums: a team's rows, up to 16 teams of a workgroup, 16 of at most 256 workgroups a thread, 16 joined."""
    T = x.shape[0]
    rdx, rdg, rdb, hat, g = _norm_back_ref(dy, x, mean, rstd, gamma)
    dx, dg, db = out
    rs = rstd.double()[:, None]
    a, b = g.abs().mean(1, keepdim=True), (g * hat).abs().mean(1, keepdim=True)
    _near(dx, rdx, U * rs * (6 * g.abs() + 70 * a + hat.abs() * 76 * b), "dx")
    depth = math.ceil(T / 256) + 16 + 16 + 24
    _near(dg, rdg, depth * U * (dy.double() * hat).abs().sum(0), "dgamma")
    _near(db, rdb, depth * U * dy.double().abs().sum(0), "dbeta")


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [
    (2100, 640), (1100, 5120), (1024, 520), (1025, 129), (1600, 2561), (1540, 4097), (1100, 8200), (1538, 16383)])
@pytest.mark.parametrize("xt,dt", [(F32, BF16), (BF16, BF16), (F16, F16), (BF16, F32), (F32, F32)])
def test_layer_norm_backward(rows, cols, xt, dt):
    _say("layer_norm_backward", rows, cols, xt, dt)
    g = _gen(rows * 11 + cols)
    for pad in (0, 8, 5):
        x, dy = _randn(g, (rows, cols), xt, 2.0, pad), _randn(g, (rows, cols), dt, 1.0, pad)
        gamma = 1 + _randn(g, (cols,), F32, 0.2)
        _, mean, rstd = fw.beam_moe_layer_norm(x, gamma, eps=1e-5)
        _norm_back_check(dy, x, mean, rstd, gamma, fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma))
        _norm_back_check(dy, x, mean, rstd, None, fw.beam_moe_layer_norm_backward(dy, x, mean, rstd))


def test_layer_norm_backward_parts_zero_rows_and_repeat():
    _say("layer_norm_backward parts")
    g = _gen(5)
    x, dy, gamma = _randn(g, (700, 264), BF16), _randn(g, (700, 264), BF16), _randn(g, (264,))
    _, mean, rstd = fw.beam_moe_layer_norm(x, gamma)
    dx, dg, db = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma)
    only = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma, want_params=False)
    assert torch.equal(only[0], dx) and only[1] is None
    only = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma, want_dx=False)
    assert only[0] is None and torch.equal(only[1], dg) and torch.equal(only[2], db)
    x, dy = _randn(g, (1700, 264), BF16), _randn(g, (1700, 264), BF16)
    _, mean, rstd = fw.beam_moe_layer_norm(x, gamma)
    both = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma)
    only = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma, want_params=False)
    assert torch.equal(only[0], both[0])
    only = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma, want_dx=False)
    assert torch.equal(only[1], both[1]) and torch.equal(only[2], both[2])
    dx, dg, db = fw.beam_moe_layer_norm_backward(dy[:0], x[:0], mean[:0], rstd[:0], gamma)
    assert dx.shape == (0, 264) and not dg.any() and not db.any()


def test_layer_norm_backward_of_few_rows_past_32_bits():
    _say("layer_norm_backward few rows far apart")
    g = _gen(17)
    T, H, ld = 1024, 100, 5 << 20
    buf = torch.empty((T, ld), dtype=BF16, device=DEV)
    x, dy = buf[:, :H], buf[:, 128: 128 + H]
    x.copy_(torch.randn((T, H), generator=g, device=DEV))
    dy.copy_(torch.randn((T, H), generator=g, device=DEV))
    _, mean, rstd = fw.beam_moe_layer_norm(x)
    a = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd)
    b = fw.beam_moe_layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_layer_norm_gradient_against_differences():
    """The kernel's own outputs on both sides of x, in fp32: the quotient carries the forward's rounding
    over the step, and the formula's own curvature, which 64 bits give exactly."""
    _say("layer_norm differences")
    g = _gen(6)
    x, v, dy = _randn(g, (5, 333)), _randn(g, (5, 333)), _randn(g, (5, 333))
    gamma = 1 + _randn(g, (333,), F32, 0.2)
    _, mean, rstd = fw.beam_moe_layer_norm(x, gamma)
    dx, _, _ = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma)
    h = 2.0 ** -7
    xp, xm = x + h * v, x - h * v
    yp, ym = (fw.beam_moe_layer_norm(t, gamma)[0] for t in (xp, xm))
    exact = (_norm_ref(xp, gamma, None, 1e-5)[0] - _norm_ref(xm, gamma, None, 1e-5)[0])
    d = dy.double()
    quot = (d * (yp.double() - ym.double())).sum(1) / (2 * h)
    moved = (xp.double() - xm.double()) / (2 * h)
    slope = (dx.double() * moved).sum(1)
    hat = _norm_ref(x, gamma, None, 1e-5)[3].abs() + 0.1
    noise = (d.abs() * U * (gamma.double().abs() * (64 + 48 * hat) + 5 * hat)).sum(1) / h
    curve = ((d * exact).sum(1) / (2 * h) - slope).abs()
    assert ((quot - slope).abs() <= noise + curve).all()
    assert (curve <= 1e-2 * (d * exact).sum(1).abs() / (2 * h) + 1e-2).all()


@pytest.mark.parametrize("rows,cols", [(5, 333), (3, 2560)])
def test_layer_norm_gradient_against_differences_with_64_bit_curvature(rows, cols):
    """The kernel's difference quotient against its own gradient, where nothing in the bound comes from that
    gradient: the forward outputs' roundings over the step, dx's own, and the difference of quotient and slope of the
    formula in 64 bits."""
    _say("layer_norm differences, 64-bit curvature", rows, cols)
    g = _gen(rows + cols)
    x, v, dy = (_randn(g, (rows, cols)) for _ in range(3))
    gamma = 1 + _randn(g, (cols,), F32, 0.2)
    _, mean, rstd = fw.beam_moe_layer_norm(x, gamma)
    dx, _, _ = fw.beam_moe_layer_norm_backward(dy, x, mean, rstd, gamma)
    h = 2.0 ** -5
    xp, xm = x + h * v, x - h * v
    yp, ym = (fw.beam_moe_layer_norm(t, gamma)[0].double() for t in (xp, xm))
    (rp, _, _, hp), (rm, _, _, hm) = (_norm_ref(t, gamma, None, 1e-5) for t in (xp, xm))
    _, m64, r64, _ = _norm_ref(x, gamma, None, 1e-5)
    rdx, _, _, hat, gg = _norm_back_ref(dy, x, m64, r64, gamma)
    d, moved = dy.double(), (xp.double() - xm.double()) / (2 * h)
    quot, slope = (d * (yp - ym)).sum(1) / (2 * h), (dx.double() * moved).sum(1)
    curve = ((d * (rp - rm)).sum(1) / (2 * h) - (rdx * moved).sum(1)).abs()
    # as in the checks of y and dx; dx takes mean and rstd rounded to FP32 besides, 64 and 40 u of them
    gd = gamma.double().abs()
    ey = sum(U * (gd * (64 + 48 * k.abs()) + 4 * y.abs()) + U * y.abs() for k, y in ((hp, rp), (hm, rm)))
    a, b = gg.abs().mean(1, keepdim=True), (gg * hat).abs().mean(1, keepdim=True)
    ex = U * r64[:, None] * (6 * gg.abs() + 70 * a + hat.abs() * 76 * b) + U * rdx.abs()
    ex = ex + U * r64[:, None] * (40 * (gg.abs() + a + 3 * hat.abs() * b) + 64 * (b + hat.abs() * a))
    bound = (d.abs() * ey).sum(1) / (2 * h) + (ex * moved.abs()).sum(1) + curve
    assert ((quot - slope).abs() <= bound).all(), (quot, slope, bound)
    assert (bound <= 0.05 * (rdx * moved).norm(dim=1) * cols ** 0.5).all()  # a bound that says something


# --------------------------------------------------------------------------
# balance loss and the router's gradient
# --------------------------------------------------------------------------
def _problem(T, E, K, lens, seed, lead=0):
    """Scores, ids with dropped slots and repeated ids, offsets of sequences of the given lengths."""
    g = _gen(seed)
    scores = torch.sigmoid(torch.randn((T, E), generator=g, device=DEV) * 1.5)
    ids = torch.rand((T, E), generator=g, device=DEV).add_(scores).topk(K, 1).indices.int()
    if T > 2:
        ids[1, 0] = -1
        ids[2, K - 1] = E
        ids[T - 1, K - 1] = ids[T - 1, 0]
    off = [lead]
    for n in lens:
        off.append(off[-1] + n)
    assert off[-1] <= T
    return scores.contiguous(), ids.contiguous(), off


def _balance_ref(scores, ids, off, alpha, K):
    s = scores.double()
    E = s.shape[1]
    tot = s.sum(1, keepdim=True)
    p = torch.where(tot == 0, torch.zeros_like(s), s / tot)
    loss, counts, prob = [], [], []
    for a, b in zip(off[:-1], off[1:]):
        n = b - a
        i = ids[a:b].reshape(-1).long()
        c = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
        m = p[a:b].sum(0) / max(n, 1)
        counts.append(c)
        prob.append(m)
        loss.append(alpha * E * (c.double() * m).sum() / (K * max(n, 1)))
    return torch.stack(loss), torch.stack(counts), torch.stack(prob)


def _dims(E, K, scaling=2.5):
    return Dims(256, 128, E, 1, 1, K, scaling)


BALANCE = [  # T, E, K, lengths, tokens before the first sequence
    (1, 256, 8, [1], 0), (4, 16, 4, [4], 0), (64, 256, 8, [64], 0), (64, 60, 3, [10, 0, 1, 50], 0),
    (500, 256, 8, [0, 0, 499], 1), (513, 256, 8, [513], 0), (700, 129, 16, [64, 64, 1, 0, 63, 400], 5),
    (3000, 200, 8, [1] * 100 + [0] * 30 + [2500], 11), (5000, 256, 8, [129, 4000, 0, 800], 64),
    (4096, 7, 2, [4096], 0), (50, 1, 1, [20, 30], 0), (600, 1, 1, [600], 0), (40000, 32, 1, [39999], 0), (2048, 256, 8, [2] * 1000, 0),
]


@pytest.mark.parametrize("T,E,K,lens,lead", BALANCE)
def test_balance_loss(T, E, K, lens, lead):
    """prob: a row's sum of depth <= 10 and its reciprocal, then sums of at most 84 rows and planes in FP32,
    all of positive terms; loss: the same errors, weighted."""
    _say("balance_loss", T, E, K, len(lens))
    scores, ids, off = _problem(T, E, K, lens, T + E, lead)
    if T > 3:
        scores[3] = 0.0                         # a token without any score adds nothing
    dev_off = torch.tensor(off, dtype=torch.int32, device=DEV)
    whole = lens == [T]
    for o in ([dev_off, None] if whole else [dev_off]):
        loss, counts, prob = fw.beam_moe_balance_loss(_dims(E, K), scores, ids, alpha=0.01, seq_offsets=o)
        rl, rc, rp = _balance_ref(scores, ids, off, 0.01, K)
        assert torch.equal(counts.long(), rc)
        _near(prob, rp, 100 * U * rp, "prob")
        _near(loss, rl, 100 * U * rl, "loss")
        again = fw.beam_moe_balance_loss(_dims(E, K), scores, ids, alpha=0.01, seq_offsets=o)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, prob)))


@pytest.mark.parametrize("T", [96, 2000])
def test_balance_loss_keeps_nan_in_its_sequence(T):
    _say("balance_loss nan", T)
    lens = [30, 40, T - 80]
    scores, ids, off = _problem(T, 256, 8, lens, 1)
    scores[35, 9] = float("nan")
    scores[T - 1] = float("inf")                # padding: never read into a result
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    loss, counts, prob = fw.beam_moe_balance_loss(_dims(256, 8), scores, ids, alpha=1.0, seq_offsets=o)
    assert loss[1].isnan() and prob[1].isnan().all()
    assert loss[[0, 2]].isfinite().all() and prob[[0, 2]].isfinite().all()
    assert torch.equal(counts.long(), _balance_ref(scores, ids, off, 1.0, 8)[1])


def _faint(T, E, K, seed):
    """Scores of logits near -95, below the smallest normal number, but for the first row."""
    g = _gen(seed)
    scores = (0.1 + 0.9 * torch.rand((T, E), generator=g, device=DEV)) * 2.0 ** -132
    scores[0] = torch.rand((E,), generator=g, device=DEV)
    assert (scores[1:] > 0).all() and float(scores[1:].max()) < torch.finfo(F32).tiny
    ids = torch.rand((T, E), generator=g, device=DEV).topk(K, dim=1).indices.int()
    return scores, ids


@pytest.mark.parametrize("T,E,K", [(40, 100, 4), (33, 101, 4), (700, 256, 8), (600, 9, 2)])
def test_faint_scores(T, E, K):
    """The shares of scores whose sum has no finite reciprocal in FP32 are as good as any others'.  Bounds as in
    the tests of ordinary scores."""
    _say("faint scores", T, E, K)
    scores, ids = _faint(T, E, K, T + E)
    loss, counts, prob = fw.beam_moe_balance_loss(_dims(E, K), scores, ids, alpha=0.3)
    rl, rc, rp = _balance_ref(scores, ids, [0, T], 0.3, K)
    assert torch.equal(counts.long(), rc)
    _near(prob, rp, 100 * U * rp, "prob")
    _near(loss, rl, 100 * U * rl, "loss")
    g = _gen(T)
    dw, dloss = torch.randn((T, K), generator=g, device=DEV), torch.randn((1,), generator=g, device=DEV)
    for w, l in ((dw, dloss), (dw, None), (None, dloss)):
        got = fw.beam_moe_route_backward(_dims(E, K), scores, ids, dw=w, dloss=l, alpha=0.5,
                                         counts=counts if l is not None else None)
        want, mag = _route_back_ref(scores, ids, w, 2.5, [0, T], 0.5, l, counts, K)
        _near(got, want, 40 * U * mag, (w is None, l is None))


def test_balance_loss_of_no_tokens_is_zero():
    _say("balance_loss T = 0")
    s, i = torch.empty((0, 64), device=DEV), torch.empty((0, 4), dtype=torch.int32, device=DEV)
    o = torch.zeros(4, dtype=torch.int32, device=DEV)
    for out in (fw.beam_moe_balance_loss(_dims(64, 4), s, i, alpha=1.0, seq_offsets=o),
                fw.beam_moe_balance_loss(_dims(64, 4), s, i, alpha=1.0)):
        assert all(t.numel() and not t.any() for t in out)
    assert fw.beam_moe_route_backward(_dims(64, 4), s, i, dw=torch.empty((0, 4), device=DEV)).shape == (0, 64)


def _route_back_ref(scores, ids, dw, scale, off, alpha, dloss, counts, K):
    """The gradient, and the magnitudes its error is bounded by."""
    s = scores.double()
    T, E = s.shape
    ds, mag = torch.zeros_like(s), torch.zeros_like(s)
    if dw is not None:
        ok = (ids >= 0) & (ids < E)
        i = torch.where(ok, ids, 0).long()
        sk = torch.where(ok, s.gather(1, i), 0.0)
        d = torch.where(ok, dw.double(), 0.0)
        tot = sk.sum(1, keepdim=True)
        inv = torch.where(tot == 0, 0.0, 1 / tot)
        a = torch.where(ok, scale * inv * (d - (d * sk).sum(1, keepdim=True) * inv), 0.0)
        m = torch.where(ok, scale * inv * (d.abs() + (d.abs() * sk).sum(1, keepdim=True) * inv), 0.0)
        ds.scatter_add_(1, i, a)
        mag.scatter_add_(1, i, m)
    if dloss is not None:
        for b in range(len(off) - 1):
            lo, hi = off[b], off[b + 1]
            n = max(hi - lo, 1)
            g = (counts[b].double() * E - K * n)[None]
            c = float(dloss[b]) * alpha / (K * n * n)
            r = s[lo:hi]
            tot = r.sum(1, keepdim=True)
            inv = torch.where(tot == 0, 0.0, 1 / tot)
            ds[lo:hi] += c * (g - (g * r).sum(1, keepdim=True) * inv) * inv
            mag[lo:hi] += abs(c) * (g.abs() + (g.abs() * r).sum(1, keepdim=True) * inv) * inv
    return ds * s * (1 - s), mag * s * (1 - s)


@pytest.mark.parametrize("T,E,K,lens,lead", BALANCE)
def test_route_backward(T, E, K, lens, lead):
    """Sums of depth <= 10 over experts and <= 6 over slots, up to 16 adds of repeated slots, and some ten
    single roundings: 40 u of the magnitudes."""
    _say("route_backward", T, E, K, len(lens))
    scores, ids, off = _problem(T, E, K, lens, T + E + 1, lead)
    if T > 3:
        scores[3] = 0.0
    g = _gen(T)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    dw, dloss = torch.randn((T, K), generator=g, device=DEV), torch.randn((len(lens),), generator=g, device=DEV)
    counts = _balance_ref(scores, ids, off, 1.0, K)[1].int()
    for w, l in ((dw, dloss), (dw, None), (None, dloss)):
        got = fw.beam_moe_route_backward(_dims(E, K), scores, ids, dw=w, dloss=l, alpha=0.5, seq_offsets=o,
                                         counts=counts if l is not None else None)
        want, mag = _route_back_ref(scores, ids, w, 2.5, off, 0.5, l, counts, K)
        _near(got, want, 40 * U * mag, (w is None, l is None))


@pytest.mark.parametrize("E", [100, 256])
def test_route_backward_keeps_nan_in_its_token(E):
    """A token's NaN stays in its row; padding has zeros whatever its scores hold, and where it has weights,
    their part alone."""
    _say("route_backward nan", E)
    T, K, lens = 90, 4, [20, 30, 20]
    scores, ids, off = _problem(T, E, K, lens, 3)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    dw, dloss = torch.ones((T, K), device=DEV), torch.ones(3, device=DEV)
    counts = _balance_ref(scores, ids, off, 1.0, K)[1].int()
    args = dict(dloss=dloss, counts=counts, alpha=1.0, seq_offsets=o)
    clean, loss_only = (fw.beam_moe_route_backward(_dims(E, K), scores, ids, dw=w, **args) for w in (dw, None))
    assert not loss_only[70:].any()
    scores[25, 7] = float("nan")
    scores[80:] = float("nan")
    got, got_loss = (fw.beam_moe_route_backward(_dims(E, K), scores, ids, dw=w, **args) for w in (dw, None))
    rows = torch.arange(T, device=DEV)
    keep = (rows != 25) & (rows < 80)
    assert torch.equal(got[keep], clean[keep]) and torch.equal(got_loss[keep], loss_only[keep])
    assert got_loss[25].isnan().all() and not got_loss[80:].any()
    assert fw.beam_moe_route_backward(_dims(E, K), scores, ids, dw=dw)[:20].isfinite().all()


def test_route_gradient_against_differences():
    """beam_moe_select's weights and beam_moe_balance_loss on scores moved along a direction of the logits;
    the same choice on both sides."""
    _say("route differences")
    T, E, K = 40, 64, 4
    dims = Dims(256, 128, E, 8, 4, K, 2.5)
    g = _gen(9)
    logits = torch.randn((T, E), generator=g, device=DEV, dtype=torch.float64)
    v = torch.randn((T, E), generator=g, device=DEV, dtype=torch.float64)
    scores = torch.sigmoid(logits).float()
    ids, _ = fw.beam_moe_select(dims, scores)
    dw = torch.randn((T, K), generator=g, device=DEV)
    _, counts, _ = fw.beam_moe_balance_loss(dims, scores, ids, alpha=2.0)
    grad = fw.beam_moe_route_backward(dims, scores, ids, dw=dw, dloss=torch.ones(1, device=DEV), counts=counts,
                                      alpha=2.0)
    h = 2.0 ** -9
    side = []
    for sign in (1, -1):
        sc = torch.sigmoid(logits + sign * h * v).float()
        picked = sc.double().gather(1, ids.long())
        w = 2.5 * picked / picked.sum(1, keepdim=True)
        loss, _, _ = fw.beam_moe_balance_loss(dims, sc, ids, alpha=2.0)
        side.append((w * dw.double()).sum() + loss.double().sum())
    quot, slope = float(side[0] - side[1]) / (2 * h), float((grad.double() * v).sum())
    # fp32 scores and loss: about 100 u of the sums over the step; curvature h^2 / 6 of a smooth sum of T K terms
    scale = float((2.5 * dw.abs()).sum()) / K + 2.0
    assert abs(quot - slope) <= 100 * U * scale / h + h * h * 10 * scale, (quot, slope)


def test_bad_offsets_do_not_fault():
    """Offsets that descend or leave the batch give undefined values, no access outside the tensors: the rows
    read are clamped to the batch, the units to the workspace."""
    _say("bad offsets")
    scores, ids, _ = _problem(1500, 256, 8, [1500], 2)
    for off in ([0, 900, 300, 1500], [-5, 700, 1 << 30], [1 << 30, -(1 << 30), 3], [1500, 0], [2000, 2000]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        loss, counts, _ = fw.beam_moe_balance_loss(_dims(256, 8), scores, ids, alpha=1.0, seq_offsets=o)
        out = fw.beam_moe_route_backward(_dims(256, 8), scores, ids, dloss=loss, counts=counts, alpha=1.0,
                                         seq_offsets=o)
        torch.cuda.synchronize()
        assert out.shape == scores.shape


def test_many_and_long_sequences():
    """70,000 sequences of one or two tokens; and one so long that its counts times E pass 24 bits."""
    _say("many sequences")
    lens = [1 + (i % 2) for i in range(70000)]
    scores, ids, off = _problem(105001, 8, 2, lens, 4)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    loss, counts, prob = fw.beam_moe_balance_loss(_dims(8, 2), scores, ids, alpha=0.01, seq_offsets=o)
    p = scores.double() / scores.double().sum(1, keepdim=True)
    total = torch.cat([torch.zeros_like(p[:1]), p.cumsum(0)])
    n = (o[1:] - o[:-1])[:, None]
    want = (total[o[1:].long()] - total[o[:-1].long()]) / n
    # the running 64-bit sums hold 1e5 terms of at most 1
    _near(prob, want, 100 * U * want + 1e-10)
    seq = torch.bucketize(torch.arange(105001, device=DEV), o[1:].long(), right=True)[:, None]
    ok = (ids >= 0) & (ids < 8) & (seq < 70000)
    c = torch.bincount((seq * 8 + ids)[ok], minlength=70000 * 8).view(70000, 8)
    assert torch.equal(counts.long(), c)
    _near(loss, 0.01 * 8 / (2 * n[:, 0]) * (c * want).sum(1), 100 * U * 0.01 * 8 + 0 * loss.double())
    dl = fw.beam_moe_route_backward(_dims(8, 2), scores, ids, dloss=torch.ones_like(loss), counts=counts, alpha=1.0,
                                    seq_offsets=o)
    g = (counts * 8.0 - 2 * n)[seq[:-1, 0]].double() / (2 * n * n)[seq[:-1, 0]]
    ref = (g - (g * p[:-1]).sum(1, keepdim=True)) / scores[:-1].double().sum(1, keepdim=True)
    mag = (g.abs() + (g.abs() * p[:-1]).sum(1, keepdim=True)) / scores[:-1].double().sum(1, keepdim=True)
    s = scores[:-1].double()
    _near(dl[:-1], ref * s * (1 - s), 40 * U * mag * s * (1 - s))
    assert not dl[-1].any()

    _say("a long sequence")
    T, E, K = 1_100_000, 8, 8
    scores, ids, off = _problem(T, E, K, [T], 5)
    loss, counts, prob = fw.beam_moe_balance_loss(_dims(E, K), scores, ids, alpha=1.0)
    rl, rc, rp = _balance_ref(scores, ids, off, 1.0, K)
    assert torch.equal(counts.long(), rc)
    # 4096 rows to a unit, 512 to each of its 8 waves, one after the other in FP32: depth 540, then FP64
    _near(prob, rp, 600 * U * rp)
    _near(loss, rl, 600 * U * rl)
    dl = fw.beam_moe_route_backward(_dims(E, K), scores, ids, dloss=loss, counts=counts, alpha=1.0)
    want, mag = _route_back_ref(scores, ids, None, 2.5, off, 1.0, loss, counts, K)
    _near(dl, want, 40 * U * mag)


# --------------------------------------------------------------------------
# linear
# --------------------------------------------------------------------------
ACTS = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}
GEMM_UP = 2.0 ** -23  # a step inside the matrix core may cut instead of round


def _depth(K):
    """Additions that a product meets: its own group of 32, then one per group (whatever the split)."""
    return 32 + K / 32 + 40


def _linear_ref(x, w, bias, act, res, keep, add):
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    y = add * ACTS[act](z)
    if res is not None:
        y = y + keep * res.double()
    return y, z, mag


def _linear_check(x, w, bias, act, res, keep, add, y, pre=None):
    ry, rz, mag = _linear_ref(x, w, bias, act, res, keep, add)
    dz = _depth(x.shape[1]) * GEMM_UP * mag
    if pre is not None:
        _near(pre, rz, dz, "pre")
    extra = 0.0 if res is None else 2 * U * (keep * res.double()).abs()
    # slopes of the activations stay below 1.13; their own evaluation is good to 8 u of |z| + 1
    _near(y, ry, abs(add) * (1.13 * dz + 8 * U * (rz.abs() + (act != "none"))) + 2 * U * ry.abs() + extra, "y")


# the last of each list are large enough for 256-row tiles: the forward product's, dx's and dw's
LARGE = [(1000, 1032, 2048), (2100, 2560, 1280), (3300, 3336, 136)]
LARGE_BACK = LARGE + [(3300, 200, 3336), (200, 3300, 3336), (136, 3584, 3584)]
LINEAR_SHAPES = [(1, 1, 1), (1, 64, 64), (1, 100, 1000), (2, 2560, 512), (3, 17, 5), (7, 33, 2049), (16, 256, 128),
                 (17, 48, 96), (33, 1000, 136), (64, 512, 2560), (65, 130, 72), (100, 64, 7), (129, 257, 65),
                 (255, 96, 520), (256, 256, 64), (300, 513, 1024), (257, 264, 192), (520, 1040, 328)]


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES + LARGE)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear(M, N, K, dt):
    g = _gen(M * 3 + N * 5 + K)
    for act, yt, res, pad in (("none", dt, False, 0), ("silu", F32, True, 0), ("gelu", dt, True, 8),
                              ("relu", dt, False, 3), ("none", F32, True, 1)):
        _say("linear", M, N, K, dt, act, yt, res, pad)
        x, w = _randn(g, (M, K), dt, 1.0, pad), _randn(g, (N, K), dt, K ** -0.5, pad)
        bias = _randn(g, (N,)) if act != "relu" else None
        r = _randn(g, (M, N), yt, 1.0, pad) if res else None
        keep, add = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if res else (1.0, 1.0)
        y, pre = fw.beam_moe_linear(x, w, bias, act=act, residual=r, keep=keep, add=add, out_dtype=yt, want_pre=True)
        _linear_check(x, w, bias, act, r, keep, add, y, pre)
        assert torch.equal(y, fw.beam_moe_linear(x, w, bias, act=act, residual=r, keep=keep, add=add, out_dtype=yt))


# rows that are no whole chunks of 16 bytes: through registers in 64- and 128-row tiles, split or not, and laid out
# anew where that costs less
@pytest.mark.parametrize("M,N,K,pad", [(17, 33, 71, 2), (200, 300, 1409, 0), (130, 70, 2050, 1), (500, 2505, 2603, 0),
                                       (513, 1001, 4100, 5), (4000, 1000, 1401, 0), (2100, 1030, 63, 1)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_rows_off_16_bytes(M, N, K, pad, dt):
    _say("linear rows off 16 bytes", M, N, K, pad, dt)
    g = _gen(M + K)
    x, w = _randn(g, (M, K), dt, 1.0, pad), _randn(g, (N, K), dt, K ** -0.5, pad)
    bias, r = _randn(g, (N,)), _randn(g, (M, N), F32, 1.0, pad)
    y, pre = fw.beam_moe_linear(x, w, bias, act="silu", residual=r, keep=0.5, add=2.0, out_dtype=F32, want_pre=True)
    _linear_check(x, w, bias, "silu", r, 0.5, 2.0, y, pre)
    # one operand's rows whole, the other's not
    z = fw.beam_moe_linear(x[:, : K // 8 * 8].contiguous(), w[:, : K // 8 * 8])
    _linear_check(x[:, : K // 8 * 8], w[:, : K // 8 * 8], None, "none", None, 1.0, 1.0, z)


# small results with a long K, split as often as it allows, in 64- and 128-row tiles
@pytest.mark.parametrize("M,N,K", [(100, 100, 65536), (300, 300, 16384), (512, 512, 9216), (640, 512, 9216),
                                   (17, 2049, 8200)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_long_k(M, N, K, dt):
    _say("linear long K", M, N, K, dt)
    g = _gen(M + K)
    x, w, bias = _randn(g, (M, K), dt), _randn(g, (N, K), dt, K ** -0.5), _randn(g, (N,))
    y, pre = fw.beam_moe_linear(x, w, bias, act="gelu", out_dtype=F32, want_pre=True)
    _linear_check(x, w, bias, "gelu", None, 1.0, 1.0, y, pre)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 70, 65), (70, 70, 65), (300, 264, 128)])
def test_linear_in_place_padding_and_nan(M, N, K):
    _say("linear in place", M, N, K)
    g = _gen(M)
    x, w = _randn(g, (M, K), BF16), _randn(g, (N, K), BF16, K ** -0.5)
    buf = torch.full((M, N + 8), 7.0, device=DEV)
    buf[:, :N] = _randn(g, (M, N))
    stream = buf[:, :N]
    before = stream.clone()
    out = fw.beam_moe_linear(x, w, residual=stream, keep=0.5, add=2.0, out=stream)
    assert out is stream and (buf[:, N:] == 7).all()
    _linear_check(x, w, None, "none", before, 0.5, 2.0, out)
    y = fw.beam_moe_linear(x, w, act="silu")
    x[M // 2, K - 1] = float("nan")
    z = fw.beam_moe_linear(x, w, act="silu")
    assert z[M // 2].isnan().all()
    keep = torch.arange(M, device=DEV) != M // 2
    assert torch.equal(z[keep], y[keep])
    w[N - 1, 0] = float("inf")
    z = fw.beam_moe_linear(x, w, act="silu")
    assert torch.equal(z[keep][:, : N - 1], y[keep][:, : N - 1])
    assert fw.beam_moe_linear(x[:0], w).shape == (0, N)


def test_activations_far_from_zero():
    """Arguments at which exponentials over- and underflow: finite values and slopes, at their limits."""
    _say("activations")
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 90.0, -90.0, 200.0, -200.0, 3e4, -3e4], device=DEV)
    w = torch.zeros((z.numel(), 8), dtype=BF16, device=DEV)
    x = torch.zeros((3, 8), dtype=BF16, device=DEV)
    for act, fn in ACTS.items():
        y = fw.beam_moe_linear(x, w, z, act=act, out_dtype=F32)
        want = fn(z.double())
        # sigmoid moves by |z| half steps of e^-z: 0.6 u of 1 in z s; erf and the rest to a few steps
        _near(y, want.expand(3, -1), 8 * U * (want.abs() + 1) * z.abs().clamp(max=1) + 2.0 ** -149, act)
        pre = z.to(BF16).expand(3, -1).contiguous()
        dy = torch.ones((3, z.numel()), device=DEV)
        _, _, db = fw.beam_moe_linear_backward(dy, x, w, pre, act=act)
        slope = _slope(pre[0], act) if act != "none" else torch.ones_like(z)
        _near(db, 3 * slope.double(), 3 * 8 * U * (slope.double().abs() + 1), act)


def test_gelu_keeps_its_digits_below_zero():
    """z times the normal distribution function, relative to itself: the fit and its evaluation 6 steps, the
    reciprocal, the exponential and four products 10, the exponent z^2 / 2 three half steps of itself."""
    _say("gelu below zero")
    z = torch.linspace(-12.0, 12.0, 24001, device=DEV)
    w = torch.zeros((z.numel(), 8), dtype=BF16, device=DEV)
    y = fw.beam_moe_linear(torch.zeros((2, 8), dtype=BF16, device=DEV), w, z, act="gelu", out_dtype=F32)
    d = z.double()
    want = d * 0.5 * torch.erfc(-d * math.sqrt(0.5))
    _near(y, want.expand(2, -1), (16 + 1.5 * d * d) * U * want.abs(), "gelu")


def _slope(z, act):
    z = z.double().requires_grad_(True)
    return torch.autograd.grad(ACTS[act](z).sum(), z)[0]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_slopes_at_infinite_pre(act, dt):
    """An fp16 pre past 65504 is stored as an infinity while y, in FP32, is finite: the slope there is its limit, 0 or 1,
    as it is from |z| = 110 on.  NaN stays NaN."""
    _say("slopes at infinite pre", act, dt)
    z = torch.tensor([7e4, -7e4, 6e4, -6e4, 1.0, float("nan"), 3e38, -3e38], device=DEV)
    x, w = torch.zeros((3, 16), dtype=dt, device=DEV), torch.ones((8, 16), dtype=dt, device=DEV)
    y, pre = fw.beam_moe_linear(x, w, z, act=act, out_dtype=F32, want_pre=True)
    if dt == F16:
        assert pre[0, 0] == float("inf") and pre[0, 1] == float("-inf")
    x.fill_(1.0)
    dy = torch.ones((3, 8), device=DEV)
    dx, dw, db = fw.beam_moe_linear_backward(dy, x, w, pre, act=act)
    for i, slope in ((0, 1.0), (1, 0.0), (2, 1.0), (3, 0.0), (6, 1.0), (7, 0.0)):
        assert y[:, i].isfinite().all() and db[i] == 3 * slope and (dw[i] == 3 * slope).all(), i
    if act == "relu":
        assert db[5] == 0  # NaN > 0 does not hold
    else:
        assert db[5].isnan() and dw[5].isnan().all() and dx.isnan().all()
    dx, _, _ = fw.beam_moe_linear_backward(dy[:, :4], x, w[:4], pre[:, :4], act=act)
    assert (dx == 2).all()


def _linear_back_check(dy, x, w, pre, act, keep, add, out):
    """dz is rounded to the products' type: half a step of each term, at worst all one way; then the sums.
    With no activation and add = 1, dz is dy, and in dy's type exact."""
    d = add * dy.double()
    if act != "none":
        d = d * _slope(pre, act)
    exact = act == "none" and add == 1.0 and dy.dtype == x.dtype
    off = 0.0 if exact else _step(x) + 16 * U
    tiny = 0.0 if exact else _tiny(x) + 8 * U * abs(add)  # slopes near zero are differences of order 1
    dx, dw, db, dres = out
    M, N = dy.shape
    a = d.abs()
    slack = tiny * (dy.double().abs() if act != "none" else 1.0)
    ez = off * a + (slack if not exact else 0.0)
    if dx is not None:
        _near(dx, d @ w.double(), (_depth(N) * GEMM_UP * a + ez) @ w.double().abs(), "dx")
    if dw is not None:
        _near(dw, d.t() @ x.double(), (_depth(M) * GEMM_UP * a + ez).t() @ x.double().abs(), "dw")
    if db is not None:
        depth = math.ceil(M / 64) + 64 + 24
        _near(db, d.sum(0), (depth * U * a + 16 * U * a + 8 * U * dy.double().abs() * abs(add)).sum(0), "dbias")
    if dres is not None:
        _near(dres, keep * dy.double(), 2 * U * (keep * dy.double()).abs(), "dres")


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES + LARGE_BACK)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_backward(M, N, K, dt):
    g = _gen(M * 3 + N * 5 + K + 1)
    for act, yt, add, pad in (("none", dt, 1.0, 0), ("silu", F32, 0.5, 0), ("gelu", dt, 1.0, 8),
                              ("relu", dt, 1.0, 3), ("none", F32, 2.0, 1), ("none", dt, 1.0, 5)):
        _say("linear_backward", M, N, K, dt, act, yt, pad)
        x, w = _randn(g, (M, K), dt, 1.0, pad), _randn(g, (N, K), dt, K ** -0.5, pad)
        dy = _randn(g, (M, N), yt, 1.0, pad)
        pre = _randn(g, (M, N), dt, 1.5) if act != "none" else None
        out = fw.beam_moe_linear_backward(dy, x, w, pre, act=act, keep=0.75, add=add, want_dres=True)
        _linear_back_check(dy, x, w, pre, act, 0.75, add, out)


# products that run together: in 64-row tiles with K of one or both split, and in 128-row tiles with none, either
# or both split, where dx's or dw's K is the longer
@pytest.mark.parametrize("M,N,K", [(181, 1838, 1863), (2000, 1280, 128), (60, 2500, 2505), (1000, 300, 5000),
                                   (500, 2560, 1400), (3600, 900, 640), (3600, 2560, 192), (1021, 1699, 1401),
                                   (2000, 4000, 2560), (6001, 999, 1399)])
@pytest.mark.parametrize("act,dt,pad", [("none", BF16, 0), ("gelu", F16, 5)])
def test_linear_backward_together(M, N, K, act, dt, pad):
    _say("linear_backward together", M, N, K, act, dt, pad)
    g = _gen(M + N + K)
    x, w = _randn(g, (M, K), dt, 1.0, pad), _randn(g, (N, K), dt, K ** -0.5, pad)
    dy, pre = _randn(g, (M, N), dt, 1.0, pad), _randn(g, (M, N), dt, 1.5, pad)
    dx, dw, db = fw.beam_moe_linear_backward(dy, x, w, pre, act=act)
    _linear_back_check(dy, x, w, pre, act, 1.0, 1.0, (dx, dw, db, None))
    again = fw.beam_moe_linear_backward(dy, x, w, pre, act=act)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
    assert torch.equal(fw.beam_moe_linear_backward(dy, None, w, pre, act=act, want_dw=False)[0], dx)
    assert torch.equal(fw.beam_moe_linear_backward(dy, x, None, pre, act=act, want_dx=False)[1], dw)


# many rows and a small dw, K of dw split often: both in 64-row tiles, dx in 256-row tiles and dw in 64-row ones, both
# in 128-row tiles
@pytest.mark.parametrize("M,N,K", [(10176, 832, 192), (18048, 192, 512), (19392, 192, 768), (15000, 65, 1727)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_backward_of_many_rows(M, N, K, dt):
    _say("linear_backward of many rows", M, N, K, dt)
    g = _gen(M + N + K)
    x, w, dy, pre = (_randn(g, s, dt) for s in ((M, K), (N, K), (M, N), (M, N)))
    dx, dw, db = fw.beam_moe_linear_backward(dy, x, w, pre, act="silu")
    _linear_back_check(dy, x, w, pre, "silu", 1.0, 1.0, (dx, dw, db, None))
    again = fw.beam_moe_linear_backward(dy, x, w, pre, act="silu")
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def _dz_check(dy, x, w, pre, act, add, out):
    """fp16: dz is scaled by the power of two that takes b = 1.13 |add| max |dy| (no slope is larger) into [2^14, 2^15),
    and rounded: half a step of each term, or 2^-25 of fp16's least subnormal, which is at most 2^-39 b."""
    d = add * dy.double()
    if act != "none":
        d = d * _slope(pre, act)
    a = d.abs()
    ez = (_step(x) + 16 * U) * a + 2.0 ** -39 * 1.13 * abs(add) * float(dy.double().abs().max())
    if act != "none":
        ez = ez + 8 * U * abs(add) * dy.double().abs()  # slopes near zero are differences of order 1
    dx, dw, db = out
    M, N = dy.shape
    if dx is not None:
        _near(dx, d @ w.double(), (_depth(N) * GEMM_UP * a + ez) @ w.double().abs(), "dx")
    if dw is not None:
        _near(dw, d.t() @ x.double(), (_depth(M) * GEMM_UP * a + ez).t() @ x.double().abs(), "dw")
    if db is not None:
        depth = math.ceil(M / 64) + 64 + 24
        _near(db, d.sum(0), (depth * U * a + 16 * U * a + 8 * U * dy.double().abs() * abs(add)).sum(0), "dbias")


# both products together in 64- and 128-row tiles, split or not, and in 256-row tiles by themselves
RANGE_SHAPES = [(1, 9, 16), (33, 100, 136), (517, 1003, 777), (60, 2500, 2505), (1000, 300, 5000), (2000, 4000, 2560),
                (3300, 3336, 136), (8192, 136, 264)]


@pytest.mark.parametrize("M,N,K", RANGE_SHAPES)
@pytest.mark.parametrize("size,add,weights", [(1e-6, 1.0, 2.0 ** 10), (1e-7, 1.0, 2.0 ** 11), (2e-8, 0.577, 2.0 ** 11),
                                              (1e-12, 1e5, 2.0 ** 11), (1e-30, 1.5e23, 2.0 ** 11), (1e6, 1.0, 2.0 ** -14)])
def test_linear_backward_keeps_small_and_large_gradients_in_fp16(M, N, K, size, add, weights):
    """FP32 gradients that fp16 cannot hold, or only as subnormals, with weights and inputs for which the results can
    be held: dx, dw and dbias of one call agree with 64 bits alike."""
    _say("linear_backward range", M, N, K, size, add)
    g = _gen(M + N + K)
    x, w = _randn(g, (M, K), F16, weights, 5), _randn(g, (N, K), F16, weights)
    dy, pre = _randn(g, (M, N), F32, size, 3), _randn(g, (M, N), F16, 1.5)
    for act in ("none", "gelu"):
        p = pre if act != "none" else None
        dx, dw, db = fw.beam_moe_linear_backward(dy, x, w, p, act=act, add=add)
        _dz_check(dy, x, w, p, act, add, (dx, dw, db))
        assert torch.equal(fw.beam_moe_linear_backward(dy, None, w, p, act=act, add=add, want_dw=False)[0], dx)
        assert torch.equal(fw.beam_moe_linear_backward(dy, x, None, p, act=act, add=add, want_dx=False)[1], dw)


@pytest.mark.parametrize("M,N,K", [(517, 1003, 777), (8192, 136, 264)])
def test_linear_backward_of_small_fp16_gradients(M, N, K):
    """fp16 dy near its least subnormal: dz = add dy act' lies below it and still counts."""
    _say("linear_backward small fp16", M, N, K)
    g = _gen(M)
    x, w = _randn(g, (M, K), F16, 2.0 ** 11), _randn(g, (N, K), F16, 2.0 ** 11)
    dy, pre = _randn(g, (M, N), F16, 2.0 ** -21), _randn(g, (M, N), F16, 1.5)
    assert (dy != 0).any()
    for act, add in (("silu", 0.1), ("relu", 0.3), ("none", 0.01)):
        p = pre if act != "none" else None
        _dz_check(dy, x, w, p, act, add, fw.beam_moe_linear_backward(dy, x, w, p, act=act, add=add))


def test_linear_backward_gradients_far_apart_in_fp16():
    """One gradient far above the others; infinities and NaN, which touch their own row and column alone and have no
    part in the scale; gradients and factors of zero."""
    _say("linear_backward far apart")
    g = _gen(21)
    M, N, K = 300, 264, 136
    x, w = _randn(g, (M, K), F16, 16.0), _randn(g, (N, K), F16, 16.0)
    dy = _randn(g, (M, N), F32, 1e-4)
    dy[7, 9] = 50.0
    _dz_check(dy, x, w, None, "none", 1.0, fw.beam_moe_linear_backward(dy, x, w))
    dy[5] = 0.0
    clean = fw.beam_moe_linear_backward(dy, x, w)
    for bad in (float("inf"), float("-inf"), float("nan")):
        d = dy.clone()
        d[5, 3] = bad
        dx, dw, db = fw.beam_moe_linear_backward(d, x, w)
        rows, cols = torch.arange(M, device=DEV) != 5, torch.arange(N, device=DEV) != 3
        assert torch.equal(dx[rows], clean[0][rows]) and not dx[5].isfinite().any()
        assert torch.equal(dw[cols], clean[1][cols]) and not dw[3].isfinite().any()
        assert torch.equal(db[cols], clean[2][cols]) and not db[3].isfinite()
    for d, add in ((torch.zeros_like(dy), 1.0), (dy, 0.0)):
        assert all(not t.any() for t in fw.beam_moe_linear_backward(d, x, w, add=add))


def test_linear_backward_scale_of_replayed_gradients():
    """The scale is the replayed call's own: gradients of other sizes in the captured buffers, and two graphs in turn."""
    _say("linear_backward replayed scale")
    g = _gen(22)
    M, N, K = 517, 264, 136
    x, w, pre = _randn(g, (M, K), F16, 256.0), _randn(g, (N, K), F16, 256.0), _randn(g, (M, N), F16, 1.5)
    dys = [_randn(g, (M, N), F32, s) for s in (1e-7, 1.0, 1e-5)]
    want = [fw.beam_moe_linear_backward(d, x, w, pre, act="silu") for d in dys]
    bufs, graphs, outs = [], [], []
    for i in (0, 1):
        bufs.append(dys[i].clone())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fw.beam_moe_linear_backward(bufs[i], x, w, pre, act="silu")
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(fw.beam_moe_linear_backward(bufs[i], x, w, pre, act="silu"))
    for i, j in ((0, 0), (1, 1), (0, 2), (1, 0), (0, 1), (1, 2)):
        bufs[i].copy_(dys[j])
        graphs[i].replay()
        eager = fw.beam_moe_linear_backward(dys[2 - j], x, w, pre, act="silu")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[j]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[2 - j]))


def test_linear_backward_parts():
    _say("linear_backward parts")
    g = _gen(4)
    M, N, K = 130, 72, 200
    x, w, dy, pre = (_randn(g, s, BF16) for s in ((M, K), (N, K), (M, N), (M, N)))
    dx, dw, db = fw.beam_moe_linear_backward(dy, x, w, pre, act="silu")
    a = fw.beam_moe_linear_backward(dy, None, w, pre, act="silu", want_dw=False, want_dbias=False)
    b = fw.beam_moe_linear_backward(dy, x, None, pre, act="silu", want_dx=False, want_dbias=False)
    c = fw.beam_moe_linear_backward(dy, x, None, pre, act="silu", want_dx=False, want_dw=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert torch.equal(b[1], dw) and torch.equal(c[2], db)
    dx, dw, db = fw.beam_moe_linear_backward(dy[:0], x[:0], w, pre[:0], act="silu")
    assert dx.shape == (0, K) and not dw.any() and not db.any() and dw.shape == (N, K)


def test_linear_offsets_past_32_bits():
    _say("linear wide rows")
    g = _gen(13)
    M, K, N, ld = 66000, 64, 40, 65600
    buf = torch.empty((M, ld), dtype=BF16, device=DEV)
    x, res, y = buf[:, :K], buf[:, 128: 128 + N], buf[:, 256: 256 + N]
    x.copy_(torch.randn((M, K), generator=g, device=DEV))
    res.copy_(torch.randn((M, N), generator=g, device=DEV))
    w = _randn(g, (N, K), BF16, 0.1)
    fw.beam_moe_linear(x, w, act="relu", residual=res, out=y)
    assert torch.equal(y, fw.beam_moe_linear(x.contiguous(), w, act="relu", residual=res.contiguous()))
    a = fw.beam_moe_linear_backward(y, x, w, res, act="silu")
    b = fw.beam_moe_linear_backward(y.contiguous(), x.contiguous(), w, res.contiguous(), act="silu")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_linear_gradient_against_differences():
    _say("linear differences")
    g = _gen(8)
    M, N, K = 9, 24, 40
    x, w, bias = _randn(g, (M, K), F16), _randn(g, (N, K), F16, 0.2), _randn(g, (N,))
    v, dy = _randn(g, (N,)), _randn(g, (M, N))
    _, pre = fw.beam_moe_linear(x, w, bias, act="gelu", want_pre=True)
    _, _, db = fw.beam_moe_linear_backward(dy, x, w, pre, act="gelu")
    h = 2.0 ** -8
    up, dn = (fw.beam_moe_linear(x, w, bias + s * h * v, act="gelu", out_dtype=F32) for s in (1, -1))
    quot = float((dy.double() * (up.double() - dn.double())).sum()) / (2 * h)
    slope = float((db.double() * v.double()).sum())
    # pre is rounded to fp16 (2^-11 of |z| <= 8 times the curvature <= 1), the outputs to fp32 over the step,
    # the third derivative <= 2 of gelu over h^2 / 6
    scale = float((dy.double().abs() * v.double().abs()).sum())
    assert abs(quot - slope) <= scale * (2.0 ** -8 + 200 * U / h + h * h), (quot, slope)


# --------------------------------------------------------------------------
# streams, graphs, and a run together
# --------------------------------------------------------------------------
def _step_inputs(seed, T=192, H=512, F=384, E=64, K=4):
    g = _gen(seed)
    return dict(stream=_randn(g, (T, H), F32, 2.0), gamma=1 + _randn(g, (H,), F32, 0.1), beta=_randn(g, (H,), F32, 0.1),
                w1=_randn(g, (F, H), BF16, H ** -0.5), b1=_randn(g, (F,), F32, 0.1),
                w2=_randn(g, (H, F), BF16, F ** -0.5), wr=_randn(g, (E, H), F32, H ** -0.5),
                dout=_randn(g, (T, H), F32), dw=_randn(g, (T, K), F32),
                off=torch.tensor([0, 70, 70, T - 9], dtype=torch.int32, device=DEV), dims=Dims(H, 128, E, 8, 4, K, 2.5))


def _train_step(s, step=3):
    """A dense sublayer (norm, up, activation, down onto the stream) and a router on the same norm, forward and
    back to the stream and every weight."""
    keep, add = math.sqrt((step - 1) / step), math.sqrt(1 / step)
    x, mean, rstd = fw.beam_moe_layer_norm(s["stream"], s["gamma"], s["beta"], out_dtype=BF16)
    h, pre = fw.beam_moe_linear(x, s["w1"], s["b1"], act="silu", want_pre=True)
    out = fw.beam_moe_linear(h, s["w2"], residual=s["stream"], keep=keep, add=add, out_dtype=F32)
    ids, w, scores = fw.beam_moe_route(s["dims"], x, s["wr"], want_scores=True)
    loss, counts, prob = fw.beam_moe_balance_loss(s["dims"], scores, ids, alpha=0.1, seq_offsets=s["off"])
    dlogits = fw.beam_moe_route_backward(s["dims"], scores, ids, dw=s["dw"], dloss=torch.ones_like(loss),
                                         counts=counts, alpha=0.1, seq_offsets=s["off"])
    dh, dw2, _, dstream = fw.beam_moe_linear_backward(s["dout"], h, s["w2"], keep=keep, add=add, want_dbias=False,
                                                      want_dres=True)
    dx, dw1, db1 = fw.beam_moe_linear_backward(dh, x, s["w1"], pre, act="silu")
    dx = dx.float() + dlogits @ s["wr"]
    dnorm, dgamma, dbeta = fw.beam_moe_layer_norm_backward(dx, s["stream"], mean, rstd, s["gamma"])
    return dict(out=out, w=w, ids=ids, loss=loss, counts=counts, dstream=dstream + dnorm, dgamma=dgamma, dbeta=dbeta,
                dw1=dw1, db1=db1, dw2=dw2, dlogits=dlogits)


def _train_step_ref(s, ids, step=3):
    f = {k: s[k].double().requires_grad_(True) for k in ("stream", "gamma", "beta", "w1", "b1", "w2")}
    x = torch.nn.functional.layer_norm(f["stream"], (f["stream"].shape[1],), f["gamma"], f["beta"], 1e-5)
    out = math.sqrt((step - 1) / step) * f["stream"] + math.sqrt(1 / step) * (
        torch.nn.functional.silu(x @ f["w1"].t() + f["b1"]) @ f["w2"].t())
    logits = x @ s["wr"].double().t()
    sc = torch.sigmoid(logits)
    picked = sc.gather(1, ids.long())
    w = 2.5 * picked / picked.sum(1, keepdim=True)
    p = sc / sc.sum(1, keepdim=True)
    off, E, K = s["off"].tolist(), sc.shape[1], ids.shape[1]
    loss = []
    for a, b in zip(off[:-1], off[1:]):
        c = torch.bincount(ids[a:b].reshape(-1).long(), minlength=E).double()
        loss.append(0.1 * E * (c * p[a:b].sum(0)).sum() / (K * max(b - a, 1) ** 2))
    loss = torch.stack(loss)
    aim = (out * s["dout"].double()).sum() + (w * s["dw"].double()).sum() + loss.sum()
    grads = torch.autograd.grad(aim, [logits, *f.values()])
    return dict(out=out.detach(), w=w.detach(), loss=loss.detach(), dlogits=grads[0], **dict(zip(("dstream", "dgamma", "dbeta", "dw1", "db1",
                                                                       "dw2"), grads[1:])))


def test_training_step_of_a_sublayer():
    """The whole run against 64-bit autograd. Rounding a tensor to bf16 changes it by at most eps / 2 of its
    2-norm; at most seven such roundings (x, h, pre, dz twice, dh, dx) lie on any path to a result, and random
    matrices of these shapes pass a relative error on with a factor of order one: 16 half steps in all."""
    _say("training step")
    s = _step_inputs(1)
    got = _train_step(s)
    want = _train_step_ref(s, got["ids"])
    torch.cuda.synchronize()
    for k, v in want.items():
        err = float((got[k].double() - v).norm() / v.norm())
        assert err <= 16 * 2.0 ** -9, (k, err)


def test_two_streams_at_once():
    _say("two streams")
    a, b = _step_inputs(2), _step_inputs(3)
    ra, rb = _train_step(a), _train_step(b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for st, inp in ((sa, a), (sb, b)):
            with torch.cuda.stream(st):
                got.append(_train_step(inp))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for k, v in (ra, rb)[i % 2].items():
            assert torch.equal(r[k], v), (i, k)
    # a stream handed over by argument: as a torch stream and as a raw handle
    x, w = a["stream"].bfloat16(), a["w1"]
    want = fw.beam_moe_linear(x, w, act="silu")
    torch.cuda.synchronize()
    for st in (sa, sa.cuda_stream):
        y = fw.beam_moe_linear(x, w, act="silu", stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_captured_and_replayed():
    """Two graphs of the same calls on different inputs, replayed in turn between eager calls."""
    _say("graphs")
    ins = [_step_inputs(4), _step_inputs(5)]

    def work(s):
        x, mean, rstd = fw.beam_moe_layer_norm(s["stream"], s["gamma"], s["beta"], out_dtype=BF16)
        h, pre = fw.beam_moe_linear(x, s["w1"], s["b1"], act="silu", want_pre=True)
        sc = torch.sigmoid(s["stream"][:, :64]).contiguous()
        ids = s["ids"]
        loss, counts, _ = fw.beam_moe_balance_loss(s["dims"], sc, ids, alpha=0.1, seq_offsets=s["off"])
        dl = fw.beam_moe_route_backward(s["dims"], sc, ids, dw=s["dw"], dloss=loss, counts=counts, alpha=0.1,
                                        seq_offsets=s["off"])
        dx, dw, db = fw.beam_moe_linear_backward(h, x, s["w1"], pre, act="silu")
        dn, dg, dbeta = fw.beam_moe_layer_norm_backward(dx, s["stream"], mean, rstd, s["gamma"])
        return [x, h, loss, counts, dl, dx, dw, db, dn, dg, dbeta]

    for s in ins:
        s["ids"] = s["stream"][:, :64].topk(4, 1).indices.int().contiguous()
    want = [[t.clone() for t in work(s)] for s in ins]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in ins:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work(s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(work(s))
        graphs.append(gr)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        eager = work(ins[1 - i])
        torch.cuda.synchronize()
        for a, b in zip(outs[i], want[i]):
            assert torch.equal(a, b)
        for a, b in zip(eager, want[1 - i]):
            assert torch.equal(a, b)


def test_binding_refusals_on_the_device():
    _say("refusals")
    x = torch.zeros((4, 16), device=DEV)
    with pytest.raises(ValueError, match="consecutive"):
        fw.beam_moe_layer_norm(torch.zeros((16, 4), device=DEV).t())
    with pytest.raises(ValueError, match="overlap"):
        fw.beam_moe_layer_norm(x[:1].expand(4, 16))
    with pytest.raises(ValueError, match="one of"):
        fw.beam_moe_layer_norm(x.double())
    with pytest.raises(ValueError, match="shape"):
        fw.beam_moe_layer_norm(x, torch.zeros(15, device=DEV))
    with pytest.raises(fw.BeamMoeError):
        fw.beam_moe_layer_norm(torch.zeros((4, 17), device=DEV)[:, 1:])  # rows start off 16 bytes
    with pytest.raises(fw.BeamMoeError):
        fw.beam_moe_layer_norm(torch.zeros((2, 20000), device=DEV))
    with pytest.raises(ValueError, match="one of"):
        fw.beam_moe_linear(x, x)
    with pytest.raises(ValueError, match="one of"):
        fw.beam_moe_linear(x.bfloat16(), x.half())
    with pytest.raises(ValueError, match="shape"):
        fw.beam_moe_linear(x.bfloat16(), x.bfloat16()[:, :8])
    with pytest.raises(ValueError, match="pre"):
        fw.beam_moe_linear_backward(x[:, :4].bfloat16(), x.bfloat16(), x.bfloat16(), act="silu")
    with pytest.raises(fw.BeamMoeError):
        fw.beam_moe_route_backward(_dims(16, 2), x, torch.zeros((4, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="offsets"):
        fw.beam_moe_balance_loss(_dims(16, 2), x, torch.zeros((4, 2), dtype=torch.int32, device=DEV), alpha=1.0,
                                 seq_offsets=torch.zeros(1, dtype=torch.int32, device=DEV))
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    with pytest.raises(fw.BeamMoeError, match="workspace"):
        fw.beam_moe_linear_backward(x.bfloat16(), x.bfloat16(), torch.zeros((16, 16), device=DEV).bfloat16(),
                                    ws=small)
