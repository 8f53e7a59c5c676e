"""GPU parity of the operators of a dense gated sublayer (the norm of all gradients and their clipping, microscaled
4-bit floating point and its product, the gated projections) with their formulas in 64 bits.

Tolerances are bounds on the kernels' own roundings: u = 2^-24 is FP32's half step, a sum of depth d is off by at most
d u times the sum of magnitudes, and a result stored in type t by at most half a step, finfo(t).eps / 2 of its value
(plus half the least subnormal of fp16).
"""
import math

import pytest
import torch

from grouped_top_routing_fp32_amd import binding as fw

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


def _say(*what):
    print("\n[case]", *what, flush=True)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=F32, scale=1.0, pad=0):
    """Normal values; with pad, the first columns of a wider buffer whose rest is NaN."""
    t = torch.full((*shape[:-1], shape[-1] + pad), NAN, device=DEV)
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
# the norm of all gradients, and clipping
# --------------------------------------------------------------------------
def _norm_of(grads, scale=1.0):
    return abs(scale) * math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in grads))


def _factor(grads, max_norm, scale=1.0, eps=1e-6, norm=None):
    norm = _norm_of(grads, scale) if norm is None else norm
    return scale * min(1.0, max_norm / (norm + eps))


def _grads(seed, sizes, kinds, scale=1.0):
    g = _gen(seed)
    return [_randn(g, (n,), k, scale) for n, k in zip(sizes, kinds)]


def _clip_check(got, grads, f):
    """The FP64 sum is exact to far below FP32's step, so the factor is off by half a step of FP32, the product by
    another, and the store by half a step of its type."""
    for a, b in zip(got, grads):
        want = b.double() * f
        _near(a, want, 2.0 * U * want.abs() + 2.0 ** -149, a.dtype)


SIZES = [[1], [7, 1, 0, 33], [8192, 8193, 8191], [100000, 3, 65537], [5] * 300, [1000 + 13 * i for i in range(130)]]
MIXES = [(BF16,), (F16,), (F32,), (BF16, F32), (F16, F32, BF16)]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("mix", MIXES, ids=lambda m: "-".join(str(k)[6:] for k in m))
def test_clip_grads(sizes, mix):
    _say("clip", len(sizes), mix)
    kinds = [mix[i % len(mix)] for i in range(len(sizes))]
    for size, scale in ((1.0, 1.0), (1e-4, 1.0), (30.0, 1 / 256)):
        grads = _grads(len(sizes), sizes, kinds, size)
        want = _norm_of(grads, scale)
        norm = fw.beam_moe_grad_norm(grads, scale=scale)
        assert norm.shape == () and norm.dtype == F32
        _near(norm, torch.tensor(want, device=DEV), 1e-12 * want)
        for max_norm in (0.0, 0.5 * want, 2 * want + 1):
            f = _factor(grads, max_norm, scale)
            to = [torch.full_like(t, NAN, dtype=F32) for t in grads]
            got = fw.beam_moe_clip_grads(grads, max_norm, scale=scale, out=to)
            assert torch.equal(got, norm)
            _clip_check(to, grads, f)
            inplace = [t.clone() for t in grads]
            assert torch.equal(fw.beam_moe_clip_grads(inplace, max_norm, scale=scale), norm)
            _clip_check(inplace, grads, f)
            again = [t.clone() for t in grads]
            fw.beam_moe_clip_grads(again, max_norm, scale=scale)
            assert all(torch.equal(a, b) for a, b in zip(inplace, again))


@pytest.mark.parametrize("to", [BF16, F16, F32])
def test_clip_grads_between_types(to):
    _say("clip between types", to)
    grads = _grads(5, [3000, 4099, 17, 8200], (BF16, F16, F32, BF16), 3.0)
    out = [torch.empty_like(t, dtype=to) for t in grads]
    fw.beam_moe_clip_grads(grads, 10.0, out=out)
    _clip_check(out, grads, _factor(grads, 10.0))


def test_clip_grads_of_a_flat_buffer():
    """Views of a flat buffer start at any element; what lies around them stays as it is."""
    _say("clip flat")
    for dt in (BF16, F32):
        flat = _randn(_gen(2), (100003,), dt)
        was = flat.clone()
        cuts = [(1, 8), (9, 9), (12, 4001), (4002, 70001), (70005, 100002)]
        views = [flat[a:b] for a, b in cuts]
        copies = [v.clone() for v in views]
        fw.beam_moe_clip_grads(views, 1.0)
        _clip_check(views, copies, _factor(copies, 1.0))
        inside = torch.zeros(100003, dtype=torch.bool, device=DEV)
        for a, b in cuts:
            inside[a:b] = True
        assert torch.equal(flat[~inside], was[~inside])


def test_clip_grads_shapes_and_transposes():
    _say("clip transposes")
    g = _gen(9)
    grads = [_randn(g, (30, 70)), _randn(g, (70, 30)).t(), _randn(g, (2, 3, 5), BF16), _randn(g, (1,))[0],
             _randn(g, (4, 1))]
    copies = [t.clone() for t in grads]
    fw.beam_moe_clip_grads(grads, 1.0)
    _clip_check(grads, copies, _factor(copies, 1.0))
    out = [torch.empty_like(t) for t in copies]
    fw.beam_moe_clip_grads(copies, 1.0, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


def test_clip_grads_by_a_given_norm():
    _say("clip given norm")
    grads = _grads(4, [5000, 70], (F32, BF16))
    norm = torch.full((), 123.5, device=DEV)
    out = [torch.empty_like(t) for t in grads]
    assert fw.beam_moe_clip_grads(grads, 2.0, scale=0.5, norm=norm, out=out) is norm
    _clip_check(out, grads, _factor(grads, 2.0, 0.5, norm=123.5))


@pytest.mark.parametrize("dt,size", [(F32, 1e-30), (F32, 1e30), (BF16, 1e-30), (BF16, 1e30), (F16, 2.0 ** -20),
                                     (F16, 1e4)])
def test_norm_of_tiny_and_huge_gradients(dt, size):
    _say("norm range", dt, size)
    grads = _grads(6, [10000, 777], (dt, dt), size)
    want = _norm_of(grads)
    _near(fw.beam_moe_grad_norm(grads), torch.tensor(want, device=DEV), 1e-12 * want)
    out = [torch.empty_like(t, dtype=F32) for t in grads]
    fw.beam_moe_clip_grads(grads, 1.0, eps=1e-30, out=out)
    f = _factor(grads, 1.0, eps=1e-30)
    if f >= 2.0 ** -120:
        _clip_check(out, grads, f)


def test_clip_grads_infinities_and_nan():
    _say("clip inf nan")
    for dt in (BF16, F16, F32):
        grads = _grads(8, [900, 50], (dt, dt))
        grads[0][77] = INF
        norm = fw.beam_moe_clip_grads(grads, 1.0)
        assert norm.item() == INF and grads[0][77].isnan()
        assert (grads[1] == 0).all() and int(grads[0].isnan().sum()) == 1
        grads = _grads(8, [900, 50], (dt, dt))
        grads[1][3] = NAN
        assert fw.beam_moe_clip_grads(grads, 1.0).isnan()
        assert all(t.isnan().all() for t in grads)


def test_clip_grads_of_nothing():
    _say("clip nothing")
    empty = [torch.empty(0, device=DEV), torch.empty(0, 5, device=DEV, dtype=BF16)]
    assert fw.beam_moe_grad_norm(empty).item() == 0 and fw.beam_moe_clip_grads(empty, 1.0).item() == 0
    zeros = [torch.zeros(100, device=DEV)]
    assert fw.beam_moe_clip_grads(zeros, 0.0).item() == 0 and (zeros[0] == 0).all()


def test_clip_grads_of_one_tensor_past_32_bits():
    _say("clip 2^31 and more")
    n = (1 << 31) + 5
    t = torch.full((n,), 2.0 ** -10, dtype=BF16, device=DEV)
    t[-1] = 1.0
    want = math.sqrt((n - 1) * 2.0 ** -20 + 1.0)
    norm = fw.beam_moe_clip_grads([t], want / 2)
    _near(norm, torch.tensor(want, device=DEV), 1e-12 * want)
    f = want / 2 / (want + 1e-6)
    ends = torch.cat([t[:9], t[-9:]])
    _near(ends, torch.tensor([2.0 ** -10] * 17 + [1.0], device=DEV).double() * f, 4 * U)


def test_clip_grads_captured_and_replayed():
    _say("clip graph")
    for sizes in ([3000, 41], [200] * 130):
        grads = _grads(3, sizes, (BF16, F32) * len(sizes))
        out = [torch.empty_like(t, dtype=F32) for t in grads]
        ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
        fw.beam_moe_clip_grads(grads, 1.0, out=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = fw.beam_moe_clip_grads(grads, 1.0, out=out, ws=ws)
        for k in range(4):
            for t in grads:
                t.mul_(1.0 + 0.5 * k)
            graph.replay()
            torch.cuda.synchronize()
            eager = [torch.empty_like(t) for t in out]
            n = fw.beam_moe_clip_grads(grads, 1.0, out=eager)
            assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(eager, out))


# --------------------------------------------------------------------------
# microscaled 4-bit floating point
# --------------------------------------------------------------------------
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_ref(x):
    """(values, scale bytes, codes) of x [M, K], from the definition in 64 bits."""
    M, K = x.shape
    blocks = -(-K // 32)
    v = torch.zeros(M, blocks * 32, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(M, blocks, 32)
    top = v.abs().amax(2)
    m, e = torch.frexp(torch.nan_to_num(top, nan=1.0, posinf=1.0))   # top = m 2^e, 1/2 <= m < 1
    e = torch.where(top > 0, e - 1 - 2, torch.full_like(e, -127)).clamp(min=-127)
    e = torch.where(top < 2.0 ** -126, torch.full_like(e, -127), e)
    unit = torch.exp2(e.double())[..., None]
    a = v.abs() / unit
    code = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):
        border = (VALUES[i] + VALUES[i + 1]) / 2
        code += ((a > border) | ((a == border) & (i % 2 == 1))).long()
    value = torch.tensor(VALUES, dtype=torch.float64, device=x.device)[code] * unit
    neg = torch.signbit(v)
    value, code = torch.where(neg, -value, value), code + 8 * neg.long()
    bad = ~torch.isfinite(top)
    value[bad], code[bad] = NAN, 0
    scales = torch.where(bad, torch.full_like(e, 255), e + 127)
    return value.view(M, -1)[:, :K], scales.to(torch.uint8), code.view(M, -1)


def _pack(code):
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)


MX_SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (64, 256), (33, 1003), (9, 2048), (130, 5120),
             (2, 8201), (1030, 40)]


@pytest.mark.parametrize("rows,cols", MX_SHAPES)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_quantize_mxfp4(rows, cols, dt):
    _say("quantize", rows, cols, dt)
    g = _gen(rows * 3 + cols)
    for pad in (0, 8, 3):
        x = _randn(g, (rows, cols + pad), F32)
        x *= torch.exp2(torch.randint(-9, 9, x.shape, generator=g, device=DEV).float())
        x = x.to(dt)[:, :cols]
        value, scales, code = _mx_ref(x)
        q = fw.beam_moe_quantize_mxfp4(x)
        assert torch.equal(q.scales, scales)
        assert torch.equal(q.codes, _pack(code))
        for yt in (dt, F32):
            y = fw.beam_moe_dequantize_mxfp4(q, cols, out_dtype=yt)
            assert y.shape == x.shape and torch.equal(y, value.to(yt))


def test_quantize_mxfp4_every_border():
    """All values and borders of the grid, their neighbours in FP32, both signs, at many scales, the ends of FP32's
    range among them."""
    _say("quantize borders")
    grid = torch.tensor([v for a, b in zip(VALUES, VALUES[1:]) for v in (a, (a + b) / 2)] + [6.0, 7.0, 7.75])
    grid = torch.cat([grid, torch.nextafter(grid, torch.tensor(INF)), torch.nextafter(grid, torch.tensor(0.0))])
    grid = grid[grid < 8]
    rows = []
    for e in list(range(-149, -120)) + [-60, -24, -1, 0, 1, 30] + list(range(118, 126)):
        for sign in (1.0, -1.0):
            for i in range(0, len(grid), 15):
                part = grid[i:i + 15].double()
                # the block's largest magnitude fixes its scale: 4 on one half, nearly 8 on the other
                block = torch.cat([torch.tensor([4.0, 7.9]).double(), part, part.flip(0)])
                block = torch.nn.functional.pad(block, (0, 32 - len(block)))
                rows.append(sign * block * 2.0 ** e)
    x = torch.stack(rows).float().to(DEV)
    x = x[x.isfinite().all(1)]
    value, scales, code = _mx_ref(x)
    q = fw.beam_moe_quantize_mxfp4(x)
    assert torch.equal(q.scales, scales)
    assert torch.equal(q.codes, _pack(code))
    assert torch.equal(fw.beam_moe_dequantize_mxfp4(q, out_dtype=F32).double(), value)


def test_every_code_and_scale():
    _say("dequantize all")
    scales = torch.arange(256, device=DEV, dtype=torch.uint8)[:, None]
    codes = torch.arange(16, device=DEV, dtype=torch.uint8)
    codes = torch.cat([codes[0::2] + 16 * codes[1::2]] * 2)[None].expand(256, 16).contiguous()
    size = torch.tensor(VALUES, dtype=torch.float64, device=DEV)
    size = torch.cat([size, -size]).repeat(2)[None]
    want = size * torch.exp2(scales.double() - 127)
    want[255] = NAN
    for dt in (F32, BF16, F16):
        y = fw.beam_moe_dequantize_mxfp4((codes, scales), out_dtype=dt)
        assert torch.equal(y[255].isnan(), torch.ones(32, dtype=torch.bool, device=DEV))
        assert torch.equal(y[:255], want[:255].to(F32).to(dt)), dt


def test_quantize_mxfp4_infinities_and_nan():
    _say("quantize inf nan")
    for dt in (BF16, F16, F32):
        x = _randn(_gen(1), (6, 96), dt)
        x[1, 40], x[2, 0], x[4, 95] = INF, NAN, -INF
        value, scales, code = _mx_ref(x)
        q = fw.beam_moe_quantize_mxfp4(x)
        assert torch.equal(q.scales, scales) and torch.equal(q.codes, _pack(code))
        y = fw.beam_moe_dequantize_mxfp4(q, 96, out_dtype=F32)
        assert torch.equal(y.isnan(), value.isnan()) and int(y.isnan().sum()) == 96
        assert torch.equal(y.nan_to_num(), value.float().nan_to_num())


def test_mxfp4_into_wider_buffers():
    """Strided codes, scales and values; what lies behind the rows stays as it is."""
    _say("mx strides")
    x = _randn(_gen(4), (37, 70), BF16, pad=3)
    want = fw.beam_moe_quantize_mxfp4(x)
    codes = torch.full((37, 64), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((37, 7), 0x5A, dtype=torch.uint8, device=DEV)
    q = fw.beam_moe_quantize_mxfp4(x, out=fw.Mxfp4(codes[:, :48], scales[:, :3]))
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    assert (codes[:, 48:] == 0xA5).all() and (scales[:, 3:] == 0x5A).all()
    y = torch.full((37, 90), 7.0, dtype=BF16, device=DEV)
    fw.beam_moe_dequantize_mxfp4(q, 70, out=y[:, :70])
    assert (y[:, 70:] == 7.0).all()
    assert torch.equal(y[:, :70], fw.beam_moe_dequantize_mxfp4(want, 70))


def test_mxfp4_offsets_past_32_bits():
    _say("mx 2^31 elements and more")
    rows, cols = 8200, 1 << 18
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    x[-1, -40:] = _randn(_gen(5), (40,), BF16)
    x[0, :40] = x[-1, -40:]
    q = fw.beam_moe_quantize_mxfp4(x)
    for r in (0, rows - 1):
        value, scales, code = _mx_ref(x[r:r + 1])
        assert torch.equal(q.codes[r:r + 1], _pack(code)) and torch.equal(q.scales[r:r + 1], scales)
    del x
    y = fw.beam_moe_dequantize_mxfp4(q)
    for r in (0, rows - 1):
        assert torch.equal(y[r], fw.beam_moe_dequantize_mxfp4((q.codes[r:r + 1], q.scales[r:r + 1]))[0])
    assert (y[1] == 0).all()
