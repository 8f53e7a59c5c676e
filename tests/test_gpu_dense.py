"""GPU parity of the operators of a dense gated sublayer (the norm of all gradients and their clipping, microscaled
4-bit floating point and its product, the gated projections) with their formulas in 64 bits.

Tolerances are bounds on the kernels' own roundings: u = 2^-24 is FP32's half step, a sum of depth d is off by at most
d u times the sum of magnitudes, and a result stored in type t by at most half a step, finfo(t).eps / 2 of its value
(plus half the least subnormal of fp16).
"""
import math
from array import array

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


SIZES = [[1], [7, 1, 0, 33], [8192, 8193, 8191], [100000, 3, 65537], [5] * 300, [1000 + 13 * i for i in range(130)],
         [16384], [16385], [32768], [30000, 2769], [40] * 112, [40] * 113, [300000, 2, 2047, 2048, 2049] * 50]
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


def test_clip_grads_of_transposes_beside_a_flat_buffer():
    """Each output by itself: contiguous ones of as many elements for contiguous gradients, the same strides for others."""
    _say("clip transposes and flat")
    g = _gen(11)
    grads = [_randn(g, (30, 70)), _randn(g, (70, 30)).t(), _randn(g, (2, 3, 5), BF16)]
    flat = torch.zeros(3000, device=DEV)
    out = [flat[:2100], torch.empty_like(grads[1]), flat[2200:2230]]
    fw.beam_moe_clip_grads(grads, 1.0, out=out)
    _clip_check([o.reshape(t.shape) for o, t in zip(out, grads)], grads, _factor(grads, 1.0))
    for bad in ([out[0], flat[:2100], out[2]], [out[0], torch.empty(30, 70, device=DEV), out[2]],
                [torch.empty(70, 30, device=DEV).t(), out[1], out[2]], [flat[:2099], out[1], out[2]]):
        with pytest.raises(ValueError):
            fw.beam_moe_clip_grads(grads, 1.0, out=bad)


def test_clip_grads_partly_in_place():
    _say("clip partly in place")
    for n in (300, 9000):
        grads = _grads(n, [n, 70, n], (F32, BF16, BF16))
        copies = [t.clone() for t in grads]
        out = [grads[0], torch.empty(70, device=DEV), grads[2]]
        fw.beam_moe_clip_grads(grads, 1.0, out=out)
        _clip_check(out, copies, _factor(copies, 1.0))
        assert torch.equal(grads[1], copies[1])


def test_clip_grads_by_a_given_norm():
    _say("clip given norm")
    grads = _grads(4, [5000, 70], (F32, BF16))
    norm = torch.full((3,), 123.5, device=DEV)[1]
    out = [torch.empty_like(t) for t in grads]
    assert fw.beam_moe_clip_grads(grads, 2.0, scale=0.5, norm=norm, out=out) is norm
    _clip_check(out, grads, _factor(grads, 2.0, 0.5, norm=123.5))


def test_the_norm_is_one_whatever_the_call():
    """Squares whose FP64 sum lies within its own rounding of a border of FP32: 24 of just below 2^-53 count beside the
    largest or do not, by the order of the sum. Clipping in place, apart and the norm alone agree in every bit."""
    _say("norm order")
    c, (b, d) = 2.0 ** -26.5 * 0.99, (3.4526692e-04, 2.1562738e-07)
    for n in (2048, 16385, 20000, 32768, 40000, 65536, 65537, 140000):
        g = torch.zeros(n, device=DEV)
        g[0], g[8], g[16] = 1.0, b, d
        for i in (512, 1024, 1536):
            g[i:i + 8] = c
        norm = fw.beam_moe_grad_norm([g])
        assert abs(norm.item() - 1.0) <= 2.0 ** -23
        for grads in ([g.clone()], [g.clone(), torch.zeros(0, device=DEV)]):
            assert torch.equal(fw.beam_moe_clip_grads(grads, 1.0, out=[torch.empty_like(t) for t in grads]), norm), n
            assert torch.equal(fw.beam_moe_clip_grads(grads, 1.0), norm), n


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


@pytest.mark.parametrize("size", [None, 0, 9])
def test_a_given_norm_is_written_whatever_the_list(size):
    """The C entry point hands a given norm on, also where the list holds no element."""
    _say("clip norm handed on", size)
    lib = fw.load_library()
    grads = [] if size is None else [torch.ones(size, device=DEV)]
    at, types, sizes = (array(c, v) for c, v in (("Q", [t.data_ptr() for t in grads]), ("i", [fw.BEAM_MOE_F32] * len(grads)),
                                                 ("q", [t.numel() for t in grads])))
    given, norm = torch.full((1,), 8.0, device=DEV), torch.full((4,), NAN, device=DEV)
    ws = torch.empty(lib.beam_moe_grad_norm_workspace_bytes(len(grads)), dtype=torch.uint8, device=DEV)
    status = lib.beam_moe_clip_grads(len(grads), at.buffer_info()[0], types.buffer_info()[0], sizes.buffer_info()[0], 1.0,
                                     4.0, 2.0 ** -40, given.data_ptr(), None, None, norm.data_ptr(), ws.data_ptr(),
                                     ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert status == 0 and norm[0].item() == 8.0 and norm[1:].isnan().all()
    assert all((t == 0.5).all() for t in grads)


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


def test_codes_past_the_range_of_fp32():
    """Values in 64 bits: exact up to scale 252, infinite above where they are 2^128 and more, exact elsewhere; the
    quantisation writes no scale above 252 but 255."""
    _say("dequantize ends")
    scales = torch.arange(250, 255, device=DEV, dtype=torch.uint8)[:, None]
    codes = torch.arange(16, device=DEV, dtype=torch.uint8)
    codes = torch.cat([codes[0::2] + 16 * codes[1::2]] * 2)[None].expand(5, 16).contiguous()
    size = torch.tensor(VALUES, dtype=torch.float64, device=DEV)
    want = torch.cat([size, -size]).repeat(2)[None] * torch.exp2(scales.double() - 127)
    past = want.abs() >= 2.0 ** 128
    assert past.sum(1).tolist() == [0, 0, 0, 8, 16]
    y = fw.beam_moe_dequantize_mxfp4((codes, scales), out_dtype=F32).double()
    assert torch.equal(y[~past], want[~past]) and torch.equal(y[past], want[past].sign() * INF)
    x = torch.tensor([[3.4028234e38, -1.0, 6e-39] + [0.0] * 29], device=DEV)
    assert fw.beam_moe_quantize_mxfp4(x).scales.item() == 252


def test_clip_grads_of_a_norm_past_fp32():
    """Finite gradients of a norm of some 1.4e40: infinite as FP32, and clipped by its value."""
    _say("clip past fp32")
    for n in (20000, 200000):
        g = torch.full((n,), 1e38, device=DEV)
        out = [torch.empty_like(g)]
        assert fw.beam_moe_grad_norm([g]).item() == INF
        assert fw.beam_moe_clip_grads([g], 1e38, out=out).item() == INF
        _clip_check(out, [g], 1 / math.sqrt(n))  # the limit is rounded to FP32 as the elements are
        fw.beam_moe_clip_grads([g], 1e38, norm=torch.full((), INF, device=DEV), out=out)
        assert not out[0].any()


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


# --------------------------------------------------------------------------
# the gated projections
# --------------------------------------------------------------------------
ACTS = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}
GEMM_UP = 2.0 ** -23  # a step inside the matrix core may cut instead of round


def _depth(K):
    """Additions that a product meets: its own group of 32, then one per group (whatever the split)."""
    return 32 + K / 32 + 40


def _slope(z, act):
    z = z.double().requires_grad_(True)
    return torch.autograd.grad(ACTS[act](z).sum(), z)[0]


def _gated_inputs(M, N, K, dt, pad=0, bias=True, seed=0):
    g = _gen(M * 3 + N * 5 + K + seed)
    x, wg, wu = _randn(g, (M, K), dt, 1.0, pad), _randn(g, (N, K), dt, K ** -0.5, pad), _randn(g, (N, K), dt, K ** -0.5)
    return g, x, wg, wu, _randn(g, (N,)) if bias else None, _randn(g, (N,)) if bias else None


def _gated_check(x, wg, wu, bg, bu, act, h, zg=None, zu=None):
    """Sums of depth d; act is good to 8 u of |z| + 1 and its slope stays below 1.13; the product adds a step."""
    def arg(w, b):
        z, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
        if b is not None:
            z, mag = z + b.double(), mag + b.double().abs()
        return z, _depth(x.shape[1]) * GEMM_UP * mag
    (rg, eg), (ru, eu) = arg(wg, bg), arg(wu, bu)
    if zg is not None:
        _near(zg, rg, eg, "pre_gate")
        _near(zu, ru, eu, "pre_up")
    a = ACTS[act](rg)
    ea = 1.13 * eg + 8 * U * (rg.abs() + (act != "none"))
    _near(h, a * ru, ea * (ru.abs() + eu) + a.abs() * eu + 2 * U * (a * ru).abs(), "h")


# the last are large enough for 256-row tiles
# in one of the gradients' products; the forward product's are in test_gated_linear_large and GATED_TILES_256
GATED_SHAPES = [(1, 1, 1), (1, 64, 64), (1, 100, 1000), (2, 2560, 512), (3, 17, 5), (7, 33, 2049), (16, 256, 128),
                (17, 48, 96), (33, 1000, 136), (64, 512, 2560), (65, 130, 72), (100, 64, 7), (129, 257, 65),
                (255, 96, 520), (256, 256, 64), (300, 513, 1024), (257, 264, 192), (520, 1040, 328), (1000, 1032, 2048),
                (2100, 1280, 1280)]


@pytest.mark.parametrize("M,N,K", GATED_SHAPES)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear(M, N, K, dt):
    for act, yt, bias, pad in (("silu", dt, False, 0), ("gelu", F32, True, 0), ("relu", dt, True, 8),
                               ("silu", dt, True, 3), ("none", F32, False, 1)):
        _say("gated", M, N, K, dt, act, yt, bias, pad)
        _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, dt, pad, bias)
        h, zg, zu = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, act=act, out_dtype=yt, want_pre=True)
        _gated_check(x, wg, wu, bg, bu, act, h, zg, zu)
        assert torch.equal(fw.beam_moe_gated_linear(x, wg, wu, bg, bu, act=act, out_dtype=yt), h)


# 256-row tiles with K of whole stages: whole tiles, rows and columns that end inside a tile or a chunk of eight, one tile
# to a workgroup and several
@pytest.mark.parametrize("M,N,K", [(4096, 2048, 640), (4000, 2043, 192), (3900, 2040, 320), (8100, 2036, 192),
                                   (16384, 1024, 256)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_large(M, N, K, dt):
    for act, yt, bias, pre, pad in (("silu", dt, False, False, 0), ("gelu", F32, True, True, 8),
                                    ("relu", dt, True, False, 3), ("silu", dt, False, True, 0),
                                    ("none", F32, False, False, 0)):
        _say("gated large", M, N, K, dt, act, yt, bias, pre, pad)
        _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, dt, pad, bias)
        buf = torch.full((M, N + 8), 7.0, dtype=yt, device=DEV)
        out = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, act=act, out=buf[:, :N], want_pre=pre)
        h, zg, zu = out if pre else (out, None, None)
        _gated_check(x, wg, wu, bg, bu, act, h, zg, zu)
        assert (buf[:, N:] == 7.0).all()


# 256-row tiles with K that ends inside a stage: whole and ragged chunks, the last laid out anew; rows and columns that end
# inside a tile, and whole ones
GATED_TILES_256 = [(4096, 2048, 328), (4000, 2043, 331), (4096, 2048, 1000), (3900, 2040, 200), (8100, 1021, 777)]


@pytest.mark.parametrize("M,N,K", GATED_TILES_256)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_large_with_a_ragged_k(M, N, K, dt):
    for act, yt, bias, pre, pad in (("silu", dt, False, False, 0), ("gelu", F32, True, True, 8),
                                    ("relu", dt, True, True, 3), ("none", F32, False, False, 0)):
        _say("gated large ragged", M, N, K, dt, act, yt, bias, pre, pad)
        _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, dt, pad, bias)
        buf = torch.full((M, N + 8), 7.0, dtype=yt, device=DEV)
        out = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, act=act, out=buf[:, :N], want_pre=pre)
        h, zg, zu = out if pre else (out, None, None)
        _gated_check(x, wg, wu, bg, bu, act, h, zg, zu)
        assert (buf[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(5, 70, 65), (100, 130, 72), (200, 131, 71), (300, 150, 16384), (4096, 2048, 328),
                                   (4000, 2043, 192), (4096, 2048, 192)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_pre_into_wider_buffers(M, N, K, dt):
    """The C entry point's strided pre, each with a stride of its own: the binding's bits, and nothing behind the rows."""
    _say("gated strided pre", M, N, K, dt)
    lib = fw.load_library()
    _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, dt)
    h, zg, zu = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, want_pre=True)
    ws = torch.empty(lib.beam_moe_gated_linear_workspace_bytes(M, N, K, K, K, K) + 16, dtype=torch.uint8, device=DEV)
    for both in ((True, True), (True, False), (False, True)):
        bufs = [torch.full((M, N + p), 7.0, dtype=dt, device=DEV) for p in (3, 5, 8)]
        pre = [(b.data_ptr() if w else None, b.shape[1]) for b, w in zip(bufs[1:], both)]
        status = lib.beam_moe_gated_linear(M, N, K, fw.ELEM_TYPES[dt], x.data_ptr(), K, wg.data_ptr(), K, wu.data_ptr(), K,
                                           bg.data_ptr(), bu.data_ptr(), fw.ACTIVATIONS["silu"], bufs[0].data_ptr(),
                                           fw.ELEM_TYPES[dt], N + 3, *pre[0], *pre[1], ws.data_ptr(), ws.numel(),
                                           torch.cuda.current_stream().cuda_stream)
        assert status == 0
        for b, want, wrote in zip(bufs, (h, zg, zu), (True, *both)):
            assert (b[:, N:] == 7.0).all() and (torch.equal(b[:, :N], want) if wrote else (b == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(100, 50, 65536), (300, 150, 16384), (512, 256, 9216), (20, 100, 2050)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_long_k(M, N, K, dt):
    _say("gated long K", M, N, K, dt)
    _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, dt)
    h, zg, zu = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, want_pre=True)
    _gated_check(x, wg, wu, bg, bu, "silu", h, zg, zu)


def test_gated_linear_of_one_fused_weight():
    """Both weights as halves of one matrix, or as its alternate rows."""
    _say("gated fused weight")
    for M in (5, 200):
        g = _gen(M)
        x, w = _randn(g, (M, 136), BF16), _randn(g, (300, 136), BF16, 0.1)
        for wg, wu in ((w[:150], w[150:]), (w[0::2], w[1::2])):
            h = fw.beam_moe_gated_linear(x, wg, wu)
            assert torch.equal(h, fw.beam_moe_gated_linear(x, wg.contiguous(), wu.contiguous()))
            _gated_check(x, wg, wu, None, None, "silu", h)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 70, 65), (70, 70, 65), (300, 264, 128)])
def test_gated_linear_padding_and_nan(M, N, K):
    """What lies behind the rows of h stays; a NaN row of x stays in its row."""
    _say("gated padding", M, N, K)
    _, x, wg, wu, bg, bu = _gated_inputs(M, N, K, BF16, 8)
    buf = torch.full((M, N + 9), 7.0, dtype=BF16, device=DEV)
    want = fw.beam_moe_gated_linear(x, wg, wu, bg, bu)
    fw.beam_moe_gated_linear(x, wg, wu, bg, bu, out=buf[:, :N])
    assert torch.equal(buf[:, :N], want) and (buf[:, N:] == 7.0).all()
    x = x.clone()
    x[M // 2, K // 2] = NAN
    got = fw.beam_moe_gated_linear(x, wg, wu, bg, bu)
    assert got[M // 2].isnan().all()
    keep = torch.arange(M, device=DEV) != M // 2
    assert torch.equal(got[keep], want[keep])


def test_gated_linear_of_no_rows():
    _say("gated no rows")
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(40, 64, dtype=BF16, device=DEV)
    assert fw.beam_moe_gated_linear(x, w, w).shape == (0, 40)
    z = torch.empty(0, 40, dtype=BF16, device=DEV)
    dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(z, x, w, w, z, z)
    assert dx.shape == (0, 64) and all(t.shape[0] == 40 and not t.any() for t in (dwg, dwu, dbg, dbu))


def _gated_back_check(dh, x, wg, wu, zg, zu, act, out):
    """dz is rounded to the products' type: half a step of each term, at worst all one way, or in fp16, where the
    largest lies in [2^14, 2^15) of its scale, 2^-25 of it, at most 2^-39 of the largest; then the sums. Slopes near zero
    are differences of order 1."""
    d, g, u = dh.double(), zg.double(), zu.double()
    M, N = dh.shape
    dg, du = d * u * _slope(zg, act), d * ACTS[act](g)
    off = _step(x) + 24 * U
    top = 2.0 ** -39 * float(torch.maximum(dg.abs().max(), du.abs().max())) if x.dtype == F16 else 0.0
    near = 8 * U * (act != "none") * d.abs()
    eg, eu = off * dg.abs() + near * u.abs() + top, off * du.abs() + near * (g.abs() + 1) + top
    dx, dwg, dwu, dbg, dbu = out
    if dx is not None:
        w, v = wg.double(), wu.double()
        dep = _depth(2 * N) * GEMM_UP
        _near(dx, dg @ w + du @ v, (dep * dg.abs() + eg) @ w.abs() + (dep * du.abs() + eu) @ v.abs(), "dx")
    if dwg is not None:
        dep = _depth(M) * GEMM_UP
        ax = x.double().abs()
        _near(dwg, dg.t() @ x.double(), (dep * dg.abs() + eg).t() @ ax, "dw_gate")
        _near(dwu, du.t() @ x.double(), (dep * du.abs() + eu).t() @ ax, "dw_up")
    if dbg is not None:
        dep = (math.ceil(M / 64) + 64 + 24 + 24) * U
        _near(dbg, dg.sum(0), (dep * dg.abs() + near * u.abs()).sum(0), "dbias_gate")
        _near(dbu, du.sum(0), (dep * du.abs() + near * (g.abs() + 1)).sum(0), "dbias_up")


LARGE_BACK = [(1000, 520, 2048), (3300, 1700, 136), (3300, 100, 3336), (200, 1650, 3336), (4096, 1024, 1280),
              (5150, 1029, 5169)]


@pytest.mark.parametrize("M,N,K", GATED_SHAPES + LARGE_BACK)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_backward(M, N, K, dt):
    for act, yt, pad in (("silu", dt, 0), ("gelu", F32, 8), ("relu", dt, 3), ("none", F32, 1)):
        _say("gated_backward", M, N, K, dt, act, yt, pad)
        g, x, wg, wu, _, _ = _gated_inputs(M, N, K, dt, pad)
        dh, zg, zu = _randn(g, (M, N), yt, 1.0, pad), _randn(g, (M, N), dt, 1.0, pad), _randn(g, (M, N), dt)
        out = fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu, act=act)
        _gated_back_check(dh, x, wg, wu, zg, zu, act, out)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_backward_parts(dt):
    """Each result by itself has the bits that it has among all."""
    for M, N, K in ((70, 130, 72), (517, 203, 777), (3300, 1700, 136)):
        _say("gated_backward parts", M, N, K, dt)
        g, x, wg, wu, _, _ = _gated_inputs(M, N, K, dt)
        dh, zg, zu = (_randn(g, (M, N), dt) for _ in range(3))
        dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu)
        _gated_back_check(dh, x, wg, wu, zg, zu, "silu", (dx, dwg, dwu, dbg, dbu))
        only = fw.beam_moe_gated_linear_backward(dh, x, None, None, zg, zu, want_dx=False)
        assert only[0] is None
        _gated_back_check(dh, x, None, None, zg, zu, "silu", only)
        only = fw.beam_moe_gated_linear_backward(dh, None, wg, wu, zg, zu, want_dw=False, want_dbias=False)
        assert only[1:] == (None,) * 4
        _gated_back_check(dh, torch.empty(M, K, dtype=dt), wg, wu, zg, zu, "silu", only)
        only = fw.beam_moe_gated_linear_backward(dh, x, None, None, zg, zu, want_dx=False, want_dw=False)
        assert torch.equal(only[3], dbg) and torch.equal(only[4], dbu)


@pytest.mark.parametrize("M,N,K", [(1, 9, 16), (33, 100, 136), (517, 203, 777), (3300, 1700, 136)])
@pytest.mark.parametrize("size,weights", [(1e-7, 2.0 ** 11), (1e-12, 2.0 ** 11), (1e6, 2.0 ** -14)])
def test_gated_backward_keeps_small_and_large_gradients_in_fp16(M, N, K, size, weights):
    """FP32 gradients that fp16 cannot hold, with weights and inputs for which the results can be held."""
    _say("gated_backward range", M, N, K, size)
    g = _gen(M + N + K)
    x, wg, wu = (_randn(g, s, F16, weights) for s in ((M, K), (N, K), (N, K)))
    dh, zg, zu = _randn(g, (M, N), F32, size, 3), _randn(g, (M, N), F16, 1.5), _randn(g, (M, N), F16, 1.5)
    for act in ("silu", "gelu"):
        out = fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu, act=act)
        _gated_back_check(dh, x, wg, wu, zg, zu, act, out)


def test_gated_backward_nan_and_infinite_gradients_in_fp16():
    """They touch their own row of dx and their own row of dw alone, and have no part in the scale."""
    _say("gated_backward nan")
    M, N, K = 90, 70, 136
    g, x, wg, wu, _, _ = _gated_inputs(M, N, K, F16)
    dh, zg, zu = (_randn(g, (M, N), F16) for _ in range(3))
    clean = fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu)
    # what the poisoned elements would have been the scale of stays
    assert dh[3, 5].abs() < dh.abs().max() and dh[40, 6].abs() < dh.abs().max()
    dh = dh.clone()
    dh[3, 5], dh[40, 6] = NAN, INF
    dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu)
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    rows[[3, 40]] = False
    cols = torch.ones(N, dtype=torch.bool, device=DEV)
    cols[[5, 6]] = False
    assert torch.equal(dx[rows], clean[0][rows]) and not dx[~rows].isfinite().any()
    for got, was in ((dwg, clean[1]), (dwu, clean[2]), (dbg, clean[3]), (dbu, clean[4])):
        assert torch.equal(got[cols], was[cols]) and not got[~cols].isfinite().any()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("wide", [False, True], ids=["own", "f32"])
def test_gated_gradients_at_infinite_pre(act, dt, wide):
    """Every pair of a finite, infinite and NaN argument of either projection. An activation and its slope are their
    limits at infinity, and 0 times an infinite argument or activation is 0, as times the finite one it stands for."""
    _say("gated infinite pre", act, dt, wide)
    vals = torch.tensor([-INF, INF, -200.0, 1.0, 0.0, NAN], dtype=torch.float64, device=DEV)
    g, u = (t.reshape(-1) for t in torch.meshgrid(vals, vals, indexing="ij"))
    N, K = g.numel(), 16
    # at +-200 the forms are within e^-200 of their limits, 2^-280 with the factor 200: rounded to FP32, whose least is
    # 2^-149, they are the limits. NaN stays
    big = g.clamp(-200.0, 200.0)
    a = torch.where(g == INF, g, ACTS[act](big).float().double()) if act != "none" else g
    slope = torch.where(g.isnan(), torch.zeros_like(g), (g > 0).double()) if act == "relu" else _slope(big, act)
    slope = slope.float().double()
    times = lambda p, q: torch.where((p == 0) & q.isinf(), torch.zeros_like(q), p * q)  # noqa: E731
    x, w = torch.ones(1, K, dtype=dt, device=DEV), torch.ones(N, K, dtype=dt, device=DEV)
    for d in (1.0, -2.0, 0.0):
        dh = torch.full((1, N), d, dtype=F32 if wide else dt, device=DEV)
        zg, zu = g[None].to(dt), u[None].to(dt)
        wg, wu = times(d * slope, u), times(torch.full_like(a, d), a)
        dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(dh, x, w, w, zg, zu, act=act)
        for got, want, steps in ((dbg, wg, 0), (dbu, wu, 0), (dwg[:, 3], wg, 2), (dwu[:, 3], wu, 2)):
            assert torch.equal(got.isnan(), want.isnan()), (d, got, want)
            assert torch.equal(got == INF, want == INF) and torch.equal(got == -INF, want == -INF), (d, got, want)
            got, want = got[want.isfinite()], want[want.isfinite()]
            _near(got, want, steps * _step(dx) * want.abs() + 32 * U * abs(d) * (1 + want.abs()))
        # a row of dx holds what its columns do
        fine = wg.isfinite() & wu.isfinite()
        dx, _, _, _, _ = fw.beam_moe_gated_linear_backward(dh[:, fine], x, w[fine], w[fine], zg[:, fine], zu[:, fine],
                                                           act=act)
        terms = wg[fine].abs().sum() + wu[fine].abs().sum()
        _near(dx, (wg[fine].sum() + wu[fine].sum()).expand(1, K), 2 * _step(dx) * terms + 64 * U * (abs(d) * 400 + terms))


def test_gated_step_past_the_range_of_fp16():
    """Arguments past 65504 are stored as infinities while h, in FP32, is finite: a gate far below zero lets no gradient
    through, whatever stands beside it."""
    _say("gated past fp16")
    x, w = torch.zeros(3, 16, dtype=F16, device=DEV), torch.ones(8, 16, dtype=F16, device=DEV)
    bg = torch.tensor([-7e4, -7e4, -7e4, -3e38, 2.0, 2.0, -7e4, 7e4], device=DEV)
    bu = torch.tensor([1.0, 7e4, -7e4, 7e4, 0.5, -1.0, 0.0, 0.0], device=DEV)
    for act in ("relu", "silu", "gelu"):
        h, zg, zu = fw.beam_moe_gated_linear(x, w, w, bg, bu, act=act, out_dtype=F32, want_pre=True)
        assert h.isfinite().all() and (h[:, :4] == 0).all() and zg[:, :4].isinf().all() and zu[:, 1:4].isinf().all()
        for dh in (torch.ones(3, 8, device=DEV), torch.ones(3, 8, dtype=F16, device=DEV)):
            dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(dh, x + 1, w, w, zg, zu, act=act)
            for t in (dwg, dwu, dbg, dbu):
                assert (t[:4] == 0).all() and t[4:7].isfinite().all()
            for n in (4, 7):
                dx, _, _, _, _ = fw.beam_moe_gated_linear_backward(dh[:, :n], x + 1, w[:n], w[:n], zg[:, :n], zu[:, :n],
                                                                   act=act)
                assert dx.isfinite().all() and (n > 4 or (dx == 0).all())


def test_gated_gradients_whose_products_pass_fp32():
    """dh times the up argument may leave FP32's range where the gate's slope takes it back."""
    _say("gated products past fp32")
    d = torch.tensor([[1e38, -1e38, 3e38, 1e38]], device=DEV)
    zg = torch.tensor([[-30.0, -40.0, -1000.0, -INF]], dtype=BF16, device=DEV)
    zu = torch.tensor([[1e3, 1e4, -1e6, 1e3]], dtype=BF16, device=DEV)
    w, x = torch.full((4, 16), 1e-30, dtype=BF16, device=DEV), torch.ones(1, 16, dtype=BF16, device=DEV)
    for act in ("relu", "silu"):
        want = d.double() * zu.double() * _slope(zg.double().clamp_min(-1000.0), act)
        out = fw.beam_moe_gated_linear_backward(d, x, w, w, zg, zu, act=act)
        assert all(t.isfinite().all() for t in out)
        # the exponent of e^-z is rounded at |z| half steps of FP32
        _near(out[3][None], want, 64 * U * want.abs())


def test_gated_gradient_against_differences():
    """Differences of the call itself in FP32 outputs: with loss L = sum(h r), (L(x + t v) - L(x - t v)) / 2t against
    dx . v and the like. x holds multiples of 2^-6 and t v too, so both arguments are exact in bf16. h is off by
    40 u of its magnitudes, the third derivative of silu(a) b along the line by at most 3 of |v w|^3 / 6 t^2."""
    _say("gated differences")
    M, N, K, t = 6, 40, 32, 2.0 ** -4
    g = _gen(77)
    grid = lambda s, top: torch.randint(-top, top + 1, s, generator=g, device=DEV).to(BF16) / 64  # noqa: E731
    x, wg, wu = grid((M, K), 64), grid((N, K), 32), grid((N, K), 32)
    r = _randn(g, (M, N))
    h, zg, zu = fw.beam_moe_gated_linear(x, wg, wu, out_dtype=F32, want_pre=True)
    dx, dwg, dwu, _, _ = fw.beam_moe_gated_linear_backward(r, x, wg, wu, zg, zu)

    def loss(x, wg, wu):
        return float((fw.beam_moe_gated_linear(x, wg, wu, out_dtype=F32).double() * r.double()).sum())

    size = float((h.double().abs() * r.double().abs()).sum())
    for k, (arg, grad) in enumerate(((x, dx), (wg, dwg), (wu, dwu))):
        v = torch.randint(-1, 2, arg.shape, generator=g, device=DEV).to(BF16)
        ends = [[a if i != k else (a.float() + s * t * v.float()).to(BF16) for i, a in enumerate((x, wg, wu))]
                for s in (1, -1)]
        assert all(torch.equal(e[k].float(), arg.float() + s * t * v.float()) for e, s in zip(ends, (1, -1)))
        quot = (loss(*ends[0]) - loss(*ends[1])) / (2 * t)
        slope = float((grad.double() * v.double()).sum())
        xd, vd = x.double().abs(), v.double().abs()
        # |d zg|, |d zu| along v
        if k == 0:
            ag, au = vd @ wg.double().abs().t(), vd @ wu.double().abs().t()
        elif k == 1:
            ag, au = xd @ vd.t(), torch.zeros(M, N, device=DEV, dtype=torch.float64)
        else:
            ag, au = torch.zeros(M, N, device=DEV, dtype=torch.float64), xd @ vd.t()
        # |silu''| <= 1/2, |silu'''| <= 0.31
        third = ((0.31 * ag ** 3 * zu.double().abs() + 3 * 0.5 * ag ** 2 * au) * r.double().abs()).sum()
        # pre, both dz and the gradient itself are rounded to bf16: at most eight half steps of what they are made of
        made = ((1.1 * ag * zu.double().abs() + au * zg.double().abs()) * r.double().abs()).sum()
        tol = 8 * 2.0 ** -8 * float(made) + float(third) * t * t / 6 + 40 * U * size / t * 4
        assert abs(quot - slope) <= tol, (k, quot, slope, tol)
        assert tol < 0.2 * max(abs(slope), float(made) / 3), (k, tol, slope)


def _gated_step_inputs(seed, T=192, H=512, F=328):
    g = _gen(seed)
    return dict(stream=_randn(g, (T, H), F32, 2.0), gamma=1 + _randn(g, (H,), F32, 0.1), beta=_randn(g, (H,), F32, 0.1),
                wg=_randn(g, (F, H), BF16, H ** -0.5), wu=_randn(g, (F, H), BF16, H ** -0.5),
                bg=_randn(g, (F,), F32, 0.1), bu=_randn(g, (F,), F32, 0.1), wd=_randn(g, (H, F), BF16, F ** -0.5),
                dout=_randn(g, (T, H), F32))


def _gated_step(s, max_norm=1.0, step=3):
    """A dense gated sublayer (norm, gated projections, down onto the stream) forward and back to the stream and every
    weight, and all weights' gradients clipped into 32 bits."""
    keep, add = math.sqrt((step - 1) / step), math.sqrt(1 / step)
    x, mean, rstd = fw.beam_moe_layer_norm(s["stream"], s["gamma"], s["beta"], out_dtype=BF16)
    h, zg, zu = fw.beam_moe_gated_linear(x, s["wg"], s["wu"], s["bg"], s["bu"], want_pre=True)
    out = fw.beam_moe_linear(h, s["wd"], residual=s["stream"], keep=keep, add=add, out_dtype=F32)
    dh, dwd, _, dstream = fw.beam_moe_linear_backward(s["dout"], h, s["wd"], keep=keep, add=add, want_dbias=False,
                                                      want_dres=True)
    dx, dwg, dwu, dbg, dbu = fw.beam_moe_gated_linear_backward(dh, x, s["wg"], s["wu"], zg, zu)
    dnorm, dgamma, dbeta = fw.beam_moe_layer_norm_backward(dx, s["stream"], mean, rstd, s["gamma"])
    grads = dict(gamma=dgamma, beta=dbeta, wg=dwg, wu=dwu, bg=dbg, bu=dbu, wd=dwd)
    clipped = {k: torch.empty_like(v, dtype=F32) for k, v in grads.items()}
    norm = fw.beam_moe_clip_grads(list(grads.values()), max_norm, out=list(clipped.values()))
    return dict(out=out, dstream=dstream + dnorm, norm=norm, **clipped)


def _gated_step_ref(s, max_norm=1.0, step=3):
    f = {k: v.double().requires_grad_(True) for k, v in s.items() if k != "dout"}
    x = torch.nn.functional.layer_norm(f["stream"], (f["stream"].shape[1],), f["gamma"], f["beta"], 1e-5)
    h = torch.nn.functional.silu(x @ f["wg"].t() + f["bg"]) * (x @ f["wu"].t() + f["bu"])
    out = math.sqrt((step - 1) / step) * f["stream"] + math.sqrt(1 / step) * (h @ f["wd"].t())
    grads = dict(zip(f, torch.autograd.grad((out * s["dout"].double()).sum(), list(f.values()))))
    dstream = grads.pop("stream")
    norm = torch.stack([(v * v).sum() for v in grads.values()]).sum().sqrt()
    c = min(1.0, max_norm / (float(norm) + 1e-6))
    return dict(out=out.detach(), dstream=dstream, norm=norm, **{k: v * c for k, v in grads.items()})


def test_training_step_of_a_gated_sublayer():
    """The whole run against 64-bit autograd. Rounding a tensor to bf16 changes it by at most eps / 2 of its 2-norm; at
    most eight such roundings (x, h, both pre, dh, both dz, dx) lie on any path to a result, and random matrices
    of these shapes pass a relative error on with a factor of order one: 16 half steps in all, and as much again
    for the norm that every clipped gradient is divided by."""
    _say("gated training step")
    s = _gated_step_inputs(1)
    got, want = _gated_step(s), _gated_step_ref(s)
    torch.cuda.synchronize()
    assert float(want["norm"]) > 2.0
    for k, v in want.items():
        err = float((got[k].double() - v).norm() / v.norm())
        assert err <= (16 if k in ("out", "dstream", "norm") else 32) * 2.0 ** -9, (k, err)


def test_gated_sublayer_on_two_streams_at_once():
    _say("gated two streams")
    a, b = _gated_step_inputs(2), _gated_step_inputs(3)
    alone = [_gated_step(v) for v in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for v, st in zip((a, b), streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(_gated_step(v))
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            assert all(torch.equal(x[k], y[k]) for k in x)


def test_gated_sublayer_captured_and_replayed():
    _say("gated graph")
    for T in (8, 192):
        s = _gated_step_inputs(4, T)
        _gated_step(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = _gated_step(s)
        for k in range(4):
            s["stream"].copy_(_gated_step_inputs(10 + k, T)["stream"])
            s["wg"].mul_(1.0 + 0.25 * (k % 2))
            graph.replay()
            torch.cuda.synchronize()
            eager = _gated_step(s)
            torch.cuda.synchronize()
            assert all(torch.equal(got[n], eager[n]) for n in got)


def test_gated_linear_offsets_past_32_bits():
    _say("gated offsets")
    M, N, K = 40000, 100, 64
    ld = 60000
    buf = torch.zeros(M, ld, dtype=BF16, device=DEV)       # 2.4e9 elements
    x, h = buf[:, :K], buf[:, K + 8:K + 8 + N]
    g = _gen(6)
    wg, wu = _randn(g, (N, K), BF16, 0.1), _randn(g, (N, K), BF16, 0.1)
    x[-300:] = _randn(g, (300, K), BF16)
    fw.beam_moe_gated_linear(x, wg, wu, out=h)
    _gated_check(x[-300:], wg, wu, None, None, "silu", h[-300:])
    assert not h[:100].any()


# a row stride in 256-row tiles just inside the persistent kernel's bound, and past it
@pytest.mark.parametrize("ld", [(1 << 22) - 8, 1 << 22])
@pytest.mark.parametrize("M,N,K", [(520, 16384, 192), (13056, 640, 192)])
def test_gated_linear_of_far_rows(M, N, K, ld):
    """Rows of x, or of both weights, that span more than 2^31 elements."""
    _say("gated far rows", M, N, K, ld)
    g, x, wg, wu, bg, bu = _gated_inputs(M, N, K, BF16)
    far = torch.zeros(min(M, N), ld, dtype=BF16, device=DEV)
    assert far.numel() > 1 << 31
    if M < N:
        far[:, :K] = x
        x = far[:, :K]
    else:
        far[:, :K], far[:, 1 << 21:(1 << 21) + K] = wg, wu
        wg, wu = far[:, :K], far[:, 1 << 21:(1 << 21) + K]
    h, zg, zu = fw.beam_moe_gated_linear(x, wg, wu, bg, bu, want_pre=True)
    _gated_check(x, wg, wu, bg, bu, "silu", h, zg, zu)


@pytest.mark.parametrize("M,N,K", [(600, 72, 136), (600, 71, 131)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gated_linear_backward_of_far_rows(M, N, K, dt):
    _say("gated backward far rows", M, N, K, dt)
    g, x, wg, wu, _, _ = _gated_inputs(M, N, K, dt)
    rows, cols = (torch.zeros(*s, dtype=dt, device=DEV) for s in ((M, 1 << 22), (N, 1 << 25)))
    assert min(rows.numel(), cols.numel()) > 1 << 31
    parts = []
    for k, (buf, t) in enumerate(((rows, _randn(g, (M, N), dt)), (rows, _randn(g, (M, N), dt)), (rows, _randn(g, (M, N), dt)),
                                  (rows, x), (cols, wg), (cols, wu))):
        view = buf[:, 4096 * k:4096 * k + t.shape[1]]
        view.copy_(t)
        parts.append(view)
    dh, zg, zu, x, wg, wu = parts
    _gated_back_check(dh, x, wg, wu, zg, zu, "silu", fw.beam_moe_gated_linear_backward(dh, x, wg, wu, zg, zu))


# --------------------------------------------------------------------------
# the product of 4-bit operands
# --------------------------------------------------------------------------
def _mx_weights(g, N, K, pad=0, spread=2):
    """Random codes and scales of a deviation of about K^-1/2, zero codes past K; rows in wider buffers with pad."""
    blocks = -(-K // 32)
    code = torch.randint(0, 16, (N, 32 * blocks), generator=g, device=DEV)
    code[:, K:] = 0
    mid = 127 - round(0.5 * math.log2(K)) - 2
    codes = torch.full((N, 16 * blocks + 16 * pad), 0x77, dtype=torch.uint8, device=DEV)
    codes[:, : 16 * blocks] = _pack(code)
    scales = torch.full((N, blocks + pad), 255, dtype=torch.uint8, device=DEV)
    scales[:, :blocks] = torch.randint(mid - spread, mid + spread + 1, (N, blocks), generator=g, device=DEV)
    return fw.Mxfp4(codes[:, : 16 * blocks], scales[:, :blocks])


def _mx_values(q, K):
    code = torch.stack([q.codes & 15, q.codes >> 4], 2).view(q.codes.shape[0], -1).long()
    size = torch.tensor(VALUES, dtype=torch.float64, device=DEV)
    v = torch.cat([size, -size])[code].view(code.shape[0], -1, 32)
    scale = torch.exp2(q.scales.double() - 127)
    scale[q.scales == 255] = NAN
    return (v * scale[..., None]).view(code.shape[0], -1)[:, :K]


def _mx_linear_check(x, w, bias, act, res, keep, add, y):
    """x and w [.., K] in 64 bits; products are exact, sums of depth d, the activation as in the gated product's."""
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ry = add * ACTS[act](z)
    extra = 0.0
    if res is not None:
        ry, extra = ry + keep * res.double(), 2 * U * (keep * res.double()).abs()
    # a matrix instruction adds up to 128 products; 32 + K / 32 + 40 covers them and the splits
    dz = (128 + _depth(x.shape[1])) * GEMM_UP * mag
    _near(y, ry, abs(add) * (1.13 * dz + 8 * U * (z.abs() + (act != "none"))) + 2 * U * ry.abs() + extra, "y")


MX_LINEAR = [(1, 1, 1), (1, 64, 64), (1, 100, 1000), (2, 2560, 512), (3, 17, 5), (7, 33, 2049), (16, 256, 128),
             (17, 48, 96), (33, 1000, 136), (64, 512, 2560), (65, 130, 72), (100, 64, 7), (129, 257, 65), (255, 96, 520),
             (256, 256, 64), (300, 513, 1024), (257, 264, 192), (520, 1040, 328), (1000, 1032, 2048), (2100, 2560, 1280),
             (3300, 3336, 136), (100, 100, 65536), (300, 300, 16384), (2048, 2100, 8200)]


@pytest.mark.parametrize("M,N,K", MX_LINEAR)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_mxfp4(M, N, K, dt):
    """x in 16 bits."""
    g = _gen(M * 3 + N * 5 + K)
    for act, yt, res, pad in (("none", dt, False, 0), ("silu", F32, True, 0), ("gelu", dt, True, 8), ("relu", dt, False, 3)):
        _say("linear_mxfp4", M, N, K, dt, act, yt, res, pad)
        x, w = _randn(g, (M, K), dt, 1.0, pad), _mx_weights(g, N, K, pad)
        bias = _randn(g, (N,)) if act != "relu" else None
        r = _randn(g, (M, N), yt, 1.0, pad) if res else None
        keep, add = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if res else (1.0, 1.0)
        y = fw.beam_moe_linear_mxfp4(x, w, bias, act=act, residual=r, keep=keep, add=add, out_dtype=yt)
        _mx_linear_check(x.double(), _mx_values(w, K), bias, act, r, keep, add, y)


# one and two row fragments to a wave; parts of K of one stage of 128 up to more than LDS holds, whole and ragged ones
MX_ROWS = [(17, 129, 4104), (32, 2000, 2048), (24, 40, 16392), (33, 132, 776), (64, 5120, 2560), (100, 1030, 4104),
           (257, 640, 1160), (384, 2560, 5120), (48, 8192, 1536), (256, 5120, 2560), (63, 126, 128), (1000, 1000, 904),
           (16, 16384, 2048), (16, 40000, 520), (40, 40000, 1000)]


@pytest.mark.parametrize("M,N,K", MX_ROWS)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_linear_mxfp4_of_some_rows(M, N, K, dt):
    """x in 16 bits, rows of whole chunks: padding around every operand, then scales of NaN at both ends of K."""
    _say("linear_mxfp4 rows", M, N, K, dt)
    g = _gen(M + N + K)
    x, w, bias = _randn(g, (M, K), dt, 1.0, 8), _mx_weights(g, N, K, 1), _randn(g, (N,))
    for act, yt, res in (("none", F32, True), ("gelu", dt, False)):
        buf = torch.full((M, N + 5), 7.0, device=DEV, dtype=yt)
        r = _randn(g, (M, N), yt, 1.0, 3) if res else None
        fw.beam_moe_linear_mxfp4(x, w, bias, act=act, residual=r, keep=0.5, add=0.75, out=buf[:, :N])
        _mx_linear_check(x.double(), _mx_values(w, K), bias, act, r, 0.5, 0.75, buf[:, :N])
        assert (buf[:, N:] == 7.0).all()
    want = fw.beam_moe_linear_mxfp4(x, w)
    assert torch.equal(want, fw.beam_moe_linear_mxfp4(x, w))
    w.scales[N // 2, 0] = w.scales[N - 1, -1] = 255
    got = fw.beam_moe_linear_mxfp4(x, w)
    bad = torch.zeros(N, dtype=torch.bool, device=DEV)
    bad[[N // 2, N - 1]] = True
    assert torch.equal(got[:, ~bad], want[:, ~bad]) and got[:, bad].isnan().all()


@pytest.mark.parametrize("M,N,K", MX_LINEAR)
def test_linear_mxfp4_of_two(M, N, K):
    """Both operands in 4 bits."""
    g = _gen(M * 3 + N * 5 + K + 1)
    for act, yt, res, pad in (("none", BF16, False, 0), ("silu", F32, True, 0), ("gelu", F16, True, 1),
                              ("relu", F16, False, 3), ("none", F32, False, 0)):
        _say("linear_mxfp4 of two", M, N, K, act, yt, res, pad)
        x, w = _mx_weights(g, M, K, pad, 3), _mx_weights(g, N, K, pad)
        bias = _randn(g, (N,)) if act != "relu" else None
        r = _randn(g, (M, N), yt, 1.0, pad) if res else None
        keep, add = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if res else (1.0, 1.0)
        y = fw.beam_moe_linear_mxfp4(x, w, bias, act=act, residual=r, keep=keep, add=add, out_dtype=yt)
        _mx_linear_check(_mx_values(x, K), _mx_values(w, K), bias, act, r, keep, add, y)


# 256-row tiles, whose scales need a workspace: rows and columns that end inside a tile or a chunk of eight, one tile to
# a workgroup and several, K inside a block, a half and a stage
MX_LARGE = [(4096, 4096, 512), (3900, 3995, 1003), (3990, 3992, 520), (4000, 3905, 256), (5000, 5003, 300), (9000, 4360, 96),
            (2500, 5120, 2600)]


@pytest.mark.parametrize("M,N,K", MX_LARGE)
def test_linear_mxfp4_of_two_large(M, N, K):
    g = _gen(M * 3 + N * 5 + K + 2)
    for act, yt, res, pad in (("none", BF16, False, 0), ("silu", F32, True, 0), ("gelu", F16, True, 1),
                              ("relu", BF16, True, 3), ("none", F16, False, 5), ("none", F32, False, 1)):
        _say("linear_mxfp4 large", M, N, K, act, yt, res, pad)
        x, w = _mx_weights(g, M, K, pad, 3), _mx_weights(g, N, K, pad)
        assert fw.load_library().beam_moe_linear_mxfp4_workspace_bytes(M, N, K, 3, x.codes.stride(0),
                                                                       w.codes.stride(0)) > 0
        bias = _randn(g, (N,)) if act in ("silu", "gelu") else None
        r = _randn(g, (M, N), yt, 1.0, pad) if res else None
        keep, add = (math.sqrt(2 / 3), math.sqrt(1 / 3)) if res else (1.0, 1.0)
        buf = torch.full((M, N + pad), 7.0, dtype=yt, device=DEV)
        y = fw.beam_moe_linear_mxfp4(x, w, bias, act=act, residual=r, keep=keep, add=add, out=buf[:, :N])
        _mx_linear_check(_mx_values(x, K), _mx_values(w, K), bias, act, r, keep, add, y)
        assert (buf[:, N:] == 7.0).all()
        again = fw.beam_moe_linear_mxfp4(x, w, bias, act=act, residual=r, keep=keep, add=add, out_dtype=yt)
        assert torch.equal(again, y)


def test_linear_mxfp4_large_nan_and_replay():
    """A NaN scale in its own row or column alone; captured and replayed beside eager calls."""
    _say("linear_mxfp4 large nan")
    M, N, K = 3900, 3995, 300
    g = _gen(12)
    x, w = _mx_weights(g, M, K), _mx_weights(g, N, K)
    want = fw.beam_moe_linear_mxfp4(x, w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = fw.beam_moe_linear_mxfp4(x, w)
    for k in range(3):
        x.scales[1000 + k, 9] = 255
        w.scales[3990 - 300 * k, 0] = 255
        graph.replay()
        torch.cuda.synchronize()
        rows, cols = torch.ones(M, dtype=torch.bool, device=DEV), torch.ones(N, dtype=torch.bool, device=DEV)
        rows[1000:1001 + k] = False
        cols[[3990 - 300 * i for i in range(k + 1)]] = False
        assert torch.equal(got[rows][:, cols], want[rows][:, cols])
        assert got[~rows].isnan().all() and got[:, ~cols].isnan().all()
        assert torch.equal(fw.beam_moe_linear_mxfp4(x, w).nan_to_num(), got.nan_to_num())


@pytest.mark.parametrize("M,N,K", [(3, 40, 100), (70, 90, 1003), (300, 264, 128)])
def test_linear_mxfp4_places(M, N, K):
    """Each block of K by itself: one code of x and of w set, every other zero, so that a wrong block, scale or order
    shows whatever the values; scales differ in every block."""
    _say("linear_mxfp4 places", M, N, K)
    blocks = -(-K // 32)
    g = _gen(K)
    xs = torch.randint(100, 150, (M, blocks), generator=g, device=DEV).to(torch.uint8)
    ws = torch.randint(100, 150, (N, blocks), generator=g, device=DEV).to(torch.uint8)
    for k in sorted({0, 1, 31, 32, K // 2, K - 1}):
        code = torch.zeros(max(M, N), 32 * blocks, dtype=torch.int64, device=DEV)
        code[:, k] = torch.randint(1, 16, (max(M, N),), generator=g, device=DEV)
        x, w = fw.Mxfp4(_pack(code[:M]), xs), fw.Mxfp4(_pack(code[:N].flip(0)), ws)
        want = _mx_values(x, K) @ _mx_values(w, K).t()
        assert torch.equal(fw.beam_moe_linear_mxfp4(x, w, out_dtype=F32).double(), want)
        got = fw.beam_moe_linear_mxfp4(_mx_values(x, K).to(BF16), w, out_dtype=F32)
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("M", [5, 70, 300])
def test_linear_mxfp4_in_place_padding_and_nan(M):
    _say("linear_mxfp4 places and nan", M)
    N, K = 70, 100
    g = _gen(M)
    w, x = _mx_weights(g, N, K, 1), _randn(g, (M, K), BF16)
    q = fw.beam_moe_quantize_mxfp4(x)
    for a in (x, q):
        buf = torch.full((M, N + 9), 7.0, device=DEV)
        buf[:, :N] = _randn(g, (M, N))
        want = fw.beam_moe_linear_mxfp4(a, w, residual=buf[:, :N], keep=0.5, out_dtype=F32)
        fw.beam_moe_linear_mxfp4(a, w, residual=buf[:, :N], keep=0.5, out=buf[:, :N])
        assert torch.equal(buf[:, :N], want) and (buf[:, N:] == 7.0).all()
        assert torch.equal(fw.beam_moe_linear_mxfp4(a, w), fw.beam_moe_linear_mxfp4(a, w))
    # NaN of one row of x, and of one block of one column of w
    want = fw.beam_moe_linear_mxfp4(q, w)
    q.scales[M // 2, 1] = 255
    got = fw.beam_moe_linear_mxfp4(q, w)
    rows = torch.arange(M, device=DEV) != M // 2
    assert torch.equal(got[rows], want[rows]) and got[M // 2].isnan().all()
    want = fw.beam_moe_linear_mxfp4(x, w)
    w.scales[9, 2] = 255
    cols = torch.arange(N, device=DEV) != 9
    for a, was in ((x, want), (q, got)):
        got = fw.beam_moe_linear_mxfp4(a, w)
        assert torch.equal(got[:, cols].nan_to_num(), was[:, cols].nan_to_num()) and got[:, 9].isnan().all()


def test_linear_mxfp4_scales_at_the_ends():
    """Scales at the ends of their range: 2^-127 times 2^127, and products that leave FP32 in neither direction."""
    _say("linear_mxfp4 ends")
    for M in (4, 40):
        K, N = 64, 48
        g = _gen(M)
        code = torch.randint(0, 16, (max(M, N), K), generator=g, device=DEV)
        for xs, ws in ((0, 254), (254, 0), (1, 250), (0, 127), (127, 127), (100, 10)):
            x = fw.Mxfp4(_pack(code[:M]), torch.full((M, 2), xs, dtype=torch.uint8, device=DEV))
            w = fw.Mxfp4(_pack(code[:N]), torch.full((N, 2), ws, dtype=torch.uint8, device=DEV))
            vx, vw = _mx_values(x, K), _mx_values(w, K)
            y = fw.beam_moe_linear_mxfp4(x, w, out_dtype=F32)
            _near(y, vx @ vw.t(), 200 * GEMM_UP * (vx.abs() @ vw.abs().t()) + 64 * 2.0 ** -149)


def test_serving_a_gated_sublayer_in_four_bits():
    """The sublayer of the training step with its weights quantised once: both projections of the quantised weights,
    the activation and the product, and the down projection onto the stream, against 64 bits on the same quantised
    weights. Four roundings to bf16 lie on the way (norm, gate, up, h)."""
    _say("serving in four bits")
    for T in (1, 9, 192):
        s = _gated_step_inputs(1, T)
        q = {k: fw.beam_moe_quantize_mxfp4(s[k]) for k in ("wg", "wu", "wd")}
        x, _, _ = fw.beam_moe_layer_norm(s["stream"], s["gamma"], s["beta"], out_dtype=BF16)
        gate = fw.beam_moe_linear_mxfp4(x, q["wg"], s["bg"], act="silu")
        up = fw.beam_moe_linear_mxfp4(x, q["wu"], s["bu"])
        out = fw.beam_moe_linear_mxfp4(gate * up, q["wd"], residual=s["stream"], keep=0.8, add=0.6, out_dtype=F32)
        w = {k: fw.beam_moe_dequantize_mxfp4(v, s[k].shape[1], out_dtype=F32).double() for k, v in q.items()}
        xr = torch.nn.functional.layer_norm(s["stream"].double(), (s["stream"].shape[1],), s["gamma"].double(),
                                            s["beta"].double(), 1e-5)
        h = torch.nn.functional.silu(xr @ w["wg"].t() + s["bg"].double()) * (xr @ w["wu"].t() + s["bu"].double())
        want = 0.8 * s["stream"].double() + 0.6 * (h @ w["wd"].t())
        err = float((out.double() - want).norm() / want.norm())
        assert err <= 8 * 2.0 ** -9, (T, err)


# strides of codes just inside the persistent kernel's bound, and past it
@pytest.mark.parametrize("ld", [(1 << 23) - 16, 1 << 23])
@pytest.mark.parametrize("M,N,K", [(520, 16384, 2560), (16384, 520, 2560)])
def test_linear_mxfp4_of_two_with_far_rows(M, N, K, ld):
    """Codes whose rows span more than 2^32 bytes."""
    _say("linear_mxfp4 far rows", M, N, K, ld)
    g = _gen(M + N)
    x, w = _mx_weights(g, M, K, 0, 3), _mx_weights(g, N, K)
    far = torch.zeros(min(M, N), ld, dtype=torch.uint8, device=DEV)
    assert far.numel() > 1 << 32
    q = x if M < N else w
    far[:, : K // 2] = q.codes
    q = fw.Mxfp4(far[:, : K // 2], q.scales)
    x, w = (q, w) if M < N else (x, q)
    need = fw.load_library().beam_moe_linear_mxfp4_workspace_bytes(M, N, K, 3, x.codes.stride(0), w.codes.stride(0))
    assert (need > 0) == (ld < 1 << 23)
    y = fw.beam_moe_linear_mxfp4(x, w, out_dtype=F32)
    _mx_linear_check(_mx_values(x, K), _mx_values(w, K), None, "none", None, 1.0, 1.0, y)


# the kernel for few rows, tiles that hold codes, codes through registers, and w laid out as x's type
@pytest.mark.parametrize("M,K", [(8, 2560), (64, 2560), (64, 2557), (3000, 2560)])
def test_linear_mxfp4_with_far_rows(M, K):
    """Weights whose codes span more than 2^32 bytes, and rows of x more than 2^31 elements."""
    N = 520
    _say("linear_mxfp4 far rows", M, N, K)
    g = _gen(M + K)
    w, x0 = _mx_weights(g, N, K), _randn(g, (M, K), BF16)
    far = torch.zeros(N, 1 << 23, dtype=torch.uint8, device=DEV)
    wide = torch.zeros(M, -(-(9 << 28) // M // 8) * 8, dtype=BF16, device=DEV)
    assert far.numel() > 1 << 32 and wide.numel() > 1 << 31
    far[:, : w.codes.shape[1]] = w.codes
    wide[:, :K] = x0
    w = fw.Mxfp4(far[:, : w.codes.shape[1]], w.scales)
    y = fw.beam_moe_linear_mxfp4(wide[:, :K], w, out_dtype=F32)
    _mx_linear_check(x0.double(), _mx_values(w, K), None, "none", None, 1.0, 1.0, y)
