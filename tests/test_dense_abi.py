"""Host-side validation of the operators of a dense gated sublayer (gradient norm and clipping, microscaled 4-bit
floating point, the gated projections): every rejected call returns before any device work.  CPU only."""
import ctypes

import pytest
import torch

from grouped_top_routing_fp32_amd import binding
from test_sublayer_abi import BAD, BF16, F16, F32, FAKE, ODD, OK, UNSUP, WS, Call

A = [ctypes.c_void_p((k + 1) << 24) for k in range(8)]     # apart from each other, never dereferenced


def ptrs(*p):
    return (ctypes.c_void_p * len(p))(*[q.value if q is not None else None for q in p])


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def sizes(*v):
    return (ctypes.c_int64 * len(v))(*v)


GATED = Call("beam_moe_gated_linear", rows=40, cols=10, inner=12, type=BF16, x=FAKE, ldx=12, w_gate=FAKE, ldg=12,
             w_up=FAKE, ldu=12, bias_gate=FAKE, bias_up=FAKE, act=2, h=FAKE, h_type=F32, ldh=10, pre_gate=FAKE, ldpg=10,
             pre_up=FAKE, ldpu=10, ws=FAKE, ws_bytes=1 << 40, stream=None)
GATED_BACK = Call("beam_moe_gated_linear_backward", rows=4, cols=10, inner=12, type=F16, dh=FAKE, dh_type=F32, lddh=10,
                  x=FAKE, ldx=12, w_gate=FAKE, ldg=12, w_up=FAKE, ldu=12, pre_gate=FAKE, ldpg=10, pre_up=FAKE, ldpu=10,
                  act=2, dx=FAKE, lddx=12, dw_gate=FAKE, lddwg=12, dw_up=FAKE, lddwu=12, dbias_gate=FAKE,
                  dbias_up=FAKE, ws=FAKE, ws_bytes=1 << 40, stream=None)
NORM = Call("beam_moe_grad_norm", count=2, grads=ptrs(A[0], A[1]), types=ints(BF16, F32), sizes=sizes(5, 7), scale=1.0,
            norm=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
CLIP = Call("beam_moe_clip_grads", count=2, grads=ptrs(A[0], A[1]), types=ints(BF16, F32), sizes=sizes(5, 7), scale=1.0,
            max_norm=1.0, eps=1e-6, norm_in=None, outs=ptrs(A[2], A[3]), out_types=ints(F32, F32), norm=FAKE, ws=FAKE,
            ws_bytes=1 << 30, stream=None)
QUANT = Call("beam_moe_quantize_mxfp4", rows=4, cols=70, x=FAKE, x_type=BF16, ldx=70, codes=FAKE, ldc=48, scales=FAKE,
             lds=3, stream=None)
DEQUANT = Call("beam_moe_dequantize_mxfp4", rows=4, cols=70, codes=FAKE, ldc=48, scales=FAKE, lds=3, y=FAKE,
               y_type=BF16, ldy=70, stream=None)

MX = binding.BEAM_MOE_MXFP4
MX_LINEAR = Call("beam_moe_linear_mxfp4", rows=4, cols=10, inner=70, x_type=BF16, x=FAKE, ldx=70, x_scales=None, ldxs=0,
                 w=FAKE, ldw=48, w_scales=FAKE, ldws=3, bias=FAKE, act=1, res=FAKE, ldr=10, keep=0.5, add=0.5,
                 y=ctypes.c_void_p(2 << 20), y_type=F32, ldy=10, ws=FAKE, ws_bytes=1 << 40, stream=None)
MX_BOTH = Call("beam_moe_linear_mxfp4", **{**MX_LINEAR.defaults, "x_type": MX, "ldx": 48, "x_scales": FAKE, "ldxs": 3})


@pytest.mark.parametrize("call, required, optional", [
    (NORM, ("norm",), ()), (CLIP, (), ("norm",)), (QUANT, ("x", "codes", "scales"), ()),
    (DEQUANT, ("codes", "scales", "y"), ()),
    (MX_LINEAR, ("x", "w", "w_scales", "y"), ("bias", "res")),
    (MX_BOTH, ("x", "x_scales", "w", "w_scales", "y"), ("bias", "res")),
    (GATED, ("x", "w_gate", "w_up", "h"), ("bias_gate", "bias_up", "pre_gate", "pre_up")),
    (GATED_BACK, ("dh", "pre_gate", "pre_up"), ("x", "w_gate", "w_up", "dx", "dw_gate", "dw_up", "dbias_gate",
                                                "dbias_up")),
], ids=lambda v: v.fn if isinstance(v, Call) else "")
def test_pointers(call, required, optional):
    for name in required:
        assert call(**{name: None}) == BAD, name
    for name in required + optional:
        assert call(**{name: ODD}) == BAD, name


@pytest.mark.parametrize("call, bad", [
    (c, b) for c in (NORM, CLIP) for b in (
        dict(count=-1), dict(grads=None), dict(types=None), dict(sizes=None), dict(types=ints(BF16, 3)),
        dict(sizes=sizes(5, -1)), dict(grads=ptrs(A[0], None)), dict(scale=float("nan")), dict(scale=float("inf")),
        dict(grads=ptrs(ctypes.c_void_p(A[0].value + 1), A[1])), dict(grads=ptrs(A[0], ctypes.c_void_p(A[1].value + 2))))
] + [
    (CLIP, dict(max_norm=-1.0)), (CLIP, dict(max_norm=float("inf"))), (CLIP, dict(max_norm=float("nan"))),
    (CLIP, dict(norm_in=ctypes.c_void_p((1 << 20) + 2))), (CLIP, dict(eps=0.0)), (CLIP, dict(eps=-1e-6)), (CLIP, dict(eps=float("nan"))), (CLIP, dict(outs=None)),
    (CLIP, dict(out_types=ints(F32, 9))), (CLIP, dict(outs=ptrs(A[2], None))),
    (CLIP, dict(outs=ptrs(ctypes.c_void_p(A[2].value + 2), A[3]))),
    # outputs that overlap each other, another gradient, or their own of another type
    (CLIP, dict(outs=ptrs(A[2], A[2]))), (CLIP, dict(outs=ptrs(A[2], ctypes.c_void_p(A[2].value + 16)))),
    (CLIP, dict(outs=ptrs(A[1], A[2]))), (CLIP, dict(outs=ptrs(A[2], ctypes.c_void_p(A[0].value + 8)))),
    (CLIP, dict(outs=ptrs(A[0], A[3]))), (CLIP, dict(outs=ptrs(A[2], ctypes.c_void_p(A[1].value + 4)))),
    (CLIP, dict(grads=ptrs(A[0], A[0]), types=ints(BF16, BF16), outs=None, out_types=None)),
    (QUANT, dict(rows=-1)), (QUANT, dict(x_type=3)), (QUANT, dict(ldx=69)), (QUANT, dict(ldc=32)),
    (QUANT, dict(ldc=56)), (QUANT, dict(lds=2)), (QUANT, dict(lds=1 << 41)),
    (DEQUANT, dict(rows=-1)), (DEQUANT, dict(y_type=-1)), (DEQUANT, dict(ldy=69)), (DEQUANT, dict(ldc=40)),
    (DEQUANT, dict(lds=2)),
    (MX_LINEAR, dict(x_type=F32)), (MX_LINEAR, dict(x_type=4)), (MX_LINEAR, dict(y_type=F16)),
    (MX_LINEAR, dict(ldx=69)), (MX_BOTH, dict(y_type=3)), (MX_BOTH, dict(ldx=32)), (MX_BOTH, dict(ldx=56)),
    (MX_BOTH, dict(ldxs=2)),
] + [
    (c, b) for c in (MX_LINEAR, MX_BOTH) for b in (
        dict(rows=-1), dict(act=4), dict(act=-1), dict(keep=float("nan")), dict(add=float("inf")), dict(ldw=32),
        dict(ldw=56), dict(ldws=2), dict(ldy=9), dict(ldr=9), dict(y=FAKE, ldy=11), dict(ldw=1 << 41))
] + [
    (GATED, dict(rows=-1)), (GATED, dict(type=F32)), (GATED, dict(h_type=F16)), (GATED, dict(act=4)),
    (GATED, dict(act=-1)), (GATED, dict(ldx=11)), (GATED, dict(ldg=11)), (GATED, dict(ldu=11)), (GATED, dict(ldh=9)),
    (GATED, dict(ldpg=9)), (GATED, dict(ldpu=9)), (GATED, dict(ldx=1 << 41)),
    (GATED_BACK, dict(rows=-1)), (GATED_BACK, dict(type=F32)), (GATED_BACK, dict(dh_type=BF16)),
    (GATED_BACK, dict(act=9)), (GATED_BACK, dict(dw_gate=None)), (GATED_BACK, dict(dw_up=None)),
    (GATED_BACK, dict(dbias_gate=None)), (GATED_BACK, dict(dbias_up=None)), (GATED_BACK, dict(x=None)),
    (GATED_BACK, dict(w_gate=None)), (GATED_BACK, dict(w_up=None)), (GATED_BACK, dict(lddh=9)),
    (GATED_BACK, dict(ldx=11)), (GATED_BACK, dict(ldg=11)), (GATED_BACK, dict(ldu=11)), (GATED_BACK, dict(ldpg=9)),
    (GATED_BACK, dict(ldpu=9)), (GATED_BACK, dict(lddx=11)), (GATED_BACK, dict(lddwg=11)), (GATED_BACK, dict(lddwu=11)),
    (GATED_BACK, dict(dx=None, dw_gate=None, dw_up=None, dbias_gate=None, dbias_up=None)),
], ids=lambda v: v.fn if isinstance(v, Call) else "-".join(v) if isinstance(v, dict) else "")
def test_invalid_arguments(call, bad):
    assert call(**bad) == BAD


@pytest.mark.parametrize("call, big", [
    (NORM, dict(count=(1 << 16) + 1)), (CLIP, dict(count=(1 << 16) + 1)), (NORM, dict(sizes=sizes(5, (1 << 40) + 1))),
    (QUANT, dict(rows=(1 << 20) + 1)), (QUANT, dict(cols=(1 << 18) + 1)), (QUANT, dict(cols=0)),
    (DEQUANT, dict(rows=(1 << 20) + 1)), (DEQUANT, dict(cols=(1 << 18) + 1)), (DEQUANT, dict(cols=0)),
] + [
    (c, b) for c in (MX_LINEAR, MX_BOTH) for b in (dict(rows=(1 << 20) + 1), dict(cols=(1 << 18) + 1), dict(cols=0),
                                                   dict(inner=(1 << 18) + 1), dict(inner=0))
] + [
    (c, b) for c in (GATED, GATED_BACK) for b in (dict(rows=(1 << 20) + 1), dict(cols=(1 << 17) + 1), dict(cols=0),
                                                  dict(inner=(1 << 18) + 1), dict(inner=0))
], ids=lambda v: v.fn if isinstance(v, Call) else "-".join(v) if isinstance(v, dict) else "")
def test_unsupported_sizes(call, big):
    assert call(**big) == UNSUP


@pytest.mark.parametrize("bad", [dict(norm_in=A[2]), dict(norm_in=ctypes.c_void_p(A[3].value + 24)),
                                 dict(outs=None, out_types=None, norm_in=A[1]), dict(norm=A[0]), dict(norm=A[2]),
                                 dict(norm=ctypes.c_void_p(A[3].value + 16)), dict(outs=None, out_types=None, norm=A[1])])
def test_norms_inside_the_lists(bad):
    """A norm that other workgroups overwrite while it is read, or read as a gradient while it is written."""
    assert CLIP(**bad) == BAD


def test_too_many_elements_in_all():
    n = 17
    args = dict(count=n, grads=ptrs(*[A[0]] * n), types=ints(*[BF16] * n), sizes=sizes(*[1 << 40] * n))
    assert NORM(**args) == UNSUP and CLIP(**args) == UNSUP


def test_workspaces():
    lib = binding.load_library()
    need = lib.beam_moe_grad_norm_workspace_bytes(2)
    assert 0 < need < 1 << 20
    assert lib.beam_moe_grad_norm_workspace_bytes(-1) == lib.beam_moe_grad_norm_workspace_bytes((1 << 16) + 1) \
        == binding.SIZE_MAX
    for call in (NORM, CLIP):
        assert call(ws=None) == WS and call(ws=ODD) == WS and call(ws_bytes=need - 1) == WS


def test_gated_workspaces():
    lib = binding.load_library()
    need = lib.beam_moe_gated_linear_workspace_bytes
    assert need(16, 1000, 1000, 1000, 1000, 1000) == 0       # few rows
    assert need(8192, 2560, 5120, 5120, 5120, 5120) == 0     # whole tiles
    assert need(64, 2560, 5120, 5120, 5120, 5120) > 0        # split
    assert need(-1, 8, 8, 8, 8, 8) == need(8, 8, 8, 7, 8, 8) == need(8, 8, 8, 8, 8, 7) == need(8, 0, 8, 8, 8, 8) \
        == binding.SIZE_MAX
    n = need(64, 2560, 5120, 5120, 5120, 5120)
    sizes_ = dict(rows=64, cols=2560, inner=5120, ldx=5120, ldg=5120, ldu=5120, ldh=2560, ldpg=2560, ldpu=2560)
    for bad in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=n - 1)):
        assert GATED(**sizes_, **bad) == WS
    back = lib.beam_moe_gated_linear_backward_workspace_bytes
    n = back(4, 10, 12, 12, 12, 12)
    assert 0 < n < 1 << 20
    assert back(-1, 8, 8, 8, 8, 8) == back(8, 8, 8, 8, 7, 8) == binding.SIZE_MAX
    for bad in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=n - 1)):
        assert GATED_BACK(**bad) == WS


def test_mx_workspaces():
    need = binding.load_library().beam_moe_linear_mxfp4_workspace_bytes
    assert need(16, 1000, 1000, BF16, 1000, 512) == 0 and need(16, 1000, 1000, MX, 512, 512) == 0
    assert need(300, 300, 1000, MX, 512, 512) == 0
    # scales laid out by tiles: a byte to a block of 32
    assert need(8192, 2560, 5120, MX, 2560, 2560) == (8192 + 2560) * 160
    assert need(8192, 2560, 5120, MX, 2560, 1 << 23) == 0
    assert need(64, 2560, 5120, BF16, 5120, 2560) > 0                          # split
    assert need(8192, 2560, 5120, BF16, 5120, 2560) >= 2560 * 5120 * 2         # w as x's type
    assert need(-1, 8, 8, BF16, 8, 16) == need(8, 8, 8, BF16, 7, 16) == need(8, 8, 8, MX, 8, 16) \
        == need(8, 8, 8, F32, 8, 16) == need(8, 0, 8, BF16, 8, 16) == need(8, 8, 8, BF16, 8, 8) == binding.SIZE_MAX
    n = need(8192, 2560, 5120, MX, 2560, 2560)
    for bad in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=n - 1)):
        assert MX_BOTH(rows=8192, cols=2560, inner=5120, ldx=2560, ldxs=160, ldw=2560, ldws=160, ldy=2560, ldr=2560,
                       **bad) == WS


def test_no_rows():
    for call in (QUANT, DEQUANT, GATED, MX_LINEAR, MX_BOTH):
        assert call(rows=0) == OK


def test_binding_refuses_what_is_not_on_the_device():
    for grads in ([], [torch.zeros(3)], [torch.zeros(3, dtype=torch.int32)], [torch.zeros(3, 4)[:, ::2]]):
        with pytest.raises(ValueError):
            binding.beam_moe_grad_norm(grads)
        with pytest.raises(ValueError):
            binding.beam_moe_clip_grads(grads, 1.0)
    with pytest.raises(ValueError):
        binding.beam_moe_quantize_mxfp4(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        binding.beam_moe_dequantize_mxfp4((torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.uint8)))


@pytest.mark.parametrize("rows", [0, 1, 16, 17, 1 << 20])
@pytest.mark.parametrize("cols, inner", [(1, 1), (1, 1 << 18), (1 << 18, 8), (1 << 18, 1 << 18)])
def test_workspaces_at_the_ends_of_the_sizes(rows, cols, inner):
    """A size query answers for every size the header allows, no rows among them."""
    lib = binding.load_library()
    blocks = (inner + 31) // 32
    for x_type, ldx in ((BF16, inner), (F16, inner + 1), (MX, 16 * blocks)):
        assert lib.beam_moe_linear_mxfp4_workspace_bytes(rows, cols, inner, x_type, ldx, 16 * blocks) < 1 << 50
    cols = min(cols, 1 << 17)
    for query in (lib.beam_moe_gated_linear_workspace_bytes, lib.beam_moe_gated_linear_backward_workspace_bytes):
        assert query(rows, cols, inner, inner, inner, inner) < 1 << 50
