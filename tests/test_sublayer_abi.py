"""Host-side validation of the operators around the block (layer norm, balance loss, the
router's gradient, linear): every rejected call returns before any device work.  CPU only."""
import ctypes

import pytest
import torch

from grouped_top_routing_fp32_amd import binding
from grouped_top_routing_fp32_amd.synth import BEAM, Dims

FAKE = ctypes.c_void_p(1 << 20)             # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
BF16, F16, F32 = binding.BEAM_MOE_BF16, binding.BEAM_MOE_F16, binding.BEAM_MOE_F32
OK, BAD, UNSUP, WS = (binding.BEAM_MOE_OK, binding.BEAM_MOE_ERR_INVALID_ARG, binding.BEAM_MOE_ERR_UNSUPPORTED,
                      binding.BEAM_MOE_ERR_WORKSPACE)


class Call:
    """A C entry point with valid default arguments, some of them replaced by name."""

    def __init__(self, fn, **defaults):
        self.fn, self.defaults = fn, defaults

    def __call__(self, **changed):
        assert set(changed) <= set(self.defaults)
        return getattr(binding.load_library(), self.fn)(*{**self.defaults, **changed}.values())


NORM = Call("beam_moe_layer_norm", rows=4, cols=100, x=FAKE, x_type=BF16, ldx=100, gamma=FAKE, beta=FAKE, eps=1e-5,
            y=FAKE, y_type=BF16, ldy=100, mean=FAKE, rstd=FAKE, stream=None)
NORM_BACK = Call("beam_moe_layer_norm_backward", rows=4000, cols=100, dy=FAKE, dy_type=BF16, lddy=100, x=FAKE,
                 x_type=F32, ldx=100, mean=FAKE, rstd=FAKE, gamma=FAKE, dx=FAKE, lddx=100, dgamma=FAKE, dbeta=FAKE,
                 ws=FAKE, ws_bytes=1 << 40, stream=None)
BALANCE = Call("beam_moe_balance_loss", dims=ctypes.byref(binding._cdims(BEAM)), T=1024, scores=FAKE, ids=FAKE,
               num_seqs=3, off=FAKE, alpha=1e-3, loss=FAKE, counts=FAKE, prob=FAKE, ws=FAKE, ws_bytes=1 << 40,
               stream=None)
ROUTE_BACK = Call("beam_moe_route_backward", dims=ctypes.byref(binding._cdims(BEAM)), T=8, scores=FAKE, ids=FAKE,
                  dw=FAKE, num_seqs=3, off=FAKE, alpha=1e-3, dloss=FAKE, counts=FAKE, dlogits=FAKE, stream=None)
LINEAR = Call("beam_moe_linear", rows=4, cols=10, inner=12, type=BF16, x=FAKE, ldx=12, w=FAKE, ldw=12, bias=FAKE,
              act=1, res=FAKE, ldr=10, keep=0.5, add=0.5, y=ctypes.c_void_p(2 << 20), y_type=F32, ldy=10, pre=FAKE,
              ldpre=10, ws=FAKE, ws_bytes=1 << 40, stream=None)
LINEAR_BACK = Call("beam_moe_linear_backward", rows=4, cols=10, inner=12, type=F16, dy=FAKE, dy_type=F32, lddy=10,
                   x=FAKE, ldx=12, w=FAKE, ldw=12, pre=FAKE, ldpre=10, act=2, keep=1.0, add=1.0, dx=FAKE, lddx=12,
                   dw=FAKE, lddw=12, dbias=FAKE, dres=FAKE, lddres=10, ws=FAKE, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("call, required, optional", [
    (NORM, ("x", "y"), ("gamma", "beta", "mean", "rstd")),
    (NORM_BACK, ("dy", "x", "mean", "rstd"), ("gamma", "dx", "dgamma", "dbeta")),
    (BALANCE, ("scores", "ids", "loss", "counts", "prob"), ("off",)),
    (ROUTE_BACK, ("scores", "ids", "dlogits"), ("dw", "dloss", "counts", "off")),
    (LINEAR, ("x", "w", "y"), ("bias", "res", "pre")),
    (LINEAR_BACK, ("dy",), ("x", "w", "pre", "dx", "dw", "dbias", "dres")),
], ids=lambda v: v.fn if isinstance(v, Call) else "")
def test_pointers(call, required, optional):
    for name in required:
        assert call(**{name: None}) == BAD, name
    for name in required + optional:
        assert call(**{name: ODD}) == BAD, name


@pytest.mark.parametrize("call, bad", [
    (NORM, dict(rows=-1)), (NORM, dict(x_type=3)), (NORM, dict(y_type=-1)), (NORM, dict(eps=-1.0)),
    (NORM, dict(eps=float("nan"))), (NORM, dict(ldx=99)), (NORM, dict(ldy=99)), (NORM, dict(ldx=1 << 41)),
    (NORM_BACK, dict(rows=-1)), (NORM_BACK, dict(dy_type=7)), (NORM_BACK, dict(x_type=7)),
    (NORM_BACK, dict(ldx=99)), (NORM_BACK, dict(lddy=99)), (NORM_BACK, dict(lddx=99)),
    (NORM_BACK, dict(dx=None, dgamma=None, dbeta=None)),
    (BALANCE, dict(T=-1)), (BALANCE, dict(num_seqs=0)), (BALANCE, dict(off=None)),
    (BALANCE, dict(alpha=float("inf"))), (BALANCE, dict(dims=None)),
    (ROUTE_BACK, dict(T=-1)), (ROUTE_BACK, dict(num_seqs=0)), (ROUTE_BACK, dict(off=None)),
    (ROUTE_BACK, dict(dw=None, dloss=None)), (ROUTE_BACK, dict(counts=None)),
    (ROUTE_BACK, dict(alpha=float("nan"))), (ROUTE_BACK, dict(dims=None)),
    (LINEAR, dict(rows=-1)), (LINEAR, dict(type=F32)), (LINEAR, dict(y_type=F16)), (LINEAR, dict(act=4)),
    (LINEAR, dict(act=-1)), (LINEAR, dict(keep=float("nan"))), (LINEAR, dict(add=float("inf"))),
    (LINEAR, dict(ldx=11)), (LINEAR, dict(ldw=11)), (LINEAR, dict(ldy=9)), (LINEAR, dict(ldr=9)),
    (LINEAR, dict(ldpre=9)), (LINEAR, dict(y=FAKE, ldy=11)),
    (LINEAR_BACK, dict(rows=-1)), (LINEAR_BACK, dict(type=F32)), (LINEAR_BACK, dict(dy_type=BF16)),
    (LINEAR_BACK, dict(act=9)), (LINEAR_BACK, dict(pre=None)), (LINEAR_BACK, dict(x=None)),
    (LINEAR_BACK, dict(w=None)), (LINEAR_BACK, dict(lddy=9)), (LINEAR_BACK, dict(ldx=11)),
    (LINEAR_BACK, dict(lddx=11)), (LINEAR_BACK, dict(lddw=11)), (LINEAR_BACK, dict(lddres=9)),
    (LINEAR_BACK, dict(ldpre=9)), (LINEAR_BACK, dict(dx=None, dw=None, dbias=None, dres=None)),
    (LINEAR_BACK, dict(add=float("nan"))),
], ids=lambda v: v.fn if isinstance(v, Call) else ",".join(v))
def test_invalid_arguments(call, bad):
    assert call(**bad) == BAD


@pytest.mark.parametrize("call, bad", [
    (NORM, dict(cols=0)), (NORM, dict(cols=16385, ldx=1 << 20, ldy=1 << 20)), (NORM, dict(rows=(1 << 21) + 1)),
    (NORM_BACK, dict(cols=0)), (NORM_BACK, dict(cols=16385)), (NORM_BACK, dict(rows=(1 << 21) + 1)),
    (BALANCE, dict(num_seqs=(1 << 20) + 1)), (BALANCE, dict(T=(1 << 25) + 1)),
    (BALANCE, dict(dims=ctypes.byref(binding._cdims(Dims(5120, 2560, 512, 8, 4, 8))))),
    (ROUTE_BACK, dict(num_seqs=(1 << 20) + 1)), (ROUTE_BACK, dict(T=(1 << 25) + 1)),
    (ROUTE_BACK, dict(T=(1 << 25) + 1, dims=ctypes.byref(binding._cdims(Dims(5120, 2560, 256, 8, 4, 1))))),
    (LINEAR, dict(cols=0)), (LINEAR, dict(inner=0)), (LINEAR, dict(rows=(1 << 20) + 1)),
    (LINEAR, dict(cols=(1 << 18) + 1)), (LINEAR, dict(inner=(1 << 18) + 1)),
    (LINEAR_BACK, dict(cols=0)), (LINEAR_BACK, dict(inner=(1 << 18) + 1)), (LINEAR_BACK, dict(rows=(1 << 20) + 1)),
], ids=lambda v: v.fn if isinstance(v, Call) else ",".join(v))
def test_unsupported_sizes(call, bad):
    assert call(**bad) == UNSUP


@pytest.mark.parametrize("call, need", [
    (NORM_BACK, lambda lib: lib.beam_moe_layer_norm_backward_workspace_bytes(4000, 100)),
    (BALANCE, lambda lib: lib.beam_moe_balance_loss_workspace_bytes(ctypes.byref(binding._cdims(BEAM)), 1024, 3)),
    (LINEAR_BACK, lambda lib: lib.beam_moe_linear_backward_workspace_bytes(4, 10, 12, 12, 12)),
], ids=lambda v: v.fn if isinstance(v, Call) else "")
def test_workspace(call, need):
    n = need(binding.load_library())
    assert 0 < n < 1 << 30
    assert call(ws_bytes=n - 1) == WS
    assert call(ws=None) == WS
    assert call(ws=ODD) == WS


def test_workspace_queries_refuse_what_the_calls_refuse():
    lib = binding.load_library()
    none = binding.SIZE_MAX
    assert lib.beam_moe_layer_norm_backward_workspace_bytes(4, 16385) == none
    assert lib.beam_moe_layer_norm_backward_workspace_bytes(-1, 16) == none
    assert lib.beam_moe_layer_norm_backward_workspace_bytes(1024, 16) == 0
    assert lib.beam_moe_layer_norm_backward_workspace_bytes(1025, 16) == 8 * 256 * 16
    beam = ctypes.byref(binding._cdims(BEAM))
    assert lib.beam_moe_balance_loss_workspace_bytes(beam, 8, 0) == none
    assert lib.beam_moe_balance_loss_workspace_bytes(beam, -1, 1) == none
    assert lib.beam_moe_balance_loss_workspace_bytes(beam, 8, 1) == 0
    for fn in (lib.beam_moe_linear_workspace_bytes, lib.beam_moe_linear_backward_workspace_bytes):
        assert fn(4, 0, 8, 8, 8) == none
        assert fn(4, 8, 8, 7, 8) == none
        assert fn(4, 8, 8, 8, 8) != none
    with pytest.raises(binding.BeamMoeError):
        binding._scratch(none, None, torch.device("cpu"), "x")


def test_workspace_of_a_small_result_with_a_long_k():
    """16 tiles of 128 rows fill no more than the CUs however K is split: 64-row tiles, split until two workgroups a CU
    have work, eight times for 64 of them."""
    lib = binding.load_library()
    assert lib.beam_moe_linear_workspace_bytes(512, 512, 9216, 9216, 9216) == 8 * 512 * 512 * 4
    assert lib.beam_moe_linear_workspace_bytes(640, 512, 9216, 9216, 9216) == 16 * 640 * 512 * 4


def test_zero_rows_is_a_no_op_where_every_output_is_empty():
    assert NORM(rows=0, x=None, y=None, gamma=None, beta=None, mean=None, rstd=None) == OK
    assert NORM_BACK(rows=0, dy=None, x=None, mean=None, rstd=None, gamma=None, dgamma=None, dbeta=None) == OK
    assert ROUTE_BACK(T=0, scores=None, ids=None, dlogits=None) == OK
    assert LINEAR(rows=0, x=None, y=None, res=None, pre=None, ws=None, ws_bytes=0) == OK
    assert LINEAR_BACK(rows=0, dy=None, x=None, pre=None, dw=None, dbias=None, dres=None, ws=None, ws_bytes=0) == OK


def test_binding_refuses_before_the_library_is_called():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="device tensor"):
        binding.beam_moe_layer_norm(x)
    with pytest.raises(ValueError, match="matrix"):
        binding.beam_moe_layer_norm(x[0])
    with pytest.raises(ValueError, match="device tensor"):
        binding.beam_moe_linear(x.bfloat16(), x.bfloat16())
    with pytest.raises(ValueError, match="needed"):
        binding.beam_moe_linear_backward(x, None, None)
    with pytest.raises(ValueError, match="act"):
        binding._act("tanh")
    with pytest.raises(ValueError, match="device tensor"):
        binding.beam_moe_balance_loss(BEAM, torch.zeros(4, 256), torch.zeros(4, 8, dtype=torch.int32), alpha=1.0)
