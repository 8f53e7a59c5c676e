"""Beam MoE block forward on MI355X (gfx950): group-limited sigmoid router,
counting-sort dispatch, grouped bf16 SwiGLU expert GEMMs and a deterministic
combine, behind the C-ABI library ``libbeam_moe.so``; and the operators a
training step or a dense sublayer needs beside it (layer norm, the router's
balance loss and gradient, linear with bias, activation and residual; gated
projections, gradient clipping and microscaled 4-bit floating point).

The binding is loaded lazily: ``from grouped_top_routing_fp32_amd import
binding`` (or any of the ``beam_moe_*`` names below) loads the built library
and fails loudly when it is missing.
"""

_EXPORTS = ("beam_moe_route", "beam_moe_select", "beam_moe_dispatch", "beam_moe_forward", "beam_moe_forward_fp8",
            "beam_moe_residual_forward", "beam_moe_residual_forward_fp8", "beam_moe_layer_norm",
            "beam_moe_layer_norm_backward", "beam_moe_balance_loss", "beam_moe_route_backward", "beam_moe_linear",
            "beam_moe_linear_backward", "beam_moe_gated_linear", "beam_moe_gated_linear_backward",
            "beam_moe_grad_norm", "beam_moe_clip_grads", "beam_moe_quantize_mxfp4", "beam_moe_dequantize_mxfp4",
            "beam_moe_linear_mxfp4", "Mxfp4", "beam_moe_workspace_bytes", "beam_moe_status_str",
            "Dims", "BeamMoeError", "load_library")


def __getattr__(name):
    if name in _EXPORTS:
        from . import binding
        globals()[name] = value = getattr(binding, name)  # later uses find it without coming here
        return value
    raise AttributeError(name)
