"""MI355X-native (gfx950) selective scan.

The computation lives in libsss.so (hand-written HIP kernels behind the C ABI of
include/sss.h); this package is its thin Python binding:

  * ``selective_scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None)`` -> (y, h_last);
    keywords ``delta_bias``, ``delta_softplus``, ``exact_zoh`` and ``layout="bdl"``
    (channel-major operands) select the options of ``selective_scan_fwd_ex``
  * ``selective_scan_bwd(x, delta, A, B, C, D, z, h0, dy=..., dh_last=None)`` -> gradients;
    ``states=`` on both calls keeps the forward's segment entering states for the gradients
    (``selective_scan_states_size`` bytes: selective_scan_fwd_save / selective_scan_bwd_saved)
  * ``selective_state_update(x, delta, A, B, C, D=None, z=None, state=...)`` -> y (one
    decode step; ``state`` is updated in place)
  * ``causal_conv1d_fwd(x, weight, bias=None, silu=False)`` -> out (the conv front end)
  * ``causal_conv1d_packed_fwd`` / ``selective_scan_packed_fwd``: the convolution and the scan
    over packed prompts of any lengths (``cu_seqlens``), each sequence's history or state in a
    cache slot; ``causal_conv1d_update`` / ``selective_state_update_slots``: one token of each
    request on the same caches
  * ``causal_conv1d_bwd(x, weight, bias, dout=..., silu=False)`` -> the convolution's gradients
  * ``rms_norm_gated_fwd`` / ``rms_norm_gated_bwd``: the norm after the scan, fused with the gate;
    ``rms_norm_residual_fwd`` / ``rms_norm_residual_bwd``: the residual addition between blocks,
    fused with a norm of the block's output, its scale and the next block's norm
  * ``layer_norm_fwd`` / ``layer_norm_bwd``: the layer norm over rows or groups of channels (heads), alone or
    after the residual addition
  * ``linear_attention_packed_fwd`` / ``linear_attention_update_slots``: linear attention with a decay for
    each head (the scan's head form), over packed prompts and for single tokens, its states in cache
    slots; ``linear_attention_packed_bwd``: its gradients
  * ``elementwise_scan(x, A, B, C, h0=None)`` -> (y, h_last)
  * ``*_workspace_size``, raw-pointer variants ``*_raw`` and ``status_string``.

``inputs`` holds the seeded synthetic workload generators.
"""
from ._lib import (EXPORTED, LIB_PATH, SSSError, SSS_BF16, SSS_DELTA_SOFTPLUS, SSS_EXACT_ZOH, SSS_F32, SSS_LAYOUT_BDL,
                   SSS_NORM_BEFORE_GATE,
                   causal_conv1d_fwd, causal_conv1d_fwd_raw, elementwise_scan, elementwise_scan_raw,
                   selective_scan_bwd, selective_scan_bwd_raw, selective_scan_bwd_ex_raw, selective_scan_bwd_workspace_size,
                   selective_scan_fwd_ex_raw, selective_scan_fwd_noalloc_raw, selective_scan_states_size,
                   selective_scan_fwd_save_raw, selective_scan_bwd_saved_raw,
                   elementwise_scan_workspace_size, load, selective_scan_fwd, selective_scan_fwd_raw,
                   selective_scan_fwd_workspace_size, selective_scan_fwd_ex_workspace_size,
                   selective_state_update, selective_state_update_raw,
                   status_string)
from ._block import (layer_norm_bwd, layer_norm_bwd_workspace_size, layer_norm_fwd, causal_conv1d_bwd, causal_conv1d_bwd_workspace_size, causal_conv1d_packed_fwd,
                     causal_conv1d_update, rms_norm_gated_bwd, rms_norm_gated_bwd_workspace_size, rms_norm_gated_fwd,
                     rms_norm_residual_bwd, rms_norm_residual_bwd_workspace_size, rms_norm_residual_fwd,
                     selective_scan_packed_fwd, selective_scan_packed_fwd_workspace_size,
                     selective_state_update_slots)
from ._linear import (linear_attention_packed_bwd, linear_attention_packed_bwd_workspace_size,
                      linear_attention_packed_fwd, linear_attention_packed_fwd_workspace_size,
                      linear_attention_update_slots)

__all__ = ["causal_conv1d_packed_fwd", "causal_conv1d_update", "causal_conv1d_bwd", "causal_conv1d_bwd_workspace_size",
           "selective_scan_packed_fwd", "selective_scan_packed_fwd_workspace_size", "selective_state_update_slots",
           "rms_norm_gated_fwd", "rms_norm_gated_bwd", "rms_norm_gated_bwd_workspace_size", "rms_norm_residual_fwd",
           "rms_norm_residual_bwd", "rms_norm_residual_bwd_workspace_size", "SSS_NORM_BEFORE_GATE",
           "selective_scan_fwd", "selective_scan_bwd", "selective_scan_bwd_raw", "selective_scan_bwd_ex_raw", "selective_scan_bwd_workspace_size",
           "selective_state_update", "causal_conv1d_fwd", "causal_conv1d_fwd_raw", "selective_state_update_raw", "elementwise_scan",
           "selective_scan_fwd_workspace_size",
           "elementwise_scan_workspace_size", "selective_scan_fwd_raw", "elementwise_scan_raw", "status_string",
           "SSSError", "SSS_F32", "SSS_BF16", "SSS_EXACT_ZOH", "SSS_DELTA_SOFTPLUS", "SSS_LAYOUT_BDL",
           "selective_scan_fwd_ex_workspace_size", "selective_scan_fwd_ex_raw", "selective_scan_fwd_noalloc_raw",
           "selective_scan_states_size", "selective_scan_fwd_save_raw", "selective_scan_bwd_saved_raw",
           "linear_attention_packed_fwd", "linear_attention_packed_fwd_workspace_size", "linear_attention_update_slots",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_size",
           "linear_attention_packed_bwd", "linear_attention_packed_bwd_workspace_size",
           "LIB_PATH", "EXPORTED", "load"]
