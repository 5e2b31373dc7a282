"""Fused cross-entropy over a large vocabulary for AMD MI355X (gfx950).

The computation lives in ``libvce.so`` (HIP kernels behind the C-ABI declared
in ``include/vce.h``); ``binding`` marshals torch tensors into it.
"""
from .binding import (AdamWState, adamw_state, adamw_step, beam_reorder, beam_step,
                      beam_workspace, beam_workspace_size, ce_backward, ce_backward_shard,  # noqa: F401
                      ce_forward, ce_sample, ce_sample_workspace, ce_sample_workspace_size,
                      ce_forward_backward, ce_forward_shard, ce_merge_shards, gemm_bf16,
                      grad_norm,
                      lce_backward, lce_backward_f32,
                      lce_backward_shard, lce_forward, lce_forward_f32, lce_forward_noalloc,
                      lce_forward_shard,
                      lora_backward, lora_backward_workspace, lora_backward_workspace_size,
                      lora_forward, lora_forward_workspace, lora_forward_workspace_size,
                      lce_workspace, lce_workspace_size, lce_workspace_size_f32, lib,
                      mx_dequantize, mx_logits, mx_quantize, rms_backward, rms_backward_workspace,
                      rms_backward_workspace_size, rms_forward, rms_forward_mx8,
                      shift_targets, strerror, VceError)
