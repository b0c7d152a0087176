"""MI355X (gfx950) top-k routed MoE SwiGLU FFN: forward and backward.

Hand-written HIP kernels behind a C ABI (include/moe_ffn.h, built into
libmoe_ffn.so): stable counting-sort expert permute, bf16-MFMA grouped
GEMMs over [W1|W3] with a fused silu(g)*u epilogue and over W2, and a
deterministic unpermute/combine, and the layer's backward; and, around it,
the layer norm with its backward and the Muon step on the weights'
gradients; and a model's two ends: embedding lookup, and cross entropy and
distillation over a vocabulary, each with its gradient.  This package is the
Python binding: torch supplies device memory and streams, nothing else.
"""
from ._lib import (MoeError, alloc_workspace, backward, backward_workspace_layout,  # noqa: F401
                   cross_entropy, cross_entropy_backward, cross_entropy_workspace_size,
                   device_clock_sample, device_error, distillation, distillation_backward,
                   distillation_workspace_size, embedding, embedding_backward,
                   embedding_backward_workspace_size, engine_clock_ghz, expert_permute, forward,
                   forward_noalloc, forward_routed, forward_save_gu, layer_norm, layer_norm_backward,
                   layer_norm_backward_workspace_size, lib,
                   muon_step, newton_schulz, newton_schulz_workspace_size, router_topk, status_string,
                   stream_read, tile_rows,
                   workspace_layout, workspace_size, EXPORTS, LIB_PATH, NOALLOC_SCRATCH_BYTES, NS_COEFFS)
