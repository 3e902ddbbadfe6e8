"""MI355X (gfx950) Kimi Delta Attention chunked forward pass.

``fwd(...)`` runs the forward pass: a thin binding over the C-ABI library
``libkda.so`` (declared in ``include/kda.h``), whose hand-written HIP kernels
run every step of it.  Beside it stand the operators of the layer around it:
``short_conv`` (the short causal convolution in front, with the L2 norm of q
and k), ``ssm_fwd`` (the selective state space scan), ``delta_fwd`` (the delta
rule with one decay per head), ``gated_norm`` (the norm of the heads with
their gate) and ``residual_norm`` (the residual update with the norms after
and before a block); and those of the attention layers that a hybrid model
puts between: ``qk_norm_rotary``, ``append_kv`` and ``paged_attention`` over a
paged cache.  ``synth`` draws the seeded synthetic inputs of the named
workloads.
"""
from ._lib import KdaLibraryMissing
from .api import KdaArgumentError, KdaError, auto_segment_chunks, fwd, fwd_kernel
from .attention import append_kv, paged_attention, qk_norm_rotary
from .layer import delta_fwd, gated_norm, residual_norm, short_conv, ssm_fwd

__all__ = ["fwd", "fwd_kernel", "auto_segment_chunks", "short_conv", "ssm_fwd", "gated_norm",
           "residual_norm", "delta_fwd", "qk_norm_rotary", "append_kv", "paged_attention", "KdaError",
           "KdaArgumentError", "KdaLibraryMissing"]
