"""GB300-native per-token RMS normalization.

Two hot paths, both hand-written sm_103a CUDA behind a C ABI (include/nts.h):

* ``qknorm_rms``      layerwise QK-RMSNorm with split-H scalar partial sums,
                      the shards mapped onto the CTAs of a thread-block cluster
                      (SwiftQK, Eq. (1) and Algorithm 1);
* ``rmsnorm_mxcast``  RMSNorm fused with the MX block cast (E4M3 / E2M1 values,
                      E8M0 scales);
* ``mxnorm_cast``     MXNorm: the RMS estimated from the MX block absmaxes,
                      fused with the same cast (MXNorm card, Fig. 1).

Around the QKV projection between the two:

* ``rmsnorm_blockcast``, ``blockcast``, ``blockcast_t``  E4M3 casts with one
                      fp32 scale per 128 values;
* ``add_rmsnorm_blockcast``, ``add_rmsnorm_backward``  the first of them with the
                      residual's addition in front, and its gradient;
* ``gemm_blockscaled``  the matrix product of such operands on the tensor
                      cores, from single tokens to training batches;
* ``gemv_groupscaled``, ``groupcast``  products of few rows with weights of 4 bits
                      and a scale per group, and the cast of the weights;
* ``qknorm_rope``, ``qknorm_rope_backward``  headwise QK-RMSNorm of Q and K
                      with the rotary position embedding, and its gradient;
* ``qknorm_rope_axes``, ``qknorm_rope_axes_backward``  the same with a position
                      on each of several axes (images, video).

Build the library with ``python -m normalization_token_split_gb300.build``.
"""
from ._lib import NtsError
from .ops import (FMT_E2M1, FMT_E4M3, FMT_NVFP4, MxOut, check_status, codes_row_bytes, mxnorm_cast,
                  mxnorm_cast_host, mxnorm_cast_host_noalloc, mxnorm_correction, mxnorm_postround_cast, qknorm_rms, qknorm_rms_host, qknorm_rms_qk_host,
                  qknorm_rms_fp8, qknorm_rms_heads, qknorm_rms_qk, layernorm_split, qknorm_rms_mxcast,
                  qknorm_rms_qk_mxcast,
                  rmsnorm_mxcast, rmsnorm_mxcast_host, set_missing_tx, set_schedule, set_direct, set_tuning,
                  set_wait_limit_ns, check_nvfp4_scale, set_pdl, set_host_chunks,
                  check_e8m0, inject_failure,
                  AddNormOut, BlockOut, GroupOut, add_rmsnorm_backward, add_rmsnorm_backward_workspace,
                  add_rmsnorm_blockcast, blockcast, blockcast_t, gemm_blockscaled, gemv_groupscaled, groupcast, qknorm_rope,
                  qknorm_rope_axes, qknorm_rope_axes_backward, qknorm_rope_backward,
                  rmsnorm_blockcast, rope_axes, rope_backward_workspace, rope_table)

__all__ = [
    "NtsError", "FMT_E4M3", "FMT_E2M1", "FMT_NVFP4", "MxOut", "qknorm_rms", "qknorm_rms_fp8", "qknorm_rms_heads", "qknorm_rms_qk", "layernorm_split", "qknorm_rms_mxcast", "qknorm_rms_qk_mxcast", "rmsnorm_mxcast", "mxnorm_cast", "mxnorm_postround_cast",
    "mxnorm_correction", "check_status", "codes_row_bytes", "qknorm_rms_host", "qknorm_rms_qk_host",
    "rmsnorm_mxcast_host", "mxnorm_cast_host", "mxnorm_cast_host_noalloc", "set_tuning", "set_wait_limit_ns",
    "set_missing_tx", "set_schedule", "set_direct", "check_nvfp4_scale", "set_pdl", "set_host_chunks", "check_e8m0", "inject_failure",
    "BlockOut", "rmsnorm_blockcast", "blockcast", "blockcast_t", "gemm_blockscaled", "qknorm_rope",
    "qknorm_rope_backward", "rope_backward_workspace", "rope_table", "rope_axes", "qknorm_rope_axes",
    "qknorm_rope_axes_backward", "AddNormOut", "add_rmsnorm_blockcast", "add_rmsnorm_backward",
    "add_rmsnorm_backward_workspace", "GroupOut", "groupcast", "gemv_groupscaled",
]
