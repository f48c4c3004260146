// block_internal.h -- host-side interfaces of the operators around a QKV
// projection: requests from the C ABI (block_api.cpp) to the launchers, and
// their part of nts_check_status (nts_api.cpp).  Apart from nts_internal.h, whose
// content the measured traffic of the split-H kernels is tied to.
#pragma once

#include "nts_internal.h"

namespace nts {

// A status bit beside kStatusTimeout: a token position outside the rotation table.
constexpr unsigned kStatusPosition = 2u;

// Whether this call is to meet a C++ exception (nts_debug_inject_failure).
bool take_injected_throw();
// CTAs of this kernel that fit an SM (cached per device).
int blocks_per_sm(const void* kernel, int threads, size_t smem, int* out);

// Headwise QK-RMSNorm of Q (ten[0]) and K (ten[1]) with the rotary position
// embedding, and its gradient (rope_kernel.cu).
struct RopeOperand {
  const void* x;
  const void* dy;      // backward
  void* out;           // y, or dx
  const float* gamma;
  float* rinv;         // forward, nullable
  int64_t ldx, lddy, ldout;
  int64_t nheads;
};
struct RopeRequest {
  RopeOperand ten[2];
  const int64_t* pos;
  const float* table;
  int64_t P, T, head_dim, rot_dim;
  int interleaved;
  float eps;
};
// Most CTAs (rows of partial sums in the workspace) of a gradient launch.
constexpr int kRopePartials = 1024;
int launch_rope(const RopeRequest& rq, cudaStream_t stream, const LaunchTuning& tune);
int launch_rope_backward(const RopeRequest& rq, float* dgamma_q, float* dgamma_k,
                         float* workspace, cudaStream_t stream, const LaunchTuning& tune);

// Casts to E4M3 codes with an fp32 scale per 128 values (blockcast_kernel.cu).
enum CastKind { kCastNorm, kCastPlain, kCastTiles, kCastTranspose };
struct BlockcastRequest {
  CastKind kind;
  const void* X;
  const float* gamma;  // kCastNorm, nullable
  uint8_t* codes;
  float* scales;
  float* rinv;         // kCastNorm, nullable
  int64_t T, D;
  float eps;
};
int launch_blockcast(const BlockcastRequest& rq, cudaStream_t stream, const LaunchTuning& tune);

// Block-scaled product of E4M3 operands (gemm_kernel.cu).
struct GemmRequest {
  const void* A;
  const float* a_scales;
  const void* W;
  const float* w_scales;
  int w_rows;          // 128 or 1: rows of W per scale
  void* Y;
  int fp32_out;
  int64_t M, N, K;
};
int launch_gemm(const GemmRequest& rq, cudaStream_t stream, const LaunchTuning& tune);

// The operators around a projection whose kernels this process has launched or
// captured: nts_check_status reads the status words of those alone (a blocking
// copy of ~13 us each), so the other operators' users do not pay for them.
enum StatusUnit { kCastUnit, kGemmUnit, kRopeUnit, kStatusUnits };
void note_launch(StatusUnit unit);
int read_and_clear_cast_status(unsigned* out);
int read_and_clear_gemm_status(unsigned* out);
int read_and_clear_rope_status(unsigned* out);

}  // namespace nts
