// block_api.cpp -- the C ABI of the operators around the QKV projection:
// argument checks of the block-128 casts, the block-scaled product and the
// headwise QK-RMSNorm with rotation, and the rotation table on the host.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <exception>
#include <new>

#include "block_internal.h"
#include "nts.h"

using namespace nts;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxIndex = int64_t(1) << 31;

int check_eps(float eps) {
  if (!(eps > 0.f) || !std::isfinite(eps))
    return fail(NTS_ERR_INVALID_ARG, "eps must be positive and finite");
  return NTS_OK;
}

// The checks of a rotation call that involve no tensor.
int check_rope_shape(int64_t P, int64_t T, int64_t nheads_q, int64_t nheads_k, int64_t head_dim,
                     int64_t rot_dim, float eps) {
  if (T < 0) return fail(NTS_ERR_INVALID_ARG, "T must be >= 0, got %lld", (long long)T);
  if (P <= 0) return fail(NTS_ERR_INVALID_ARG, "the table must have rows, got P = %lld", (long long)P);
  if (nheads_q <= 0 || nheads_k <= 0)
    return fail(NTS_ERR_INVALID_ARG, "Q and K must have heads, got %lld and %lld",
                (long long)nheads_q, (long long)nheads_k);
  if (head_dim <= 0) return fail(NTS_ERR_INVALID_ARG, "head_dim must be > 0");
  if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 2 != 0)
    return fail(NTS_ERR_INVALID_ARG, "rot_dim (%lld) must be even and in [2, head_dim]",
                (long long)rot_dim);
  const int rc = check_eps(eps);
  if (rc != NTS_OK) return rc;
  if (head_dim % 16 != 0 || head_dim > 512)
    return fail(NTS_ERR_UNSUPPORTED, "head_dim (%lld) must be a multiple of 16 up to 512",
                (long long)head_dim);
  if (rot_dim % 16 != 0)
    return fail(NTS_ERR_UNSUPPORTED, "rot_dim (%lld) must be a multiple of 16", (long long)rot_dim);
  if (T >= kMaxIndex || nheads_q > 65536 || nheads_k > 65536)
    return fail(NTS_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens or 65536 heads");
  return NTS_OK;
}

// A [T, nheads * head_dim] bf16 operand with a row stride.
int check_rows(const char* name, const void* p, int64_t ld, int64_t width, int64_t T) {
  if (T > 0 && p == nullptr) return fail(NTS_ERR_INVALID_ARG, "%s must be non-NULL", name);
  if (ld < width)
    return fail(NTS_ERR_INVALID_ARG, "%s: row stride %lld below the row's %lld values", name,
                (long long)ld, (long long)width);
  if (!aligned(p, 16) || ld % 8 != 0)
    return fail(NTS_ERR_UNSUPPORTED, "%s: rows must start on 16-byte boundaries", name);
  return NTS_OK;
}

int check_vec(const char* name, const float* p, int64_t T, size_t align) {
  if (T > 0 && p == nullptr) return fail(NTS_ERR_INVALID_ARG, "%s must be non-NULL", name);
  if (!aligned(p, align))
    return fail(NTS_ERR_UNSUPPORTED, "%s must be %d-byte aligned", name, (int)align);
  return NTS_OK;
}

int check_table(const int64_t* positions, const float* table, int64_t T) {
  if (T > 0 && positions == nullptr)
    return fail(NTS_ERR_INVALID_ARG, "positions must be non-NULL");
  if (!aligned(positions, 8)) return fail(NTS_ERR_UNSUPPORTED, "positions must be 8-byte aligned");
  return check_vec("table", table, T, 16);
}

int check_cast(const void* X, const uint8_t* codes, const float* scales, int64_t T, int64_t D) {
  if (T < 0) return fail(NTS_ERR_INVALID_ARG, "T must be >= 0, got %lld", (long long)T);
  if (D <= 0) return fail(NTS_ERR_INVALID_ARG, "D must be > 0, got %lld", (long long)D);
  if (T > 0 && (X == nullptr || codes == nullptr || scales == nullptr))
    return fail(NTS_ERR_INVALID_ARG, "X, codes and scales must be non-NULL");
  if (D % 16 != 0)
    return fail(NTS_ERR_UNSUPPORTED, "D (%lld) must be a multiple of 16", (long long)D);
  if (T >= kMaxIndex || D >= kMaxIndex)
    return fail(NTS_ERR_UNSUPPORTED, "T and D must stay below 2^31");
  if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(NTS_ERR_UNSUPPORTED, "X and codes must be 16-byte aligned, scales 4-byte");
  return NTS_OK;
}

// Runs a launch; what it throws (the host out of memory, a lock that fails) ends
// as a status, not in the caller's C frames.
template <typename F>
int guarded(F f) noexcept {
  try {
    if (take_injected_throw()) throw std::bad_alloc();
    return f();
  } catch (const std::exception& e) {
    return fail(NTS_ERR_CUDA, "host failure in a launch: %s", e.what());
  } catch (...) {
    return fail(NTS_ERR_CUDA, "host failure in a launch");
  }
}

int cast(const BlockcastRequest& rq, void* stream) {
  return guarded(
      [&] { return launch_blockcast(rq, static_cast<cudaStream_t>(stream), current_tuning()); });
}

}  // namespace

extern "C" {

int nts_rope_table_host(int64_t P, int64_t rot_dim, double base, float* table_host) {
  if (P < 0) return fail(NTS_ERR_INVALID_ARG, "P must be >= 0, got %lld", (long long)P);
  if (rot_dim <= 0 || rot_dim % 2 != 0)
    return fail(NTS_ERR_INVALID_ARG, "rot_dim (%lld) must be positive and even", (long long)rot_dim);
  if (!(base > 0.0) || !std::isfinite(base))
    return fail(NTS_ERR_INVALID_ARG, "base must be positive and finite");
  if (P > 0 && table_host == nullptr)
    return fail(NTS_ERR_INVALID_ARG, "table_host must be non-NULL");
  const int64_t half = rot_dim / 2;
  for (int64_t i = 0; i < half; ++i) {
    const double w = std::pow(base, -2.0 * (double)i / (double)rot_dim);
    for (int64_t pos = 0; pos < P; ++pos) {
      float* row = table_host + pos * rot_dim;
      row[i] = (float)std::cos((double)pos * w);
      row[half + i] = (float)std::sin((double)pos * w);
    }
  }
  return NTS_OK;
}

int nts_qknorm_rope(const void* Q_dev, int64_t ldq, const float* gamma_q_dev, void* Yq_dev,
                    int64_t ldyq, float* rinv_q_dev, const void* K_dev, int64_t ldk,
                    const float* gamma_k_dev, void* Yk_dev, int64_t ldyk, float* rinv_k_dev,
                    const int64_t* positions_dev, const float* table_dev, int64_t P, int64_t T,
                    int64_t nheads_q, int64_t nheads_k, int64_t head_dim, int64_t rot_dim,
                    int interleaved, float eps, void* stream) {
  int rc = check_rope_shape(P, T, nheads_q, nheads_k, head_dim, rot_dim, eps);
  const int64_t wq = nheads_q * head_dim, wk = nheads_k * head_dim;
  if (rc == NTS_OK) rc = check_rows("Q", Q_dev, ldq, wq, T);
  if (rc == NTS_OK) rc = check_rows("K", K_dev, ldk, wk, T);
  if (rc == NTS_OK) rc = check_rows("Yq", Yq_dev, ldyq, wq, T);
  if (rc == NTS_OK) rc = check_rows("Yk", Yk_dev, ldyk, wk, T);
  if (rc == NTS_OK) rc = check_vec("gamma_q", gamma_q_dev, T, 16);
  if (rc == NTS_OK) rc = check_vec("gamma_k", gamma_k_dev, T, 16);
  if (rc == NTS_OK) rc = check_table(positions_dev, table_dev, T);
  if (rc != NTS_OK) return rc;
  if (!aligned(rinv_q_dev, 4) || !aligned(rinv_k_dev, 4))
    return fail(NTS_ERR_UNSUPPORTED, "rinv must be 4-byte aligned");
  if (T == 0) return NTS_OK;
  const RopeRequest rq{{{Q_dev, nullptr, Yq_dev, gamma_q_dev, rinv_q_dev, ldq, 0, ldyq, nheads_q},
                        {K_dev, nullptr, Yk_dev, gamma_k_dev, rinv_k_dev, ldk, 0, ldyk, nheads_k}},
                       positions_dev, table_dev, P, T, head_dim, rot_dim, interleaved != 0, eps};
  return guarded(
      [&] { return launch_rope(rq, static_cast<cudaStream_t>(stream), current_tuning()); });
}

int nts_qknorm_rope_backward_workspace(int64_t head_dim, int64_t* bytes_out) {
  if (bytes_out == nullptr) return fail(NTS_ERR_INVALID_ARG, "bytes_out is NULL");
  if (head_dim <= 0) return fail(NTS_ERR_INVALID_ARG, "head_dim must be > 0");
  *bytes_out = (int64_t)kRopePartials * head_dim * (int64_t)sizeof(float);
  return NTS_OK;
}

int nts_qknorm_rope_backward(const void* dYq_dev, int64_t lddyq, const void* dYk_dev,
                             int64_t lddyk, const void* Q_dev, int64_t ldq,
                             const float* gamma_q_dev, const void* K_dev, int64_t ldk,
                             const float* gamma_k_dev, const int64_t* positions_dev,
                             const float* table_dev, int64_t P, void* dQ_dev, int64_t lddq,
                             void* dK_dev, int64_t lddk, float* dgamma_q_dev, float* dgamma_k_dev,
                             void* workspace_dev, int64_t workspace_bytes, int64_t T,
                             int64_t nheads_q, int64_t nheads_k, int64_t head_dim,
                             int64_t rot_dim, int interleaved, float eps, void* stream) {
  int rc = check_rope_shape(P, T, nheads_q, nheads_k, head_dim, rot_dim, eps);
  const int64_t wq = nheads_q * head_dim, wk = nheads_k * head_dim;
  if (rc == NTS_OK) rc = check_rows("dYq", dYq_dev, lddyq, wq, T);
  if (rc == NTS_OK) rc = check_rows("dYk", dYk_dev, lddyk, wk, T);
  if (rc == NTS_OK) rc = check_rows("Q", Q_dev, ldq, wq, T);
  if (rc == NTS_OK) rc = check_rows("K", K_dev, ldk, wk, T);
  if (rc == NTS_OK) rc = check_rows("dQ", dQ_dev, lddq, wq, T);
  if (rc == NTS_OK) rc = check_rows("dK", dK_dev, lddk, wk, T);
  if (rc == NTS_OK) rc = check_vec("gamma_q", gamma_q_dev, T, 16);
  if (rc == NTS_OK) rc = check_vec("gamma_k", gamma_k_dev, T, 16);
  if (rc == NTS_OK) rc = check_table(positions_dev, table_dev, T);
  if (rc == NTS_OK && eps < FLT_MIN)   // rinv^2 of a row of zeros would overflow
    rc = fail(NTS_ERR_UNSUPPORTED, "eps must be at least 2^-126 for the gradient");
  // the gains' gradients are written for an empty batch too
  if (rc == NTS_OK) rc = check_vec("dgamma_q", dgamma_q_dev, 1, 4);
  if (rc == NTS_OK) rc = check_vec("dgamma_k", dgamma_k_dev, 1, 4);
  if (rc != NTS_OK) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(dgamma_q_dev, 0, head_dim * sizeof(float), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dgamma_k_dev, 0, head_dim * sizeof(float), s);
    return e == cudaSuccess ? NTS_OK : fail_cuda(e, "clearing the gains' gradients");
  }
  int64_t need = 0;
  nts_qknorm_rope_backward_workspace(head_dim, &need);
  if (workspace_dev == nullptr || workspace_bytes < need)
    return fail(NTS_ERR_INVALID_ARG, "the workspace needs %lld bytes, got %lld", (long long)need,
                (long long)(workspace_dev == nullptr ? 0 : workspace_bytes));
  if (!aligned(workspace_dev, 4))
    return fail(NTS_ERR_UNSUPPORTED, "the workspace must be 4-byte aligned");
  const RopeRequest rq{{{Q_dev, dYq_dev, dQ_dev, gamma_q_dev, nullptr, ldq, lddyq, lddq, nheads_q},
                        {K_dev, dYk_dev, dK_dev, gamma_k_dev, nullptr, ldk, lddyk, lddk, nheads_k}},
                       positions_dev, table_dev, P, T, head_dim, rot_dim, interleaved != 0, eps};
  return guarded([&] {
    return launch_rope_backward(rq, dgamma_q_dev, dgamma_k_dev, static_cast<float*>(workspace_dev),
                                s, current_tuning());
  });
}

int nts_rmsnorm_blockcast(const void* X_dev, const float* gamma_dev, uint8_t* codes_dev,
                          float* scales_dev, float* rinv_dev, int64_t T, int64_t D, float eps,
                          void* stream) {
  int rc = check_cast(X_dev, codes_dev, scales_dev, T, D);
  if (rc == NTS_OK) rc = check_eps(eps);
  if (rc != NTS_OK) return rc;
  if (D > 32768) return fail(NTS_ERR_UNSUPPORTED, "D (%lld) exceeds 32768", (long long)D);
  if (!aligned(gamma_dev, 16) || !aligned(rinv_dev, 4))
    return fail(NTS_ERR_UNSUPPORTED, "gamma must be 16-byte aligned, rinv 4-byte");
  if (T == 0) return NTS_OK;
  const BlockcastRequest rq{kCastNorm, X_dev, gamma_dev, codes_dev, scales_dev, rinv_dev, T, D, eps};
  return cast(rq, stream);
}

int nts_blockcast(const void* X_dev, uint8_t* codes_dev, float* scales_dev, int64_t T, int64_t D,
                  int block_rows, void* stream) {
  if (block_rows != 1 && block_rows != 128)
    return fail(NTS_ERR_INVALID_ARG, "block_rows must be 1 or 128, got %d", block_rows);
  const int rc = check_cast(X_dev, codes_dev, scales_dev, T, D);
  if (rc != NTS_OK) return rc;
  if (T == 0) return NTS_OK;
  const BlockcastRequest rq{block_rows == 1 ? kCastPlain : kCastTiles, X_dev, nullptr, codes_dev,
                            scales_dev, nullptr, T, D, 0.f};
  return cast(rq, stream);
}

int nts_blockcast_t(const void* X_dev, uint8_t* codes_dev, float* scales_dev, int64_t T, int64_t D,
                    void* stream) {
  const int rc = check_cast(X_dev, codes_dev, scales_dev, T, D);
  if (rc != NTS_OK) return rc;
  if (T == 0) return NTS_OK;
  const BlockcastRequest rq{kCastTranspose, X_dev, nullptr, codes_dev, scales_dev, nullptr, T, D,
                            0.f};
  return cast(rq, stream);
}

int nts_gemm_blockscaled(const uint8_t* A_codes_dev, const float* a_scales_dev,
                         const uint8_t* W_codes_dev, const float* w_scales_dev, int w_block_rows,
                         void* Y_dev, int out_type, int64_t M, int64_t N, int64_t K, void* stream) {
  if (w_block_rows != 1 && w_block_rows != 128)
    return fail(NTS_ERR_INVALID_ARG, "w_block_rows must be 1 or 128, got %d", w_block_rows);
  if (out_type != NTS_OUT_BF16 && out_type != NTS_OUT_FP32)
    return fail(NTS_ERR_INVALID_ARG, "unknown output type %d", out_type);
  if (M < 0) return fail(NTS_ERR_INVALID_ARG, "M must be >= 0, got %lld", (long long)M);
  if (N <= 0 || K <= 0)
    return fail(NTS_ERR_INVALID_ARG, "N and K must be > 0, got %lld and %lld", (long long)N,
                (long long)K);
  if (M > 0 && (A_codes_dev == nullptr || a_scales_dev == nullptr || W_codes_dev == nullptr ||
                w_scales_dev == nullptr || Y_dev == nullptr))
    return fail(NTS_ERR_INVALID_ARG, "operands, scales and Y must be non-NULL");
  if (K % 16 != 0)
    return fail(NTS_ERR_UNSUPPORTED, "K (%lld) must be a multiple of 16", (long long)K);
  const int64_t most = kMaxIndex - 256;   // tiles end inside 32-bit coordinates
  if (M >= most || N >= most || K >= most)
    return fail(NTS_ERR_UNSUPPORTED, "M, N and K must stay below 2^31 - 256");
  if (!aligned(A_codes_dev, 16) || !aligned(W_codes_dev, 16) || !aligned(a_scales_dev, 4) ||
      !aligned(w_scales_dev, 4) || !aligned(Y_dev, 16))
    return fail(NTS_ERR_UNSUPPORTED, "codes and Y must be 16-byte aligned, scales 4-byte");
  if (M == 0) return NTS_OK;
  const GemmRequest rq{A_codes_dev, a_scales_dev, W_codes_dev, w_scales_dev, w_block_rows, Y_dev,
                       out_type == NTS_OUT_FP32, M, N, K};
  return guarded(
      [&] { return launch_gemm(rq, static_cast<cudaStream_t>(stream), current_tuning()); });
}

}  // extern "C"
