// rope_kernel.cu -- headwise QK-RMSNorm of Q and K with the rotary position
// embedding in the same pass, and its gradient, on one GB300.
//
// Forward, per head of head_dim = d values at position pos:
//     rinv = 1 / sqrt((1/d) sum x^2 + eps),   n_j = (x_j * gamma_j) * rinv,
//     every pair (a, b) of the first rot values, with its angle's cosine c
//     and sine s from row pos of the table:
//         y_a = n_a c - n_b s,   y_b = n_b c + n_a s,
//     y_j = n_j beyond rot; one rounding to bf16 at the end.
// Backward, with g = the rotation by the opposite angle of dy:
//     dgamma_j = sum over tokens and heads of g_j x_j rinv,
//     dx_j = rinv (u_j - x_j rinv^2 (1/d) sum u x),   u_j = g_j gamma_j.
//
// GB300 mapping: both are bound by HBM (4 and 6 bytes per value; 7 and 15
// flops).  Lane p of a head owns two 16-byte vectors so that both members of
// every pair meet in one thread: vectors p and p + rot/16 while p < rot/16
// (half-split pairs lie rot/2 values apart, interleaved ones side by side),
// two neighbouring vectors of the unrotated rest beyond.  d/16 lanes, rounded
// up to a power of two, hold a head, so the row sums are xor-shuffles inside
// a warp and nothing crosses a warp.  A warp takes one token and U rounds of
// heads at once: 2U independent 16-byte loads per thread in flight, and one
// read of the table row and the gain for all of them.
#include <cuda_runtime.h>

#include <algorithm>

#include "nts_device.cuh"
#include "nts_internal.h"

namespace nts {

namespace {

// kStatusPosition bits of these kernels.
__device__ unsigned int g_rope_status;

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeTensor {
  const __nv_bfloat16* x;
  const __nv_bfloat16* dy;   // backward
  __nv_bfloat16* out;        // y, or dx
  const float* gamma;
  float* rinv;               // forward, [T, nheads] or nullptr
  int64_t ldx, lddy, ldout;  // row strides in elements
  int nheads;
  unsigned chunks;           // warp items per token
};

struct RopeParams {
  RopeTensor ten[2];
  const int64_t* pos;
  const float* table;        // [P, rot]: cosines, then sines
  int64_t P;
  unsigned T;
  int d, rot;
  int pairs;                 // d / 16: lanes in use per head
  int lshift;                // log2 of the lanes per head
  float eps, inv_d;
  float* partial;            // backward: [CTAs, d] sums for the gains' gradients
  unsigned ctas_q;           // backward: CTAs of Q; the others take K
};

// A lane's place: the element offsets of its two vectors, whether it rotates
// and the offsets of its eight cosines (two groups of four).
struct RopeLane {
  int e0, e1;
  int c0, c1;
  bool active, turns;
};

template <bool IL>
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p, int pi) {
  RopeLane l;
  const int hr = p.rot >> 4;   // rotating lanes
  l.active = pi < p.pairs;
  l.turns = pi < hr;
  if (l.turns) {
    l.e0 = 8 * pi;
    l.e1 = 8 * (pi + hr);
    l.c0 = IL ? 4 * pi : 8 * pi;
    l.c1 = IL ? 4 * (pi + hr) : 8 * pi + 4;
  } else {
    l.e0 = p.rot + 16 * (pi - hr);
    l.e1 = l.e0 + 8;
    l.c0 = l.c1 = 0;
  }
  return l;
}

__device__ __forceinline__ void load8(float (&v)[8], const float* a, const float* b) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(a));
  const float4 y = __ldg(reinterpret_cast<const float4*>(b));
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
}

// Rotate the pairs of a (vector at e0) and b (vector at e1) in place.
// Half-split: pair j is (a[j], b[j]).  Interleaved: pairs (a[2j], a[2j+1])
// with the first four angles and (b[2j], b[2j+1]) with the last four.
template <bool IL, bool BACK>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&c)[8],
                                       const float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float& x = IL ? (j < 4 ? a[2 * j] : b[2 * j - 8]) : a[j];
    float& y = IL ? (j < 4 ? a[2 * j + 1] : b[2 * j - 7]) : b[j];
    const float sj = BACK ? -s[j] : s[j];
    const float u = x * c[j] - y * sj;
    y = y * c[j] + x * sj;
    x = u;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                    pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
}

__device__ __forceinline__ uint4 ldg_stream(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

// Sum over the lanes of a head (aligned groups of a power of two of lanes).
__device__ __forceinline__ float head_sum(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The table row of token t: false for a padding row (pos < 0) and for a
// position outside the table, which is reported.
__device__ __forceinline__ bool table_row(const RopeParams& p, unsigned t, int lane,
                                          const float** row) {
  const int64_t pos = __ldg(p.pos + t);
  const bool ok = pos >= 0 && pos < p.P;
  if (pos >= p.P && lane == 0) atomicOr(&g_rope_status, kStatusPosition);
  *row = p.table + (ok ? pos : 0) * p.rot;
  return ok;
}

template <int U, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_forward_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const int hps = 32 >> p.lshift;   // heads per round
  const unsigned per_token = p.ten[0].chunks + p.ten[1].chunks;
  const unsigned items = p.T * per_token;
  const unsigned nwarps = gridDim.x * kRopeWarps;
  grid_dependency_wait();
  allow_dependent_launch();
  for (unsigned item = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); item < items;) {
    const unsigned t = item / per_token;
    unsigned chunk = item - t * per_token;
    const int ti = chunk >= p.ten[0].chunks;
    const RopeTensor& tn = p.ten[ti];
    if (ti) chunk -= p.ten[0].chunks;
    const int h0 = (int)chunk * U * hps + (lane >> p.lshift);

    uint4 x[U][2];
    const __nv_bfloat16* xrow = tn.x + (int64_t)t * tn.ldx;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * hps;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (l.active && h < tn.nheads) {
        x[i][0] = ldg_stream(xrow + (int64_t)h * p.d + l.e0);
        x[i][1] = ldg_stream(xrow + (int64_t)h * p.d + l.e1);
      }
    }
    const float* row;
    const bool ok = table_row(p, t, lane, &row);
    float c[8] = {}, s[8] = {}, g0[8] = {}, g1[8] = {};
    if (l.active) {
      load8(g0, tn.gamma + l.e0, tn.gamma + l.e0 + 4);
      load8(g1, tn.gamma + l.e1, tn.gamma + l.e1 + 4);
    }
    if (l.turns) {
      load8(c, row + l.c0, row + l.c1);
      load8(s, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
    }

    __nv_bfloat16* yrow = tn.out + (int64_t)t * tn.ldout;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * hps;
      float a[8], b[8];
      bf16x8_to_f32(x[i][0], a);
      bf16x8_to_f32(x[i][1], b);
      float ss = 0.f, tt = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(a[j], a[j], ss);
        tt = fmaf(b[j], b[j], tt);
      }
      const float rinv = rsqrtf(fmaf(head_sum(ss + tt, lanes), p.inv_d, p.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = a[j] * g0[j] * rinv;
        b[j] = b[j] * g1[j] * rinv;
      }
      if (l.turns) rotate<IL, false>(a, b, c, s);
      if (l.active && h < tn.nheads) {
        uint4 ya = pack8(a), yb = pack8(b);
        if (!ok) ya = yb = make_uint4(0, 0, 0, 0);
        st_global_v4_stream(yrow + (int64_t)h * p.d + l.e0, ya);
        st_global_v4_stream(yrow + (int64_t)h * p.d + l.e1, yb);
        if (tn.rinv != nullptr && l.e0 == 0)
          tn.rinv[(int64_t)t * tn.nheads + h] = ok ? rinv : 0.f;
      }
    }
    if (items - item <= nwarps) break;   // item + nwarps could pass 2^32
    item += nwarps;
  }
}

// The first ctas_q CTAs walk the items of Q, the others those of K, in a
// fixed order, so a thread keeps its gain and its sums for dgamma in
// registers and the result does not depend on timing.  Every CTA leaves one
// row of partial sums.
template <int U, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_backward_kernel(const RopeParams p) {
  extern __shared__ float red[];   // [warps][d]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const int hps = 32 >> p.lshift;
  const int ti = blockIdx.x >= p.ctas_q;
  const RopeTensor& tn = p.ten[ti];
  const unsigned ctas = ti ? gridDim.x - p.ctas_q : p.ctas_q;
  const unsigned cta = ti ? blockIdx.x - p.ctas_q : blockIdx.x;
  const unsigned items = p.T * tn.chunks;
  const unsigned nwarps = ctas * kRopeWarps;
  grid_dependency_wait();
  allow_dependent_launch();

  float g0[8] = {}, g1[8] = {}, s0[8] = {}, s1[8] = {};
  if (l.active) {
    load8(g0, tn.gamma + l.e0, tn.gamma + l.e0 + 4);
    load8(g1, tn.gamma + l.e1, tn.gamma + l.e1 + 4);
  }
  for (unsigned item = cta * kRopeWarps + warp; item < items;) {
    const unsigned t = item / tn.chunks;
    const unsigned chunk = item - t * tn.chunks;
    const int h0 = (int)chunk * U * hps + (lane >> p.lshift);
    uint4 x[U][2], dy[U][2];
    const __nv_bfloat16* xrow = tn.x + (int64_t)t * tn.ldx;
    const __nv_bfloat16* dyrow = tn.dy + (int64_t)t * tn.lddy;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * hps;
      x[i][0] = x[i][1] = dy[i][0] = dy[i][1] = make_uint4(0, 0, 0, 0);
      if (l.active && h < tn.nheads) {
        x[i][0] = ldg_stream(xrow + (int64_t)h * p.d + l.e0);
        x[i][1] = ldg_stream(xrow + (int64_t)h * p.d + l.e1);
        dy[i][0] = ldg_stream(dyrow + (int64_t)h * p.d + l.e0);
        dy[i][1] = ldg_stream(dyrow + (int64_t)h * p.d + l.e1);
      }
    }
    const float* row;
    const bool ok = table_row(p, t, lane, &row);
    float c[8] = {}, s[8] = {};
    if (l.turns) {
      load8(c, row + l.c0, row + l.c1);
      load8(s, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
    }
    __nv_bfloat16* orow = tn.out + (int64_t)t * tn.ldout;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * hps;
      if (!ok) x[i][0] = x[i][1] = dy[i][0] = dy[i][1] = make_uint4(0, 0, 0, 0);
      float a[8], b[8], u[8], v[8];
      bf16x8_to_f32(x[i][0], a);
      bf16x8_to_f32(x[i][1], b);
      bf16x8_to_f32(dy[i][0], u);
      bf16x8_to_f32(dy[i][1], v);
      if (l.turns) rotate<IL, true>(u, v, c, s);
      float ss = 0.f, ux = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
        ux = fmaf(u[j] * g0[j], a[j], fmaf(v[j] * g1[j], b[j], ux));
      }
      ss = head_sum(ss, lanes);
      ux = head_sum(ux, lanes);
      const float rinv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
      const float k = ux * p.inv_d * rinv * rinv;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s0[j] = fmaf(u[j], a[j] * rinv, s0[j]);
        s1[j] = fmaf(v[j], b[j] * rinv, s1[j]);
        a[j] = rinv * fmaf(-a[j], k, u[j] * g0[j]);
        b[j] = rinv * fmaf(-b[j], k, v[j] * g1[j]);
      }
      if (l.active && h < tn.nheads) {
        st_global_v4_stream(orow + (int64_t)h * p.d + l.e0, pack8(a));
        st_global_v4_stream(orow + (int64_t)h * p.d + l.e1, pack8(b));
      }
    }
    if (items - item <= nwarps) break;
    item += nwarps;
  }

  // the CTA's sums: over the heads of a warp, then over its warps
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o >= lanes) {
        s0[j] += __shfl_xor_sync(0xFFFFFFFFu, s0[j], o);
        s1[j] += __shfl_xor_sync(0xFFFFFFFFu, s1[j], o);
      }
    if (l.active && lane < lanes) {
      red[warp * p.d + l.e0 + j] = s0[j];
      red[warp * p.d + l.e1 + j] = s1[j];
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.d; j += kRopeThreads) {
    float v = 0.f;
    for (int w = 0; w < kRopeWarps; ++w) v += red[w * p.d + j];
    p.partial[(int64_t)blockIdx.x * p.d + j] = v;
  }
}

// dgamma = the sum of the CTAs' rows, in a fixed order: block (32 columns) x
// (32 strided rows), blockIdx.y the tensor.
__global__ void __launch_bounds__(1024) rope_gain_grad_kernel(const float* partial, unsigned nq,
                                                              unsigned n, int d, float* dgamma_q,
                                                              float* dgamma_k) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  const unsigned r0 = blockIdx.y ? nq : 0, r1 = blockIdx.y ? n : nq;
  grid_dependency_wait();
  allow_dependent_launch();
  float v = 0.f;
  if (col < d)
#pragma unroll 8
    for (unsigned r = r0 + threadIdx.y; r < r1; r += 32) v += partial[(int64_t)r * d + col];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < d) (blockIdx.y ? dgamma_k : dgamma_q)[out] = v;
}

using RopeKernel = void (*)(RopeParams);

RopeKernel pick_forward(int u, bool il) {
  switch (u) {
    case 1: return il ? rope_forward_kernel<1, true> : rope_forward_kernel<1, false>;
    default: return il ? rope_forward_kernel<4, true> : rope_forward_kernel<4, false>;
  }
}

RopeKernel pick_backward(int u, bool il) {
  switch (u) {
    case 1: return il ? rope_backward_kernel<1, true> : rope_backward_kernel<1, false>;
    default: return il ? rope_backward_kernel<2, true> : rope_backward_kernel<2, false>;
  }
}

RopeParams common_params(const RopeRequest& rq) {
  RopeParams p = {};
  for (int i = 0; i < 2; ++i) {
    const RopeOperand& o = rq.ten[i];
    p.ten[i].x = static_cast<const __nv_bfloat16*>(o.x);
    p.ten[i].dy = static_cast<const __nv_bfloat16*>(o.dy);
    p.ten[i].out = static_cast<__nv_bfloat16*>(o.out);
    p.ten[i].gamma = o.gamma;
    p.ten[i].rinv = o.rinv;
    p.ten[i].ldx = o.ldx;
    p.ten[i].lddy = o.lddy;
    p.ten[i].ldout = o.ldout;
    p.ten[i].nheads = (int)o.nheads;
  }
  p.pos = rq.pos;
  p.table = rq.table;
  p.P = rq.P;
  p.T = (unsigned)rq.T;
  p.d = (int)rq.head_dim;
  p.rot = (int)rq.rot_dim;
  p.pairs = p.d / 16;
  while ((1 << p.lshift) < p.pairs) ++p.lshift;
  p.eps = rq.eps;
  p.inv_d = 1.0f / (float)p.d;
  return p;
}

// Warp items per token of a tensor when a warp takes u rounds of heads.
unsigned chunks_for(const RopeParams& p, int i, int u) {
  const int heads = u * (32 >> p.lshift);
  return (unsigned)((p.ten[i].nheads + heads - 1) / heads);
}

// Fills in the chunks for u rounds per warp; UNSUPPORTED if the launch's
// items pass 32 bits.
int set_chunks(RopeParams* p, int u) {
  uint64_t items = 0;
  for (int i = 0; i < 2; ++i) {
    p->ten[i].chunks = chunks_for(*p, i, u);
    items += (uint64_t)p->T * p->ten[i].chunks;
  }
  if (items >= (1ull << 32)) return fail(NTS_ERR_UNSUPPORTED, "too many token-heads in one call");
  return NTS_OK;
}

uint64_t warp_items(const RopeParams& p, int u) {
  return (uint64_t)p.T * (chunks_for(p, 0, u) + chunks_for(p, 1, u));
}

template <typename... A>
int launch(void (*kern)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
           A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return fail_cuda(e, "launching the headwise QK-Norm with rotation");
  return NTS_OK;
}

}  // namespace

int launch_rope(const RopeRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  RopeParams p = common_params(rq);
  const int u = warp_items(p, 1) <= (uint64_t)dev.sm_count * 16 ? 1 : 4;
  const int rc = set_chunks(&p, u);
  if (rc != NTS_OK) return rc;
  const uint64_t items = (uint64_t)p.T * (p.ten[0].chunks + p.ten[1].chunks);
  const unsigned grid = (unsigned)std::min<uint64_t>((items + kRopeWarps - 1) / kRopeWarps, 1u << 24);
  log_launch("qknorm_rope", "T=%u heads=%d+%d d=%d rot=%d u=%d grid=%u", p.T, p.ten[0].nheads,
             p.ten[1].nheads, p.d, p.rot, u, grid);
  return launch(pick_forward(u, rq.interleaved), dim3(grid), dim3(kRopeThreads), 0, stream,
                tune.pdl != 0, p);
}

int launch_rope_backward(const RopeRequest& rq, float* dgamma_q, float* dgamma_k,
                         float* workspace, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  RopeParams p = common_params(rq);
  const int u = warp_items(p, 1) <= (uint64_t)dev.sm_count * 16 ? 1 : 2;
  int rc = set_chunks(&p, u);
  if (rc != NTS_OK) return rc;
  const RopeKernel kern = pick_backward(u, rq.interleaved);
  const size_t smem = (size_t)kRopeWarps * p.d * sizeof(float);
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kRopeThreads, smem);
  if (e != cudaSuccess) return fail_cuda(e, "occupancy query for the headwise QK-Norm gradient");
  if (per_sm < 1) return fail(NTS_ERR_UNSUPPORTED, "the gradient kernel does not fit on an SM");
  // CTAs in proportion to the tensors' items, one at least for each
  const uint64_t iq = (uint64_t)p.T * p.ten[0].chunks, ik = (uint64_t)p.T * p.ten[1].chunks;
  const uint64_t nq = (iq + kRopeWarps - 1) / kRopeWarps, nk = (ik + kRopeWarps - 1) / kRopeWarps;
  const uint64_t most = std::min<uint64_t>((uint64_t)per_sm * dev.sm_count, kRopePartials);
  uint64_t gq = nq, gk = nk;
  if (gq + gk > most) {
    gq = std::max<uint64_t>(1, std::min<uint64_t>(most - 1, (most * iq + (iq + ik) / 2) / (iq + ik)));
    gk = std::min<uint64_t>(nk, most - gq);
    gq = std::min<uint64_t>(nq, gq);
  }
  p.ctas_q = (unsigned)gq;
  p.partial = workspace;
  const unsigned grid = (unsigned)(gq + gk);
  log_launch("qknorm_rope_backward", "T=%u heads=%d+%d d=%d rot=%d u=%d grid=%u (%llu for Q)", p.T,
             p.ten[0].nheads, p.ten[1].nheads, p.d, p.rot, u, grid, (unsigned long long)gq);
  rc = launch(kern, dim3(grid), dim3(kRopeThreads), smem, stream, tune.pdl != 0, p);
  if (rc != NTS_OK) return rc;
  return launch(rope_gain_grad_kernel, dim3((p.d + 31) / 32, 2), dim3(32, 32), 0, stream,
                tune.pdl != 0, (const float*)workspace, (unsigned)gq, grid, p.d, dgamma_q,
                dgamma_k);
}

int read_and_clear_rope_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_status, sizeof(v));
  if (e != cudaSuccess) return fail_cuda(e, "reading the rotation status word");
  if (v != 0) e = cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return fail_cuda(e, "clearing the rotation status word");
  *out = v;
  return NTS_OK;
}

}  // namespace nts
