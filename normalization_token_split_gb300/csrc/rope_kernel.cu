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
// a warp and nothing crosses a warp.  A warp takes a few heads of one token at
// a time, with one read of the table row and the gain for all of them: that read
// and the position's latency are what a round of heads costs beside its data.
//
// Measured (us, back to back in a graph; of the copy's rate): forward [8192, 40
// + 40 heads of 128] 53.4, 0.94; [1237, 20 + 4 heads of 96, 64 turned] 5.8; one
// token of 32 + 32 heads 1.9 (an empty launch 1.0 to 1.5).  Backward [8192, 40 +
// 40] 90.2, 0.83: two values in for each out, and 127 registers leave 16 warps
// an SM to cover the ring's latencies; [333, 32 + 8 heads of 64] 5.6.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_internal.h"
#include "nts_device.cuh"

namespace nts {

namespace {

// kStatusPosition and kStatusTimeout bits of these kernels.
__device__ unsigned int g_rope_status;

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

// Warp items per SM up to which nothing is staged: a launch that small is over
// before a ring of copies pays (32 + 8 heads of 128, us in a graph: forward, T =
// 120: 2.1 direct, 3.6 by the ring; 300: 3.7 both; backward, T = 30: 4.6 and
// 5.3; 60: 5.9 and 5.2, 120: 7.5 and 6.8).
constexpr int kDirectItems = 16, kBackwardDirectItems = 3;
// Partial sums up to which the last CTA of an eager backward call adds them up:
// one CTA's loads take longer than a second launch from there on ([240, 32 + 8
// heads of 128], 38912 sums: 14.6 us a call by one CTA, 9.9 by a launch).
constexpr int kFusedSums = 1 << 15;
// Rounds of heads per ring stage, and stages per warp.  Fewer rounds pay the
// token's reads more often ([4096, 32 + 8 heads of 128], us: forward 27.5 with one
// round, 20.0 with two, 16.4 with four; backward 34.8 and 30.2); more rounds and
// more stages measured no faster.
constexpr int kForwardRounds = 4, kForwardStages = 2;
constexpr int kBackwardRounds = 2, kBackwardStages = 2;

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
  int heads;                 // heads per item
  int stages;                // ring kernels
  uint32_t stage_bytes;
  uint64_t wait_limit_ns;
  uint32_t missing_tx;       // test hook: bytes expected on a first stage but never sent
  float* partial;            // backward: [CTAs, d] sums for the gains' gradients
  unsigned ctas_q;           // backward: CTAs of Q; the others take K
  float* dgamma[2];          // backward
  unsigned int* sched;       // backward: zeroed counter pair of the launch (its second
                             // word counts CTAs), or nullptr: a launch of its own sums
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

// A lane's two vectors of a head (at e0 and e1) as pairs of fp32 lanes.
struct RopeValues {
  uint64_t a[4], b[4];
};

__device__ __forceinline__ void unpack8(uint64_t (&f)[4], const uint4& v) {
  f[0] = bf16x2_to_f2(v.x);
  f[1] = bf16x2_to_f2(v.y);
  f[2] = bf16x2_to_f2(v.z);
  f[3] = bf16x2_to_f2(v.w);
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
  return make_uint4(pack_bf16x2_rn(f2_lo(v[0]), f2_hi(v[0])),
                    pack_bf16x2_rn(f2_lo(v[1]), f2_hi(v[1])),
                    pack_bf16x2_rn(f2_lo(v[2]), f2_hi(v[2])),
                    pack_bf16x2_rn(f2_lo(v[3]), f2_hi(v[3])));
}

__device__ __forceinline__ uint64_t f2_swap(uint64_t v) { return f2(f2_hi(v), f2_lo(v)); }

// The lane's gains (zeros in idle lanes).
__device__ __forceinline__ RopeValues load_gain(const RopeTensor& tn, const RopeLane& l) {
  RopeValues g = {};
  if (l.active) {
    float v[8];
    load8(v, tn.gamma + l.e0, tn.gamma + l.e0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) g.a[i] = f2(v[2 * i], v[2 * i + 1]);
    load8(v, tn.gamma + l.e1, tn.gamma + l.e1 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) g.b[i] = f2(v[2 * i], v[2 * i + 1]);
  }
  return g;
}

// The factors of the rotated pairs, two values at a time: with o the other
// members of the pairs, y = x * same + o * other.  o is the lane's other
// vector (half-split) or x with its halves exchanged (interleaved).
struct RopeFactors {
  RopeValues same, other;
};

// Factors with the gains multiplied in: y_a = a (g_a c) - b (g_b s),
// y_b = b (g_b c) + a (g_a s).  Lanes that do not turn: same = gain.
template <bool IL>
__device__ __forceinline__ RopeFactors gain_factors(const RopeLane& l, const float (&g0)[8],
                                                    const float (&g1)[8], const float (&c)[8],
                                                    const float (&s)[8]) {
  RopeFactors f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 2 * i;
    if (IL) {
      f.same.a[i] = f2(g0[j] * c[i], g0[j + 1] * c[i]);
      f.same.b[i] = f2(g1[j] * c[4 + i], g1[j + 1] * c[4 + i]);
      f.other.a[i] = f2(-g0[j + 1] * s[i], g0[j] * s[i]);
      f.other.b[i] = f2(-g1[j + 1] * s[4 + i], g1[j] * s[4 + i]);
    } else {
      f.same.a[i] = f2(g0[j] * c[j], g0[j + 1] * c[j + 1]);
      f.same.b[i] = f2(g1[j] * c[j], g1[j + 1] * c[j + 1]);
      f.other.a[i] = f2(-g1[j] * s[j], -g1[j + 1] * s[j + 1]);
      f.other.b[i] = f2(g0[j] * s[j], g0[j + 1] * s[j + 1]);
    }
    if (!l.turns) {
      f.same.a[i] = f2(g0[j], g0[j + 1]);
      f.same.b[i] = f2(g1[j], g1[j + 1]);
    }
  }
  return f;
}

// The rotation by the opposite angles, in place: a' = a c + b s, b' = b c - a s.
template <bool IL>
__device__ __forceinline__ void rotate_back(RopeValues& v, const float (&c)[8],
                                            const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 2 * i;
    if (IL) {
      v.a[i] = f2_fma(f2_swap(v.a[i]), f2(s[i], -s[i]), f2_mul(v.a[i], f2(c[i], c[i])));
      v.b[i] = f2_fma(f2_swap(v.b[i]), f2(s[4 + i], -s[4 + i]),
                      f2_mul(v.b[i], f2(c[4 + i], c[4 + i])));
    } else {
      const uint64_t cc = f2(c[j], c[j + 1]), ss = f2(s[j], s[j + 1]);
      const uint64_t a = f2_fma(v.b[i], ss, f2_mul(v.a[i], cc));
      v.b[i] = f2_fma(v.a[i], f2(-s[j], -s[j + 1]), f2_mul(v.b[i], cc));
      v.a[i] = a;
    }
  }
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
// position outside the table, which is reported.  Such a row's outputs are set to
// zero, not computed: neither row 0 of the table nor the gain has to be finite.
__device__ __forceinline__ bool table_row(const RopeParams& p, unsigned t, int lane,
                                          const float** row) {
  const int64_t pos = __ldg(p.pos + t);
  const bool ok = pos >= 0 && pos < p.P;
  if (pos >= p.P && lane == 0) atomicOr(&g_rope_status, kStatusPosition);
  *row = p.table + (ok ? pos : 0) * p.rot;
  return ok;
}

// Walks a warp's items, `step` apart, without a division per item: item =
// t * per_token + chunk.
struct RopeCursor {
  unsigned t, chunk;
  unsigned step_t, step_c, per_token;
  __device__ __forceinline__ RopeCursor(unsigned first, unsigned step, unsigned per)
      : t(first / per), chunk(first % per), step_t(step / per), step_c(step % per), per_token(per) {}
  __device__ __forceinline__ void advance() {
    t += step_t;
    chunk += step_c;
    if (chunk >= per_token) {
      chunk -= per_token;
      ++t;
    }
  }
};

// A warp's item: heads [h0, h0 + heads) of token t, of one tensor.
struct RopeItem {
  unsigned t;
  int h0, heads;
};

__device__ __forceinline__ RopeItem rope_item(const RopeTensor& tn, unsigned t, unsigned chunk,
                                              int heads) {
  const int h0 = (int)chunk * heads;
  return {t, h0, min(heads, tn.nheads - h0)};
}

// One round of the forward pass: x0 and x1 are the lane's vectors of its head,
// y in their place afterwards.  The gain is part of the factors, so a value
// costs two products, a sum and the product with rinv.
template <bool IL>
__device__ __forceinline__ void forward_head(const RopeParams& p, const RopeLane& l, int lanes,
                                             uint4& x0, uint4& x1, const RopeFactors& f, bool ok,
                                             float* rinv_out) {
  RopeValues x, y;
  unpack8(x.a, x0);
  unpack8(x.b, x1);
  uint64_t q0 = 0, q1 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q0 = f2_fma(x.a[i], x.a[i], q0);
    q1 = f2_fma(x.b[i], x.b[i], q1);
  }
  q0 = f2_add(q0, q1);
  const float rinv =
      rsqrtf(fmaf(head_sum(f2_lo(q0) + f2_hi(q0), lanes), p.inv_d, p.eps));
  const uint64_t rr = f2(rinv, rinv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.a[i] = f2_mul(x.a[i], f.same.a[i]);
    y.b[i] = f2_mul(x.b[i], f.same.b[i]);
  }
  if (l.turns) {   // the others keep an infinite neighbour out of their values
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y.a[i] = f2_fma(IL ? f2_swap(x.a[i]) : x.b[i], f.other.a[i], y.a[i]);
      y.b[i] = f2_fma(IL ? f2_swap(x.b[i]) : x.a[i], f.other.b[i], y.b[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.a[i] = f2_mul(y.a[i], rr);
    y.b[i] = f2_mul(y.b[i], rr);
  }
  x0 = ok ? pack8(y.a) : make_uint4(0, 0, 0, 0);
  x1 = ok ? pack8(y.b) : make_uint4(0, 0, 0, 0);
  *rinv_out = ok ? rinv : 0.f;
}

// One round of the backward pass: x0, x1 and y0, y1 are the lane's vectors of
// x and dy of its head; dx comes back in x0, x1 and the terms of dgamma are
// added to sum.
template <bool IL>
__device__ __forceinline__ void backward_head(const RopeParams& p, const RopeLane& l, int lanes,
                                              uint4& x0, uint4& x1, const uint4& y0,
                                              const uint4& y1, const RopeValues& gain,
                                              const float (&c)[8], const float (&s)[8],
                                              RopeValues& sum) {
  RopeValues x, g;
  unpack8(x.a, x0);
  unpack8(x.b, x1);
  unpack8(g.a, y0);
  unpack8(g.b, y1);
  if (l.turns) rotate_back<IL>(g, c, s);
  RopeValues u;
  uint64_t q0 = 0, q1 = 0, w0 = 0, w1 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u.a[i] = f2_mul(g.a[i], gain.a[i]);
    u.b[i] = f2_mul(g.b[i], gain.b[i]);
    q0 = f2_fma(x.a[i], x.a[i], q0);
    q1 = f2_fma(x.b[i], x.b[i], q1);
    w0 = f2_fma(u.a[i], x.a[i], w0);
    w1 = f2_fma(u.b[i], x.b[i], w1);
  }
  q0 = f2_add(q0, q1);
  w0 = f2_add(w0, w1);
  const float ss = head_sum(f2_lo(q0) + f2_hi(q0), lanes);
  const float ux = head_sum(f2_lo(w0) + f2_hi(w0), lanes);
  const float rinv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
  const float k = -(ux * p.inv_d * rinv) * (rinv * rinv);
  const uint64_t rr = f2(rinv, rinv), kk = f2(k, k);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum.a[i] = f2_fma(g.a[i], f2_mul(x.a[i], rr), sum.a[i]);
    sum.b[i] = f2_fma(g.b[i], f2_mul(x.b[i], rr), sum.b[i]);
    x.a[i] = f2_fma(x.a[i], kk, f2_mul(u.a[i], rr));
    x.b[i] = f2_fma(x.b[i], kk, f2_mul(u.b[i], rr));
  }
  x0 = pack8(x.a);
  x1 = pack8(x.b);
}

// Threads along the columns of the sum of the CTAs' rows by one CTA (at most 32
// rows of threads are left).
__host__ __device__ __forceinline__ int sum_columns(int d) {
  int wide = kRopeThreads / 32;
  while (4 * wide < d) wide *= 2;
  return wide;
}

// The CTA's row of partial sums for dgamma: over the heads of a warp, then
// over its warps; and, by the last CTA to get here, the sum of the CTAs' rows.
// Every sum has a fixed order, whichever CTA comes last.  red: [warps][d] at
// least, and [32][8] floats.
__device__ __forceinline__ void reduce_gain_grad(const RopeParams& p, const RopeLane& l, int lanes,
                                                 const RopeValues& sum, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t a = sum.a[i], b = sum.b[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o >= lanes) {
        a = f2_add(a, __shfl_xor_sync(0xFFFFFFFFu, (unsigned long long)a, o));
        b = f2_add(b, __shfl_xor_sync(0xFFFFFFFFu, (unsigned long long)b, o));
      }
    if (l.active && lane < lanes) {
      *reinterpret_cast<float2*>(red + warp * p.d + l.e0 + 2 * i) = make_float2(f2_lo(a), f2_hi(a));
      *reinterpret_cast<float2*>(red + warp * p.d + l.e1 + 2 * i) = make_float2(f2_lo(b), f2_hi(b));
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.d; j += kRopeThreads) {
    float v = 0.f;
    for (int w = 0; w < kRopeWarps; ++w) v += red[w * p.d + j];
    p.partial[(int64_t)blockIdx.x * p.d + j] = v;
  }
  if (p.sched == nullptr) return;

  __shared__ int last;
  __threadfence();   // this thread's values of the row are visible before it is counted
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.sched + 1, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) atomicExch(p.sched + 1, 0u);   // ready for the next launch
  __threadfence();
  // four columns per thread, the rows strided over the threads, both tensors at once
  const int wide = sum_columns(p.d);
  const int c = threadIdx.x & (wide - 1), r0 = threadIdx.x / wide, rows = kRopeThreads / wide;
  float4* part = reinterpret_cast<float4*>(red);         // [kRopeThreads]
  for (int i = 0; i < 2; ++i) {
    const unsigned begin = i ? p.ctas_q : 0, end = i ? gridDim.x : p.ctas_q;
    const float4* row = reinterpret_cast<const float4*>(p.partial) + c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    // 32 strided sums per column, this thread's four at a time
    for (int w0 = r0; w0 < 32 && 4 * c < p.d; w0 += 4 * rows) {
      float4 a[4] = {};
#pragma unroll 4
      for (unsigned r = begin; r < end; r += 32)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned at = r + w0 + k * rows;
          if (w0 + k * rows < 32 && at < end) {
            const float4 x = __ldcg(row + (int64_t)at * (p.d / 4));
            a[k].x += x.x, a[k].y += x.y, a[k].z += x.z, a[k].w += x.w;
          }
        }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w0 + k * rows < 32)
          v.x += a[k].x, v.y += a[k].y, v.z += a[k].z, v.w += a[k].w;
    }
    __syncthreads();
    part[threadIdx.x] = v;
    __syncthreads();
    if (r0 == 0 && 4 * c < p.d) {
      for (int w = 1; w < rows; ++w) {
        const float4 x = part[w * wide + c];
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      float* out = p.dgamma[i] + 4 * c;
      out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
    }
  }
}

// ------------------------------------------------- few items: direct loads
//
// A warp takes one round of heads of one token straight from global memory.
// Every load of an item is issued at once; nothing is staged.

template <bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_forward_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const unsigned per_token = p.ten[0].chunks + p.ten[1].chunks;
  const unsigned item = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  allow_dependent_launch();
  if (item >= p.T * per_token) return;
  const unsigned t = item / per_token;
  unsigned chunk = item - t * per_token;
  const int ti = chunk >= p.ten[0].chunks;
  const RopeTensor& tn = p.ten[ti];
  if (ti) chunk -= p.ten[0].chunks;
  const RopeItem it = rope_item(tn, t, chunk, p.heads);
  const int sub = lane >> p.lshift;
  const bool in = l.active && sub < it.heads;
  const int64_t at = (int64_t)(it.h0 + sub) * p.d;
  uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
  float c[8] = {}, s[8] = {}, g0[8] = {}, g1[8] = {};
  if (in) {
    const __nv_bfloat16* x = tn.x + (int64_t)t * tn.ldx + at;
    x0 = ldg_stream(x + l.e0);
    x1 = ldg_stream(x + l.e1);
    load8(g0, tn.gamma + l.e0, tn.gamma + l.e0 + 4);
    load8(g1, tn.gamma + l.e1, tn.gamma + l.e1 + 4);
  }
  const float* row;
  const bool ok = table_row(p, t, lane, &row);
  if (l.turns) {
    load8(c, row + l.c0, row + l.c1);
    load8(s, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
  }
  float rinv;
  forward_head<IL>(p, l, lanes, x0, x1, gain_factors<IL>(l, g0, g1, c, s), ok, &rinv);
  if (in) {
    __nv_bfloat16* y = tn.out + (int64_t)t * tn.ldout + at;
    st_global_v4_stream(y + l.e0, x0);
    st_global_v4_stream(y + l.e1, x1);
    if (tn.rinv != nullptr && l.e0 == 0) tn.rinv[(int64_t)t * tn.nheads + it.h0 + sub] = rinv;
  }
}

// The first ctas_q CTAs take the items of Q, the others those of K, in a
// fixed order, so the result does not depend on timing.
template <bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_backward_kernel(const RopeParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const int ti = blockIdx.x >= p.ctas_q;
  const RopeTensor& tn = p.ten[ti];
  const unsigned ctas = ti ? gridDim.x - p.ctas_q : p.ctas_q;
  const unsigned items = p.T * tn.chunks;
  const unsigned step = ctas * kRopeWarps;
  const int sub = lane >> p.lshift;
  grid_dependency_wait();
  allow_dependent_launch();
  RopeValues sum = {};
  const RopeValues gain = load_gain(tn, l);
  for (unsigned item = (ti ? blockIdx.x - p.ctas_q : blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
       item < items; item += step) {
    const unsigned t = item / tn.chunks;
    const RopeItem it = rope_item(tn, t, item - t * tn.chunks, p.heads);
    const bool in = l.active && sub < it.heads;
    const int64_t at = (int64_t)(it.h0 + sub) * p.d;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, y0 = x0, y1 = x0;
    if (in) {
      const __nv_bfloat16* x = tn.x + (int64_t)t * tn.ldx + at;
      const __nv_bfloat16* y = tn.dy + (int64_t)t * tn.lddy + at;
      x0 = ldg_stream(x + l.e0);
      x1 = ldg_stream(x + l.e1);
      y0 = ldg_stream(y + l.e0);
      y1 = ldg_stream(y + l.e1);
    }
    const float* row;
    const bool ok = table_row(p, t, lane, &row);
    float c[8] = {}, s[8] = {};
    if (l.turns) {
      load8(c, row + l.c0, row + l.c1);
      load8(s, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
    }
    if (ok)   // of the whole warp
      backward_head<IL>(p, l, lanes, x0, x1, y0, y1, gain, c, s, sum);
    else
      x0 = x1 = make_uint4(0, 0, 0, 0);
    if (in) {
      __nv_bfloat16* o = tn.out + (int64_t)t * tn.ldout + at;
      st_global_v4_stream(o + l.e0, x0);
      st_global_v4_stream(o + l.e1, x1);
    }
  }
  reduce_gain_grad(p, l, lanes, sum, reinterpret_cast<float*>(smem));
}

// ------------------------------------------------- many items: a ring per warp
//
// Persistent warps, each with its own ring of S shared-memory stages that its
// lane 0 keeps filled with 1-D bulk copies of its next items (R rounds of
// heads of a token each; x, and dy in the backward pass): the loads of the
// next items are in flight while an item is computed, without a register or
// a barrier between warps.  Items go round-robin over the warps.

struct RopeRing {
  uint32_t base;        // this warp's stages
  uint32_t bars;        // its S full barriers
  uint32_t stage;       // bytes per stage
  int S;
};

__device__ __forceinline__ RopeRing rope_ring(const RopeParams& p, unsigned char* smem) {
  RopeRing r;
  const uint32_t warp = threadIdx.x >> 5;
  r.S = p.stages;
  r.stage = p.stage_bytes;
  r.base = smem_addr(smem) + warp * r.S * r.stage;
  r.bars = smem_addr(smem) + kRopeWarps * r.S * r.stage + warp * r.S * 8;
  if ((threadIdx.x & 31) == 0) {
    for (int s = 0; s < r.S; ++s) mbar_init(r.bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  return r;
}

// Waits for stage s: lane 0 tries for the warp.
__device__ __forceinline__ bool ring_wait(const RopeParams& p, const RopeRing& r, int s,
                                          uint32_t parity) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    ok = mbar_wait_bounded(r.bars + 8 * s, parity, p.wait_limit_ns);
    if (!ok) atomicOr(&g_rope_status, kStatusTimeout);
  }
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// After an expired wait at stage s: the copies in flight (every stage) land, bounded.
__device__ __forceinline__ void ring_drain(const RopeParams& p, const RopeRing& r, int s,
                                           uint32_t parity, unsigned left) {
  for (unsigned i = 0; i < left; ++i) {
    (void)mbar_wait_bounded(r.bars + 8 * s, parity, p.wait_limit_ns);
    if (++s == r.S) {
      s = 0;
      parity ^= 1u;
    }
  }
}

template <bool IL>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_forward_ring_kernel(const RopeParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const int hps = 32 >> p.lshift;
  const unsigned per_token = p.ten[0].chunks + p.ten[1].chunks;
  const unsigned items = p.T * per_token;
  const unsigned step = gridDim.x * kRopeWarps;
  const RopeRing ring = rope_ring(p, smem);
  const uint64_t policy = l2_policy_evict_first();
  grid_dependency_wait();
  allow_dependent_launch();

  auto place = [&](const RopeCursor& cur, int* ti) {
    *ti = cur.chunk >= p.ten[0].chunks;
    return rope_item(p.ten[*ti], cur.t, *ti ? cur.chunk - p.ten[0].chunks : cur.chunk, p.heads);
  };
  auto issue = [&](const RopeCursor& cur, int s, uint32_t extra) {
    int ti;
    const RopeItem it = place(cur, &ti);
    const RopeTensor& tn = p.ten[ti];
    const uint32_t bytes = (uint32_t)it.heads * p.d * 2;
    mbar_arrive_expect_tx(ring.bars + 8 * s, bytes + extra);
    bulk_g2s(ring.base + s * ring.stage, tn.x + (int64_t)it.t * tn.ldx + (int64_t)it.h0 * p.d,
             bytes, ring.bars + 8 * s, policy);
  };
  // items of this warp: first, first + step, ...
  const unsigned first = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const unsigned mine = first < items ? (items - first - 1) / step + 1 : 0;
  RopeCursor cur(first, step, per_token), next = cur;   // computed, copied
  for (unsigned n = 0; n < mine && n < (unsigned)ring.S; ++n) {
    if (lane == 0) issue(next, (int)n, n == 0 ? p.missing_tx : 0u);
    next.advance();
  }

  int s = 0;
  uint32_t parity = 0;
  for (unsigned n = 0; n < mine; ++n, cur.advance()) {
    int ti;
    const RopeItem it = place(cur, &ti);
    const RopeTensor& tn = p.ten[ti];
    const float* row;
    const bool ok = table_row(p, it.t, lane, &row);
    float c[8] = {}, sn[8] = {}, g0[8] = {}, g1[8] = {};
    if (l.active) {
      load8(g0, tn.gamma + l.e0, tn.gamma + l.e0 + 4);
      load8(g1, tn.gamma + l.e1, tn.gamma + l.e1 + 4);
    }
    if (l.turns) {
      load8(c, row + l.c0, row + l.c1);
      load8(sn, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
    }
    const RopeFactors f = gain_factors<IL>(l, g0, g1, c, sn);
    if (!ring_wait(p, ring, s, parity)) {
      ring_drain(p, ring, s, parity, min(mine - n, (unsigned)ring.S));
      break;
    }
    const unsigned char* stage =
        smem + ((threadIdx.x >> 5) * ring.S + s) * ring.stage;
    __nv_bfloat16* y = tn.out + (int64_t)it.t * tn.ldout + (int64_t)it.h0 * p.d;
    float* rinv_out =
        tn.rinv != nullptr ? tn.rinv + (int64_t)it.t * tn.nheads + it.h0 : nullptr;
    for (int h = lane >> p.lshift; h - (lane >> p.lshift) < it.heads; h += hps) {
      const bool in = l.active && h < it.heads;
      uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
      if (in) {
        x0 = lds128(stage + (h * p.d + l.e0) * 2);
        x1 = lds128(stage + (h * p.d + l.e1) * 2);
      }
      float rinv;
      forward_head<IL>(p, l, lanes, x0, x1, f, ok, &rinv);
      if (in) {
        st_global_v4_stream(y + (int64_t)h * p.d + l.e0, x0);
        st_global_v4_stream(y + (int64_t)h * p.d + l.e1, x1);
        if (rinv_out != nullptr && l.e0 == 0) rinv_out[h] = rinv;
      }
    }
    fence_proxy_async_smem();   // the stage's reads come before the copy that refills it
    __syncwarp();
    if (n + ring.S < mine) {
      if (lane == 0) issue(next, s, 0u);
      next.advance();
    }
    if (++s == ring.S) {
      s = 0;
      parity ^= 1u;
    }
  }
}

template <bool IL>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_backward_ring_kernel(const RopeParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << p.lshift;
  const RopeLane l = rope_lane<IL>(p, lane & (lanes - 1));
  const int hps = 32 >> p.lshift;
  const int ti = blockIdx.x >= p.ctas_q;
  const RopeTensor& tn = p.ten[ti];
  const unsigned ctas = ti ? gridDim.x - p.ctas_q : p.ctas_q;
  const unsigned items = p.T * tn.chunks;
  const unsigned step = ctas * kRopeWarps;
  const uint32_t half = p.stage_bytes / 2;   // x, then dy
  const RopeRing ring = rope_ring(p, smem);
  const uint64_t policy = l2_policy_evict_first();
  grid_dependency_wait();
  allow_dependent_launch();

  auto issue = [&](const RopeCursor& cur, int s, uint32_t extra) {
    const RopeItem it = rope_item(tn, cur.t, cur.chunk, p.heads);
    const uint32_t bytes = (uint32_t)it.heads * p.d * 2;
    const uint32_t at = ring.base + s * ring.stage;
    mbar_arrive_expect_tx(ring.bars + 8 * s, 2 * bytes + extra);
    bulk_g2s(at, tn.x + (int64_t)it.t * tn.ldx + (int64_t)it.h0 * p.d, bytes, ring.bars + 8 * s,
             policy);
    bulk_g2s(at + half, tn.dy + (int64_t)it.t * tn.lddy + (int64_t)it.h0 * p.d, bytes,
             ring.bars + 8 * s, policy);
  };
  const unsigned first =
      (ti ? blockIdx.x - p.ctas_q : blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const unsigned mine = first < items ? (items - first - 1) / step + 1 : 0;
  RopeCursor cur(first, step, tn.chunks), next = cur;   // computed, copied
  for (unsigned n = 0; n < mine && n < (unsigned)ring.S; ++n) {
    if (lane == 0) issue(next, (int)n, n == 0 ? p.missing_tx : 0u);
    next.advance();
  }

  RopeValues sum = {};
  const RopeValues gain = load_gain(tn, l);
  int s = 0;
  uint32_t parity = 0;
  for (unsigned n = 0; n < mine; ++n, cur.advance()) {
    const RopeItem it = rope_item(tn, cur.t, cur.chunk, p.heads);
    const float* row;
    const bool ok = table_row(p, it.t, lane, &row);
    float c[8] = {}, sn[8] = {};
    if (l.turns) {
      load8(c, row + l.c0, row + l.c1);
      load8(sn, row + p.rot / 2 + l.c0, row + p.rot / 2 + l.c1);
    }
    if (!ring_wait(p, ring, s, parity)) {
      ring_drain(p, ring, s, parity, min(mine - n, (unsigned)ring.S));
      break;
    }
    const unsigned char* stage =
        smem + ((threadIdx.x >> 5) * ring.S + s) * ring.stage;
    __nv_bfloat16* o = tn.out + (int64_t)it.t * tn.ldout + (int64_t)it.h0 * p.d;
    for (int h = lane >> p.lshift; h - (lane >> p.lshift) < it.heads; h += hps) {
      const bool in = l.active && h < it.heads;
      uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, y0 = x0, y1 = x0;
      if (in) {
        const unsigned char* at = stage + h * p.d * 2;
        x0 = lds128(at + l.e0 * 2);
        x1 = lds128(at + l.e1 * 2);
        y0 = lds128(at + half + l.e0 * 2);
        y1 = lds128(at + half + l.e1 * 2);
      }
      if (ok)
        backward_head<IL>(p, l, lanes, x0, x1, y0, y1, gain, c, sn, sum);
      else
        x0 = x1 = make_uint4(0, 0, 0, 0);
      if (in) {
        st_global_v4_stream(o + (int64_t)h * p.d + l.e0, x0);
        st_global_v4_stream(o + (int64_t)h * p.d + l.e1, x1);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (n + ring.S < mine) {
      if (lane == 0) issue(next, s, 0u);
      next.advance();
    }
    if (++s == ring.S) {
      s = 0;
      parity ^= 1u;
    }
  }
  __syncthreads();   // every warp is done with its stages
  reduce_gain_grad(p, l, lanes, sum, reinterpret_cast<float*>(smem));
}

// dgamma = the sum of the CTAs' rows as a launch of its own, for many rows (one
// CTA would take longer than the launch) and inside a graph: block (32 columns)
// x (8 threads with four of 32 strided sums each), blockIdx.y the tensor.  The
// strided sums are added in the order of the last CTA of an eager call, whose
// threads have ROWS rows: equal bits.
template <int ROWS>
__global__ void __launch_bounds__(256) rope_gain_grad_kernel(const float* partial, unsigned nq,
                                                             unsigned n, int d, float* dgamma_q,
                                                             float* dgamma_k) {
  __shared__ float red[32][32];
  const int col = blockIdx.x * 32 + threadIdx.x;
  const unsigned r0 = blockIdx.y ? nq : 0, r1 = blockIdx.y ? n : nq;
  grid_dependency_wait();
  allow_dependent_launch();
  float v[4] = {};
  if (col < d)
#pragma unroll 4
    for (unsigned r = r0 + threadIdx.y; r < r1; r += 32)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + 8 * k < r1) v[k] += partial[(int64_t)(r + 8 * k) * d + col];
#pragma unroll
  for (int k = 0; k < 4; ++k) red[threadIdx.y + 8 * k][threadIdx.x] = v[k];
  __syncthreads();
  if (threadIdx.y != 0 || col >= d) return;
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < ROWS; ++w) {
    float t = 0.f;
#pragma unroll
    for (int k = w; k < 32; k += ROWS) t += red[k][threadIdx.x];
    sum = w == 0 ? t : sum + t;
  }
  (blockIdx.y ? dgamma_k : dgamma_q)[col] = sum;
}

using GainGradKernel = void (*)(const float*, unsigned, unsigned, int, float*, float*);

GainGradKernel pick_gain_grad(int rows) {
  switch (rows) {
    case 2: return rope_gain_grad_kernel<2>;
    case 4: return rope_gain_grad_kernel<4>;
    case 8: return rope_gain_grad_kernel<8>;
    case 16: return rope_gain_grad_kernel<16>;
    default: return rope_gain_grad_kernel<32>;
  }
}

using RopeKernel = void (*)(RopeParams);

RopeParams common_params(const RopeRequest& rq, const LaunchTuning& tune) {
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
  p.wait_limit_ns = tune.wait_limit_ns;
  p.missing_tx = tune.missing_tx;
  return p;
}

// Items of a launch in which a warp takes `rounds` rounds of heads of a token
// at once; fills in the tensors' items per token.  UNSUPPORTED past 32 bits.
int set_items(RopeParams* p, int rounds, uint64_t (&items)[2]) {
  p->heads = rounds * (32 >> p->lshift);
  for (int i = 0; i < 2; ++i) {
    p->ten[i].chunks = (unsigned)((p->ten[i].nheads + p->heads - 1) / p->heads);
    items[i] = (uint64_t)p->T * p->ten[i].chunks;
  }
  if (items[0] + items[1] >= (1ull << 31))
    return fail(NTS_ERR_UNSUPPORTED, "too many token-heads in one call");
  return NTS_OK;
}

// Rounds per item: at most `most`, the rounds of a token's heads in even parts
// (Q's: it has the more).
int even_rounds(const RopeParams& p, int most) {
  const int hps = 32 >> p.lshift;
  const int all = (std::max(p.ten[0].nheads, p.ten[1].nheads) + hps - 1) / hps;
  const int parts = (all + most - 1) / most;
  return (all + parts - 1) / parts;
}

// Ring shape, `copies` operands per stage: bytes of shared memory.
size_t set_ring(RopeParams* p, int copies, int stages) {
  p->stages = stages;
  p->stage_bytes = (uint32_t)(p->heads * p->d * 2 * copies);
  const size_t ring = (size_t)kRopeWarps * stages * (p->stage_bytes + 8);
  return std::max(ring, (size_t)kRopeWarps * std::max(p->d, 128) * sizeof(float));   // the sums
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
  RopeParams p = common_params(rq, tune);
  uint64_t items[2];
  int rc = set_items(&p, 1, items);
  if (rc != NTS_OK) return rc;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  note_launch(kRopeUnit);
  const bool ring = tune.force_rows > 0 || items[0] + items[1] > (uint64_t)dev.sm_count * kDirectItems;
  size_t smem = 0;
  unsigned grid = (unsigned)((items[0] + items[1] + kRopeWarps - 1) / kRopeWarps);
  RopeKernel kern = rq.interleaved ? rope_forward_kernel<true> : rope_forward_kernel<false>;
  if (ring) {
    kern = rq.interleaved ? rope_forward_ring_kernel<true> : rope_forward_ring_kernel<false>;
    rc = set_items(&p, tune.force_rows > 0 ? tune.force_rows : even_rounds(p, kForwardRounds), items);
    if (rc != NTS_OK) return rc;
    smem = set_ring(&p, 1, tune.force_stages > 0 ? tune.force_stages : kForwardStages);
    if (smem > (size_t)dev.max_smem_optin)
      return fail(NTS_ERR_UNSUPPORTED, "the ring takes %zu bytes of shared memory", smem);
    int per_sm = 0;
    rc = prepare_kernel((const void*)kern, smem);
    if (rc == NTS_OK) rc = blocks_per_sm((const void*)kern, kRopeThreads, smem, &per_sm);
    if (rc != NTS_OK) return rc;
    grid = (unsigned)std::min<uint64_t>((items[0] + items[1] + kRopeWarps - 1) / kRopeWarps,
                                        (uint64_t)per_sm * dev.sm_count);
  }
  log_launch("qknorm_rope", "T=%u heads=%d+%d d=%d rot=%d ring=%d per item=%d S=%d smem=%zu grid=%u",
             p.T, p.ten[0].nheads, p.ten[1].nheads, p.d, p.rot, ring, p.heads, p.stages, smem, grid);
  return launch(kern, dim3(grid), dim3(kRopeThreads), smem, stream, tune.pdl != 0, p);
}

int launch_rope_backward(const RopeRequest& rq, float* dgamma_q, float* dgamma_k,
                         float* workspace, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  RopeParams p = common_params(rq, tune);
  uint64_t items[2];
  int rc = set_items(&p, 1, items);
  if (rc != NTS_OK) return rc;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  note_launch(kRopeUnit);
  const bool ring = tune.force_rows > 0 ||
                    items[0] + items[1] > (uint64_t)dev.sm_count * kBackwardDirectItems;
  size_t smem = (size_t)kRopeWarps * std::max(p.d, 128) * sizeof(float);
  RopeKernel kern = rq.interleaved ? rope_backward_kernel<true> : rope_backward_kernel<false>;
  if (ring) {
    kern = rq.interleaved ? rope_backward_ring_kernel<true> : rope_backward_ring_kernel<false>;
    rc = set_items(&p, tune.force_rows > 0 ? tune.force_rows : even_rounds(p, kBackwardRounds), items);
    if (rc != NTS_OK) return rc;
    smem = set_ring(&p, 2, tune.force_stages > 0 ? tune.force_stages : kBackwardStages);
  }
  if (smem > (size_t)dev.max_smem_optin)
    return fail(NTS_ERR_UNSUPPORTED, "the ring takes %zu bytes of shared memory", smem);
  int per_sm = 0;
  rc = prepare_kernel((const void*)kern, smem);
  if (rc == NTS_OK) rc = blocks_per_sm((const void*)kern, kRopeThreads, smem, &per_sm);
  if (rc != NTS_OK) return rc;
  // CTAs in proportion to the tensors' items, one at least for each
  const uint64_t nq = (items[0] + kRopeWarps - 1) / kRopeWarps;
  const uint64_t nk = (items[1] + kRopeWarps - 1) / kRopeWarps;
  const uint64_t most =
      std::min<uint64_t>((uint64_t)per_sm * dev.sm_count, kRopePartials);
  uint64_t gq = nq, gk = nk;
  if (gq + gk > most) {
    const uint64_t all = items[0] + items[1];
    gq = std::max<uint64_t>(1, std::min<uint64_t>(most - 1, (most * items[0] + all / 2) / all));
    gk = std::min<uint64_t>(nk, most - gq);
    gq = std::min<uint64_t>(nq, gq);
  }
  p.ctas_q = (unsigned)gq;
  p.partial = workspace;
  p.dgamma[0] = dgamma_q;
  p.dgamma[1] = dgamma_k;
  const unsigned grid = (unsigned)(gq + gk);
  // Few rows: the last CTA sums them, and the call is one launch ([333, 32 + 8
  // heads of 64], back to back from the host: 9.4 us a call, 11.4 with two).  In
  // a graph, where a launch costs less than the last CTA's latencies, two (7.2
  // us, one 8.4).
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &capture) != cudaSuccess) (void)cudaGetLastError();
  const bool few = (int64_t)grid * p.d <= kFusedSums;
  const bool wide = reinterpret_cast<uintptr_t>(workspace) % 16 == 0;   // float4 loads
  p.sched = tune.dynamic && few && wide && capture == cudaStreamCaptureStatusNone
                ? sched_counters(stream)
                : nullptr;
  log_launch("qknorm_rope_backward",
             "T=%u heads=%d+%d d=%d rot=%d ring=%d per item=%d S=%d smem=%zu grid=%u (%u for Q)",
             p.T, p.ten[0].nheads, p.ten[1].nheads, p.d, p.rot, ring, p.heads, p.stages, smem, grid,
             p.ctas_q);
  rc = launch(kern, dim3(grid), dim3(kRopeThreads), smem, stream, tune.pdl != 0, p);
  if (rc != NTS_OK || p.sched != nullptr) return rc;
  return launch(pick_gain_grad(kRopeThreads / sum_columns(p.d)), dim3((p.d + 31) / 32, 2),
                dim3(32, 8), 0, stream, tune.pdl != 0, (const float*)workspace, (unsigned)gq, grid,
                p.d, dgamma_q, dgamma_k);
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
