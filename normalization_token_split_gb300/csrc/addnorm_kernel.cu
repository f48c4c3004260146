// addnorm_kernel.cu -- the addition of a layer's output to the residual stream with
// RMSNorm and the cast to E4M3 codes with a scale per 128 values in the same pass
// (nts_rmsnorm_blockcast with an addition in front), and its gradient, on one GB300.
//
// Forward, per row of D values:
//     h_j  = round(x_j + r_j) to the stream's type (bf16 or fp32),
//     rinv = 1 / sqrt((1/D) sum h^2 + eps),  w_j = (h_j gamma_j) rinv,
// and the scales and codes of w as nts_rmsnorm_blockcast forms them.  The statistic
// is that of the h that is stored, so the gradient needs nothing but h and rinv.
// Backward, with dy the gradient of w, u_j = dy_j gamma_j and e the gradient of h from
// the layers behind:
//     dh_j = rinv u_j - h_j rinv^3 (1/D) sum u h + e_j   (of x and of r alike),
//     dgamma_j = sum over rows of dy_j h_j rinv.
//
// GB300 mapping: both are bound by HBM (7 to 11 and 8 to 16 bytes per value, 7 and 11
// flops).  A thread owns 16 neighbouring values of a row, the same ones of every row it
// meets, so its gains and its sums for dgamma stay in registers; eight lanes hold a
// block of 128.  A warp copies its part of the next rows into its own stages of shared
// memory (cp.async: no thread waits for another warp's copies), and a row's warps
// meet once, for the sum.  Rows of more than 8192 values (5120 in the gradient of an
// fp32 stream) are split over the CTAs of a cluster, whose warps write their sums into
// every CTA's shared memory.
//
// Measured (us, back to back in a graph over more than L2; of the copy's rate): forward
// [16384, 4096] bf16 73.4, 0.95; [1237, 5120] fp32 10.6, 0.97; [8, 4096] 2.1.  Gradient
// [8192, 5120] bf16 53.7, 0.92; [8192, 4096] fp32 83.8, 0.94; [333, 4096] fp32 9.2, of
// which 4.1 are its two launches at one row.  Rows of 16384, a meeting of the cluster
// each: [2000, 16384] bf16 43.6, 0.78, and [2048, 16384] bf16 53.7, 0.74.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_device.cuh"
#include "block_internal.h"

namespace nts {

namespace {

constexpr int kMaxRowThreads = 512;   // a CTA's part of a row, in units of 16 values
constexpr int kMaxWarps = kMaxRowThreads / 32;
constexpr int kGroupThreads = 256;    // narrower rows share a CTA of about this size
// Units of a row up to which one CTA takes it.  Slices of 256 instead: forward
// [8192, 8192] 120 us, 110 so; gradient [4096, 8192] 49.4 and 46.8.  The gradient of an
// fp32 stream keeps 2.5 times the bytes of a bf16 one in a stage.
constexpr int kForwardUnits = 512, kBackwardUnits = 512, kBackwardUnits32 = 320;

// Stages of a warp and registers of a thread.  The forward pass of a long call is best
// with 32 warps an SM and three stages ([16384, 4096] bf16 73.1 us; two stages 81.2; 72
// registers, 24 warps, 80.1), of a short one, or with CTAs of more than 320 threads,
// with more registers and two stages ([4000, 4096] 16.1 us, 20.9 the other way; [2000,
// 5120] fp32 15.8 and 21.1; [8000, 8192] bf16 71.1 and 77.6).  Split rows wait longest
// for each other and want the warps ([2000, 16384] bf16 43.3, 64.3 with 72 registers).
// The gradient has 32 registers of gains and sums: [8192, 5120] bf16 53.9 us with 80,
// 63.8 with 64 and spills; [8192, 4096] fp32 84.0 with 96 and three stages, 88.2 with
// two, 94.4 with 80.  In clusters [2048, 16384] bf16 53.6 with 64, 64.4 with 80; fp32
// 89.7 with two stages, 135 with three.
constexpr int64_t kFewValues = 24 << 20;
constexpr int kWideThreads = 320;
__host__ __device__ constexpr int forward_stages(bool few) { return few ? 2 : 3; }
__host__ __device__ constexpr int forward_regs(bool f32, bool few) { return !few ? 64 : f32 ? 96 : 72; }
__host__ __device__ constexpr int backward_stages(int cluster, bool f32) { return f32 && cluster == 1 ? 3 : 2; }
__host__ __device__ constexpr int backward_regs(int cluster, bool f32) { return f32 ? 96 : cluster == 1 ? 80 : 64; }

struct AddNormParams {
  const __nv_bfloat16* a;     // x, or dy
  const void* r;              // the residual, or h
  const void* e;              // backward: gradient from behind, or nullptr
  const float* gamma;         // or nullptr: ones
  void* h;                    // forward: the sum; backward: dh
  __nv_bfloat16* dx;          // backward, fp32 stream: dh in bf16, or nullptr
  uint8_t* codes;
  float* scales;
  float* rinv;                // forward: written, or nullptr
  const float* rinv_in;       // backward
  float* partial;             // backward: [CTAs per slice][D] sums for dgamma, or nullptr
  unsigned T;
  int D, blocks;
  int slice;                  // units of a row per CTA, a multiple of 8
  int tpr;                    // threads per row (slice), whole warps
  int wide;                   // rows of h start on 32-byte boundaries
  float eps, inv_d;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's 32 units of a row in shared memory: pieces of 16 bytes, two (bf16) or four
// (fp32) to a unit.  The pieces of a unit change places with the bits of the unit's
// number above those of a 128-byte line, so that the eight lanes of a phase meet
// distinct banks both when neighbouring lanes copy neighbouring pieces and when each
// reads its own unit.
template <int PIECES>
__device__ __forceinline__ uint32_t piece_turn(int lane_or_unit_line) {
  return (uint32_t)lane_or_unit_line & (PIECES - 1);
}

// Copies the warp's units, neighbouring lanes taking neighbouring pieces; units from
// `units` on become zeros.
template <int PIECES>
__device__ __forceinline__ void stage_units(uint32_t dst, const unsigned char* src, int units) {
  const int lane = threadIdx.x & 31;
  dst += 16 * (lane ^ piece_turn<PIECES>(lane >> 3));
  src += 16 * lane;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    cp_async16(dst + 512 * i, src + 512 * i, (32 * i + lane) / PIECES < units);
}

// The lane's unit of a staged bf16 operand, as it is packed.
__device__ __forceinline__ void read_packed(const unsigned char* st, uint32_t (&v)[8]) {
  const int lane = threadIdx.x & 31;
  const uint4 a = lds128(st + 32 * lane + 16 * piece_turn<2>(lane >> 2));
  const uint4 b = lds128(st + 32 * lane + 16 * (piece_turn<2>(lane >> 2) ^ 1));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void unpack(const uint32_t (&w)[8], uint64_t (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = bf16x2_to_f2(w[i]);
}

// Half `h` (8 values) of the lane's unit of a staged operand, in fp32 pairs.
template <bool F32>
__device__ __forceinline__ void read_half(const unsigned char* st, int h, uint64_t (&v)[4]) {
  const int lane = threadIdx.x & 31;
  if constexpr (!F32) {
    const uint4 a = lds128(st + 32 * lane + 16 * (piece_turn<2>(lane >> 2) ^ h));
    v[0] = bf16x2_to_f2(a.x), v[1] = bf16x2_to_f2(a.y);
    v[2] = bf16x2_to_f2(a.z), v[3] = bf16x2_to_f2(a.w);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 a = lds128(st + 64 * lane + 16 * ((2 * h + i) ^ piece_turn<4>(lane >> 1)));
      v[2 * i] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
      v[2 * i + 1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
    }
  }
}

// x + r of two packed bf16, rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t x, uint32_t r) {
  uint32_t h;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(h) : "r"(x), "r"(r));
  return h;
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], int wide) {
  if (wide) {
    st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  } else {
    st_global_v4(p, w[0], w[1], w[2], w[3]);
    st_global_v4(static_cast<unsigned char*>(p) + 16, w[4], w[5], w[6], w[7]);
  }
}

// Four pairs of fp32: 32 bytes.
__device__ __forceinline__ void store_pairs(void* p, const uint64_t (&v)[4], int wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[2 * i] = (uint32_t)v[i];
    w[2 * i + 1] = (uint32_t)(v[i] >> 32);
  }
  store32(p, w, wide);
}

// A thread's place in the grid: the rows its group takes, and its unit of each.
template <int C>
struct Place {
  int lane, warp;       // warp of the row's group in this CTA
  int group;            // group of the CTA (C == 1)
  int rank;             // CTA of the cluster
  int warps;            // warps per row in this CTA
  int unit;             // of the row
  int left;             // units of the warp: its first unit to the row's or slice's end
  bool in;
  unsigned first, step;  // rows
  __device__ __forceinline__ explicit Place(const AddNormParams& p) {
    lane = threadIdx.x & 31;
    group = C == 1 ? (int)threadIdx.x / p.tpr : 0;
    const int t = threadIdx.x - group * p.tpr;
    warp = t >> 5;
    warps = p.tpr >> 5;
    rank = C == 1 ? 0 : (int)cluster_ctarank();
    const int groups = C == 1 ? (int)blockDim.x / p.tpr : 1;
    first = blockIdx.x / C * groups + group;
    step = gridDim.x / C * groups;
    const int begin = rank * p.slice, end = min(begin + p.slice, p.D / 16);
    unit = begin + t;
    left = end - (begin + 32 * warp);
    in = unit < end;
  }
};

// The sum of v over a row: its warps (of every CTA of the cluster) write theirs into
// part[buf] and meet once.  The other buffer's readers are past that meeting.  A CTA's
// warps have `pad` places, a multiple of four, those without a warp zero from the start.
template <int C>
__device__ __forceinline__ float row_sum(float v, const Place<C>& at, const AddNormParams& p,
                                         float* part, int buf) {
  v = warp_sum(v);
  if (C == 1 && at.warps == 1) return v;
  const int pad = (at.warps + 3) & ~3;
  float* mine = part + buf * C * kMaxWarps + (C == 1 ? at.group * pad : 0);
  if (C == 1) {
    if (at.lane == 0) mine[at.warp] = v;
    named_barrier(1 + at.group, p.tpr);
  } else {
    if (at.lane < C)
      st_cluster_f32(map_to_rank(smem_addr(mine + at.rank * pad + at.warp), at.lane), v);
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int w = 0; w < C * pad; w += 4) {
    const float4 x = *reinterpret_cast<const float4*>(mine + w);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  return (s.x + s.y) + (s.z + s.w);
}

template <int C>
__device__ __forceinline__ void start_cluster() {
  if (C > 1) {   // every CTA runs, its parts cleared, before another writes into them
    cluster_arrive_release();
    cluster_wait_acquire();
  }
}

// The parts of the shared memory of a row's sums.
template <int C>
__device__ __forceinline__ void clear_parts(float* part) {
  for (int i = threadIdx.x; i < 2 * C * kMaxWarps; i += blockDim.x) part[i] = 0.f;
  __syncthreads();
}

template <int C, bool F32, bool FEW>
__global__ void __maxnreg__(forward_regs(F32, FEW)) add_rmsnorm_kernel(const AddNormParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) float part[2 * C * kMaxWarps];
  constexpr int kSize = F32 ? 4 : 2;
  constexpr int kStage = 32 * 16 * (2 + kSize);   // of a warp: x, then the residual
  constexpr int kStages = forward_stages(FEW);
  const Place<C> at(p);
  unsigned char* ring = smem + (threadIdx.x >> 5) * kStages * kStage;
  clear_parts<C>(part);
  start_cluster<C>();
  grid_dependency_wait();
  allow_dependent_launch();

  // `off`: the warp's first value of its current row
  const int64_t hop = (int64_t)at.step * p.D;
  int64_t off = (int64_t)at.first * p.D + 16 * (at.unit - at.lane);
  auto stage = [&](unsigned row, int64_t off, int s) {
    if (row < p.T) {
      const uint32_t dst = smem_addr(ring) + s * kStage;
      stage_units<2>(dst, reinterpret_cast<const unsigned char*>(p.a) + 2 * off, at.left);
      stage_units<kSize>(dst + 1024, static_cast<const unsigned char*>(p.r) + kSize * off, at.left);
    }
    cp_async_commit();   // empty groups keep the count
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) stage(at.first + s * at.step, off + s * hop, s);

  uint64_t gain[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.gamma != nullptr && at.in)
      v = __ldg(reinterpret_cast<const float4*>(p.gamma + 16 * at.unit) + j);
    gain[2 * j] = f2(v.x, v.y);
    gain[2 * j + 1] = f2(v.z, v.w);
  }

  int s = 0, buf = 0;
  for (unsigned row = at.first; row < p.T; row += at.step) {
    cp_async_wait<kStages - 1>();
    __syncwarp();   // the warp's copies are seen by all its lanes
    const unsigned char* st = ring + s * kStage;
    uint32_t x[8];
    uint64_t h[8];
    read_packed(st, x);
    if (F32) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint64_t v[4];
        read_half<true>(st + 1024, half, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[4 * half + i] = f2_add(bf16x2_to_f2(x[4 * half + i]), v[i]);
      }
    } else {
      // One rounding from the exact sum: an fp32 sum of two bf16 is inexact only when
      // they lie so far apart that it rounds to the larger one either way.
      uint32_t w[8];
      read_packed(st + 1024, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = add_bf16x2(x[i], w[i]);
    }
    __syncwarp();   // read by all before the next copy into the stage
    stage(row + kStages * at.step, off + kStages * hop, s);
    if (++s == kStages) s = 0;
    const int64_t out = off + 16 * at.lane;
    if (at.in) {
      unsigned char* to = static_cast<unsigned char*>(p.h) + kSize * out;
      if (F32) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t v[4] = {h[4 * half], h[4 * half + 1], h[4 * half + 2], h[4 * half + 3]};
          store_pairs(to + 32 * half, v, p.wide);
        }
      } else {
        store32(to, x, p.wide);
      }
    }
    if (!F32) unpack(x, h);
    uint64_t q0 = 0, q1 = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      q0 = f2_fma(h[i], h[i], q0);
      q1 = f2_fma(h[i + 1], h[i + 1], q1);
    }
    q0 = f2_add(q0, q1);
    const float ss = row_sum<C>(f2_lo(q0) + f2_hi(q0), at, p, part, buf);
    buf ^= 1;
    const float rinv = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
    if (p.rinv != nullptr && at.unit == 0) p.rinv[row] = rinv;
    const uint64_t rr = f2(rinv, rinv);
    if (!F32) unpack(x, h);   // kept packed over the sum
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f2_mul(f2_mul(h[i], gain[i]), rr);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmax3(m, fabsf(f2_lo(h[i])), fabsf(f2_hi(h[i])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float scale = block_scale(m);
    const float inv = __frcp_rn(scale);
    const uint64_t ii = f2(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t lo = f2_mul(h[2 * i], ii), hi = f2_mul(h[2 * i + 1], ii);
      c[i] = cvt_e4m3x4(f2_lo(lo), f2_hi(lo), f2_lo(hi), f2_hi(hi));
    }
    if (at.in) {
      __stcs(reinterpret_cast<uint4*>(p.codes + out), make_uint4(c[0], c[1], c[2], c[3]));
      if ((at.lane & 7) == 0) p.scales[(int64_t)row * p.blocks + (at.unit >> 3)] = scale;
    }
    off += hop;
  }
}

// The operands are read from their stage a second time after the sum, not kept in
// registers, which the gains and the sums for dgamma fill.
template <int C, bool F32>
__global__ void __maxnreg__(backward_regs(C, F32)) add_rmsnorm_backward_kernel(const AddNormParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) float part[2 * C * kMaxWarps];
  constexpr int kSize = F32 ? 4 : 2;
  constexpr int kStage = 32 * 16 * (2 + 2 * kSize);   // dy, h, the gradient from behind
  constexpr int kBehind = 1024 + 512 * kSize;
  constexpr int kStages = backward_stages(C, F32);
  const Place<C> at(p);
  unsigned char* ring = smem + (threadIdx.x >> 5) * kStages * kStage;
  clear_parts<C>(part);
  start_cluster<C>();
  grid_dependency_wait();
  allow_dependent_launch();

  const int64_t hop = (int64_t)at.step * p.D;
  int64_t off = (int64_t)at.first * p.D + 16 * (at.unit - at.lane);
  auto stage = [&](unsigned row, int64_t off, int s) {
    if (row < p.T) {
      const uint32_t dst = smem_addr(ring) + s * kStage;
      stage_units<2>(dst, reinterpret_cast<const unsigned char*>(p.a) + 2 * off, at.left);
      stage_units<kSize>(dst + 1024, static_cast<const unsigned char*>(p.r) + kSize * off, at.left);
      if (p.e != nullptr)
        stage_units<kSize>(dst + kBehind, static_cast<const unsigned char*>(p.e) + kSize * off,
                           at.left);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) stage(at.first + s * at.step, off + s * hop, s);

  uint64_t gain[8], sum[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.gamma != nullptr && at.in)
      v = __ldg(reinterpret_cast<const float4*>(p.gamma + 16 * at.unit) + j);
    gain[2 * j] = f2(v.x, v.y);
    gain[2 * j + 1] = f2(v.z, v.w);
    sum[2 * j] = sum[2 * j + 1] = 0;
  }
  float next = at.first < p.T ? __ldg(p.rinv_in + at.first) : 0.f;

  int s = 0, buf = 0;
  for (unsigned row = at.first; row < p.T; row += at.step) {
    const float rinv = next;
    if (row + at.step < p.T) next = __ldg(p.rinv_in + row + at.step);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const unsigned char* st = ring + s * kStage;
    const uint64_t rr = f2(rinv, rinv);
    uint64_t q = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint64_t g[4], h[4];
      read_half<false>(st, half, g);
      read_half<F32>(st + 1024, half, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * half + i;
        sum[j] = f2_fma(g[i], f2_mul(h[i], rr), sum[j]);
        q = f2_fma(f2_mul(g[i], gain[j]), h[i], q);
      }
    }
    const float uh = row_sum<C>(f2_lo(q) + f2_hi(q), at, p, part, buf);
    buf ^= 1;
    // dh = rinv (u - h k) + e, k = rinv^2 (1/D) sum u h: rinv^2 of a row of zeros with a
    // subnormal eps is beyond fp32, rinv u is not.  Where rinv is 0 the sum may be beyond
    // it too.
    const float k = rinv == 0.f ? 0.f : -((uh * p.inv_d) * rinv) * rinv;
    const uint64_t kk = f2(k, k);
    const int64_t out = off + 16 * at.lane;
    unsigned char* to = static_cast<unsigned char*>(p.h) + kSize * out;
    uint32_t w[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint64_t g[4], h[4];
      read_half<false>(st, half, g);
      read_half<F32>(st + 1024, half, h);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = f2_mul(f2_fma(h[i], kk, f2_mul(g[i], gain[4 * half + i])), rr);
      if (p.e != nullptr) {
        read_half<F32>(st + kBehind, half, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f2_add(h[i], g[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * half + i] = pack_bf16x2_rn(f2_lo(h[i]), f2_hi(h[i]));
      if (F32 && at.in) store_pairs(to + 32 * half, h, p.wide);
    }
    __syncwarp();
    stage(row + kStages * at.step, off + kStages * hop, s);
    if (++s == kStages) s = 0;
    if (at.in) {
      if (!F32) store32(to, w, p.wide);
      if (F32 && p.dx != nullptr) store32(p.dx + out, w, p.wide);
    }
    off += hop;
  }
  if (p.partial == nullptr) return;

  // The CTA's row of sums: over its groups, in their order.
  if (C == 1 && blockDim.x > p.tpr) {
    cp_async_wait<0>();
    __syncthreads();   // every warp is done with its stages
    float* red = reinterpret_cast<float*>(smem);   // [groups][16 slice]
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.in)
        *reinterpret_cast<float2*>(red + (at.group * p.slice + at.unit) * 16 + 2 * i) =
            make_float2(f2_lo(sum[i]), f2_hi(sum[i]));
    __syncthreads();
    const int groups = blockDim.x / p.tpr;
    for (int j = threadIdx.x; j < p.D; j += blockDim.x) {
      float v = red[j];
      for (int g = 1; g < groups; ++g) v += red[g * p.slice * 16 + j];
      p.partial[(int64_t)blockIdx.x * p.D + j] = v;
    }
    return;
  }
  if (at.in)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t id = C == 1 ? blockIdx.x : blockIdx.x / C;
      *reinterpret_cast<float4*>(p.partial + id * p.D + 16 * at.unit + 4 * i) =
          make_float4(f2_lo(sum[2 * i]), f2_hi(sum[2 * i]), f2_lo(sum[2 * i + 1]),
                      f2_hi(sum[2 * i + 1]));
    }
}

// dgamma: the sum of the CTAs' rows, in a fixed order; block (32 columns) x (32
// threads, each with every 32nd row).
__global__ void __launch_bounds__(1024) gain_grad_kernel(const float* partial, int n, int D,
                                                         float* dgamma) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  grid_dependency_wait();
  allow_dependent_launch();
  float v = 0.f;
  if (col < D)
#pragma unroll 8
    for (int r = threadIdx.y; r < n; r += 32) v += __ldcg(partial + (int64_t)r * D + col);
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < D) dgamma[out] = v;
}

using AddNormKernel = void (*)(AddNormParams);

// Rows of at most 2048 units take clusters of up to 4, of up to 8 in the gradient of an
// fp32 stream.
template <int C>
AddNormKernel pick(bool f32, bool backward, bool few) {
  if (f32 && backward) return add_rmsnorm_backward_kernel<C, true>;
  if constexpr (C <= 4) {
    if (backward) return add_rmsnorm_backward_kernel<C, false>;
    if constexpr (C == 1)
      if (few) return f32 ? add_rmsnorm_kernel<C, true, true> : add_rmsnorm_kernel<C, false, true>;
    return f32 ? add_rmsnorm_kernel<C, true, false> : add_rmsnorm_kernel<C, false, false>;
  }
  return nullptr;
}

template <typename... A>
int launch(void (*kern)(A...), cudaLaunchConfig_t cfg, int cluster, cudaStream_t stream, bool pdl,
           A... args) {
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) attr[n++] = pdl_attribute();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
  if (err != cudaSuccess) return fail_cuda(err, "launching the residual addition with RMSNorm");
  return NTS_OK;
}

}  // namespace

int launch_addnorm(const AddNormRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  const bool backward = rq.dgamma != nullptr || rq.rinv_in != nullptr;
  const bool f32 = rq.fp32 != 0;
  AddNormParams p = {};
  p.a = static_cast<const __nv_bfloat16*>(rq.a);
  p.r = rq.r;
  p.e = rq.e;
  p.gamma = rq.gamma;
  p.h = rq.h;
  p.dx = static_cast<__nv_bfloat16*>(rq.dx);
  p.codes = rq.codes;
  p.scales = rq.scales;
  p.rinv = rq.rinv;
  p.rinv_in = rq.rinv_in;
  p.T = (unsigned)rq.T;
  p.D = (int)rq.D;
  p.blocks = (int)((rq.D + 127) / 128);
  p.eps = rq.eps;
  p.inv_d = 1.0f / (float)p.D;
  p.wide = reinterpret_cast<uintptr_t>(rq.h) % 32 == 0 && reinterpret_cast<uintptr_t>(rq.dx) % 32 == 0;
  const int units = p.D / 16;
  const int most_units = !backward ? kForwardUnits : f32 ? kBackwardUnits32 : kBackwardUnits;
  int C = 1;
  while (units > C * most_units) C *= 2;
  p.slice = ((units + C - 1) / C + 7) / 8 * 8;
  p.tpr = (p.slice + 31) / 32 * 32;
  const int groups = C == 1 ? std::max(1, kGroupThreads / p.tpr) : 1;
  const bool few = C == 1 && (rq.T * rq.D <= kFewValues || p.tpr > kWideThreads);
  const AddNormKernel kern = C == 1   ? pick<1>(f32, backward, few)
                             : C == 2 ? pick<2>(f32, backward, few)
                             : C == 4 ? pick<4>(f32, backward, few)
                                      : pick<8>(f32, backward, few);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)(groups * p.tpr));
  const int unit = 32 + (backward ? 2 : 1) * (f32 ? 64 : 32);
  cfg.dynamicSmemBytes =
      (size_t)cfg.blockDim.x * unit * (backward ? backward_stages(C, f32) : forward_stages(few));
  int rc = prepare_kernel((const void*)kern, cfg.dynamicSmemBytes);
  if (rc != NTS_OK) return rc;
  int64_t most = 0;
  if (C == 1) {
    int per_sm = 0;
    rc = blocks_per_sm((const void*)kern, cfg.blockDim.x, cfg.dynamicSmemBytes, &per_sm);
    most = (int64_t)per_sm * dev.sm_count;
  } else {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    rc = max_active_clusters((const void*)kern, cfg, C, &most);
  }
  if (rc != NTS_OK) return rc;
  if (backward) most = std::min<int64_t>(most, kNormPartials);
  const int64_t rows = std::min<int64_t>((rq.T + groups - 1) / groups, most);   // CTAs or clusters
  cfg.gridDim = dim3((unsigned)(rows * C));
  if (rq.dgamma != nullptr) p.partial = rq.partial;
  log_launch(backward ? "add_rmsnorm_backward" : "add_rmsnorm_blockcast",
             "T=%lld D=%d fp32=%d cluster=%d threads=%u rows at once=%d smem=%zu grid=%u",
             (long long)rq.T, p.D, (int)f32, C, cfg.blockDim.x, groups, cfg.dynamicSmemBytes,
             cfg.gridDim.x);
  rc = launch(kern, cfg, C, stream, tune.pdl != 0, p);
  if (rc != NTS_OK || rq.dgamma == nullptr) return rc;
  cudaLaunchConfig_t sum = {};
  sum.gridDim = dim3((unsigned)((p.D + 31) / 32));
  sum.blockDim = dim3(32, 32);
  return launch(gain_grad_kernel, sum, 1, stream, tune.pdl != 0, (const float*)p.partial, (int)rows,
                p.D, rq.dgamma);
}

}  // namespace nts
