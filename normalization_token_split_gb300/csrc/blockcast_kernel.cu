// blockcast_kernel.cu -- casts to E4M3 codes with one fp32 scale for each
// block of 128 values (the operands of nts_gemm_blockscaled) on one GB300:
// of rows with or without RMSNorm in the same pass (1 x 128 blocks), of
// weights (128 x 128 blocks), and of the transpose (128 tokens x 1).
//
// For a block with the largest magnitude a of its values w:
//     scale = fp32(max(a, 2^-100) / 448),
//     code  = E4M3_rne_satfinite(fp32(w * fp32(1 / scale))),
// 448 being the largest E4M3 value.  The floor keeps 1 / scale finite for
// blocks of zeros and of values that no sum with others would show.
// RMSNorm: rinv = 1 / sqrt((1/D) sum x^2 + eps), w = fp32(fp32(x gamma) rinv).
//
// All of these are bound by HBM, 2 bytes read and 1 + 4/128 written per value,
// as far as their instructions allow.  Measured (us, back to back in a graph,
// inputs and outputs rotated over more than L2; of the copy's rate): with the norm
// [16384, 4096] 38.1, 0.79, issue slots 65 % busy with 16 warps an SM; [64, 4096]
// 2.4; without, [16384, 4096] 35.3, 0.85; weights [10240, 5120] 24.8, 0.94; the
// transpose of [4099, 5120] 13.2, 0.71.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_device.cuh"
#include "block_internal.h"

namespace nts {

namespace {

constexpr int kCastThreads = 256;
constexpr int kCastWarps = kCastThreads / 32;
// Values of X from which the ring kernel runs: below, its warps start with
// nothing in flight and the launch is over before that pays (us in a graph: with
// the norm, [256, 4096] 2.9 direct, 3.6 by the ring, [400, 5120] 3.7 and 4.1,
// [800, 5120] 6.8 and 6.5, [1000, 4096] 6.8 and 5.1; without, [1000, 4096] 3.8 and
// 4.3, [2048, 4096] 6.5 by the ring).
constexpr int64_t kRingValues = 4 << 20, kNormRingValues = 3 << 20;

// kStatusTimeout bits of these kernels.
__device__ unsigned int g_cast_status;

struct CastParams {
  const __nv_bfloat16* x;
  const float* gamma;   // RMSNorm, or nullptr
  uint8_t* codes;
  float* scales;
  float* rinv;          // RMSNorm, or nullptr
  int64_t T;
  int D;
  int units;            // D / 16
  int blocks;           // ceil(D / 128)
  int wpr;              // RMSNorm: warps per row (1, 2, 4 or 8)
  int segs;             // no norm: warp segments per row
  int64_t pitch;        // transpose: bytes per row of codes
  int tblocks;          // transpose: ceil(T / 128)
  int64_t ring_units;   // ring: units per row (a whole matrix as one row when blocks never end early)
  int seg;              // ring: units per warp's part of a row, a multiple of 8
  uint64_t wait_limit_ns;
  uint32_t missing_tx;  // test hook: bytes expected on a first stage but never sent
  float eps, inv_d;
};

// Rows in 1 x 128 blocks.  A thread owns UPT units of 16 values (two 16-byte
// loads, one 16-byte store of codes); eight neighbouring lanes hold a block,
// so its largest magnitude takes three shuffles.  With RMSNorm a row is spread
// over wpr warps, which add their sums of squares through shared memory; the
// row stays in registers between the two passes over it.  Without it a warp's
// segment of a row needs nothing from the others.
template <int UPT, bool NORM>
__global__ void __launch_bounds__(kCastThreads) blockcast_rows_kernel(const CastParams p) {
  __shared__ float part[2][kCastWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = NORM ? p.wpr : 1;
  const int rpc = kCastWarps / wpr;              // rows (segments) in flight per CTA
  const int slot = warp / wpr, sub = warp - slot * wpr;
  const int64_t items = NORM ? p.T : p.T * p.segs;
  grid_dependency_wait();
  allow_dependent_launch();
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < items; base += (int64_t)gridDim.x * rpc) {
    const int64_t item = base + slot;
    const bool live = item < items;
    const int64_t t = NORM ? item : item / p.segs;
    const int u0 = (NORM ? sub : (int)(item - t * p.segs)) * 32 * UPT + lane;
    const __nv_bfloat16* xrow = p.x + t * p.D;
    uint4 x[UPT][2];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (live && u0 + 32 * i < p.units) load16(x[i], xrow + 16 * (u0 + 32 * i));
    }
    float rinv = 1.f;
    if (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        float f[16], q[4] = {};
        unpack16(x[i], f);
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j & 3] = fmaf(f[j], f[j], q[j & 3]);
        ss += (q[0] + q[1]) + (q[2] + q[3]);
      }
      ss = warp_sum(ss);
      if (wpr > 1) {   // uniform over the CTA
        if (lane == 0) part[buf][warp] = ss;
        __syncthreads();
        ss = 0.f;
        for (int w = 0; w < wpr; ++w) ss += part[buf][slot * wpr + w];
        buf ^= 1;      // the other buffer's readers are past the barrier above
      }
      rinv = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
      if (live && p.rinv != nullptr && sub == 0 && lane == 0) p.rinv[t] = rinv;
    }
    uint8_t* crow = p.codes + t * p.D;
    float* srow = p.scales + t * p.blocks;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = u0 + 32 * i;
      const bool in = live && u < p.units;
      float f[16];
      unpack16(x[i], f);
      if (NORM) {
        if (p.gamma != nullptr && in) {
          const float4* g = reinterpret_cast<const float4*>(p.gamma + 16 * u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = __ldg(g + j);
            f[4 * j] *= v.x;
            f[4 * j + 1] *= v.y;
            f[4 * j + 2] *= v.z;
            f[4 * j + 3] *= v.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] *= rinv;
      }
      float a = absmax16(f);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      const float scale = block_scale(a);
      const uint4 c = codes16(f, 1.0f / scale);
      if (in) {
        __stcs(reinterpret_cast<uint4*>(crow + 16 * u), c);
        if ((lane & 7) == 0) srow[u >> 3] = scale;
      }
    }
  }
}

// The same for many rows: persistent warps, each with its own ring of kStages
// shared-memory stages that its lane 0 keeps filled with 1-D bulk copies, so
// that the next parts of rows are in flight while one is cast.  With RMSNorm the
// wpr warps of a row add their sums of squares through shared memory behind a
// named barrier, and the part is read a second time from shared memory, not kept
// in registers.  The barrier is what parts cost, so they are as large as the
// gain's registers allow: 160 units (5 KB; [16384, 4096] by four warps a row in
// place of two 51.1 us, 38.1 so); without the norm 128.  A thread reads the two
// vectors of its unit in the order that lets the 8 lanes of each shared-memory
// phase hit distinct banks.  GAIN: a thread meets the same units of the gain on
// every row and keeps the first four in registers (all from L1, where a warp's
// 64-byte steps take 16 passes a load: [16384, 4096] 45.3 us); a fifth is read
// from L1 ([8192, 5120] 26.8 us, 33.7 by four warps a row).
constexpr int kStages = 2;
constexpr int kPartUnits = 160, kHeldUnits = 128;

template <bool NORM, bool GAIN>
__global__ void __launch_bounds__(kCastThreads, GAIN ? 2 : 3)
blockcast_ring_kernel(const CastParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[kCastWarps][kStages];
  __shared__ float part[2][kCastWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = NORM ? p.wpr : 1;
  const int rpc = kCastWarps / wpr;
  const int slot = warp / wpr, sub = warp - slot * wpr;
  const uint32_t stage = (uint32_t)p.seg * 32;
  const unsigned char* ring = smem + warp * kStages * stage;
  const uint32_t bar = smem_addr(&bars[warp][0]);
  const int swap = (lane >> 2) & 1;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const uint64_t policy = l2_policy_evict_first();
  grid_dependency_wait();
  allow_dependent_launch();

  // items: rows (NORM) or parts of rows; this warp's: first, first + step, ...
  const int64_t items = p.T * (NORM ? 1 : p.segs);
  const int64_t first = (int64_t)blockIdx.x * rpc + slot, step = (int64_t)gridDim.x * rpc;
  const int64_t mine = first < items ? (items - first - 1) / step + 1 : 0;
  auto place = [&](int64_t n, int64_t* row, int64_t* unit) {
    const int64_t item = first + n * step;
    *row = NORM ? item : item / p.segs;
    *unit = (NORM ? sub : item - *row * p.segs) * p.seg;
    return (int)min64(p.seg, p.ring_units - *unit);   // units; <= 0: nothing for this warp
  };
  auto issue = [&](int64_t n) {
    int64_t row, unit;
    const int units = place(n, &row, &unit);
    if (units <= 0 || lane != 0) return;
    const int s = (int)(n % kStages);
    mbar_arrive_expect_tx(bar + 8 * s, (uint32_t)units * 32 + (n == 0 ? p.missing_tx : 0u));
    bulk_g2s(smem_addr(ring) + s * stage, p.x + (row * p.ring_units + unit) * 16,
             (uint32_t)units * 32, bar + 8 * s, policy);
  };
  for (int64_t n = 0; n < min64(mine, kStages); ++n) issue(n);

  float gain[GAIN ? kHeldUnits / 32 : 1][2][8];   // halves in this lane's order
  if (GAIN)
#pragma unroll
    for (int i = 0; i < kHeldUnits / 32; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int u = sub * p.seg + 32 * i + lane;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (32 * i + lane < p.seg && u < p.units) {
          const float4* g = reinterpret_cast<const float4*>(p.gamma + 16 * u + 8 * (h ^ swap));
          a = __ldg(g);
          b = __ldg(g + 1);
        }
        gain[i][h][0] = a.x, gain[i][h][1] = a.y, gain[i][h][2] = a.z, gain[i][h][3] = a.w;
        gain[i][h][4] = b.x, gain[i][h][5] = b.y, gain[i][h][6] = b.z, gain[i][h][7] = b.w;
      }

  bool dead = false;   // a wait gave up: the rest runs on without data, its barriers met
  for (int64_t n = 0; n < mine; ++n) {
    int64_t row, unit;
    const int units = place(n, &row, &unit);
    const int s = (int)(n % kStages);
    if (units > 0 && !dead) {
      int ok = 1;
      if (lane == 0) {
        ok = mbar_wait_bounded(bar + 8 * s, (uint32_t)((n / kStages) & 1), p.wait_limit_ns);
        if (!ok) {
          atomicOr(&g_cast_status, kStatusTimeout);
          for (int64_t j = n; j < min64(mine, n + kStages); ++j)   // copies in flight land
            (void)mbar_wait_bounded(bar + 8 * (int)(j % kStages),
                                    (uint32_t)((j / kStages) & 1), p.wait_limit_ns);
        }
      }
      dead = __shfl_sync(0xFFFFFFFFu, ok, 0) == 0;
    }
    const unsigned char* x = ring + s * stage;
    float rinv = 1.f;
    if (NORM) {
      uint64_t q0 = 0, q1 = 0;
      for (int u = lane; u < units; u += 32) {
        const uint4 a = lds128(x + 32 * u + 16 * swap), b = lds128(x + 32 * u + 16 * (swap ^ 1));
        uint64_t f;
        f = bf16x2_to_f2(a.x), q0 = f2_fma(f, f, q0);
        f = bf16x2_to_f2(a.y), q1 = f2_fma(f, f, q1);
        f = bf16x2_to_f2(a.z), q0 = f2_fma(f, f, q0);
        f = bf16x2_to_f2(a.w), q1 = f2_fma(f, f, q1);
        f = bf16x2_to_f2(b.x), q0 = f2_fma(f, f, q0);
        f = bf16x2_to_f2(b.y), q1 = f2_fma(f, f, q1);
        f = bf16x2_to_f2(b.z), q0 = f2_fma(f, f, q0);
        f = bf16x2_to_f2(b.w), q1 = f2_fma(f, f, q1);
      }
      q0 = f2_add(q0, q1);
      float ss = warp_sum(f2_lo(q0) + f2_hi(q0));
      if (wpr > 1) {
        const int buf = (int)(n & 1);   // the other buffer's readers are past this barrier
        if (lane == 0) part[buf][warp] = ss;
        named_barrier(1 + slot, 32 * wpr);
        ss = 0.f;
        for (int w = 0; w < wpr; ++w) ss += part[buf][slot * wpr + w];
      }
      rinv = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
      if (p.rinv != nullptr && sub == 0 && lane == 0) p.rinv[row] = rinv;
    }
    uint8_t* codes = p.codes + (row * p.ring_units + unit) * 16;
    float* scales = p.scales + row * ((p.ring_units + 7) / 8) + unit / 8;
    const float* gamma = NORM && !GAIN && p.gamma != nullptr ? p.gamma + unit * 16 : nullptr;
    auto cast_unit = [&](int u, const float (&g)[2][8]) {
      const bool in = u < units;
      float f[2][8];   // the unit's halves: values 8 (h ^ swap) .. + 7
      float a = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int half = h ^ swap;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = lds128(x + 32 * u + 16 * half);
        bf16x8_to_f32(v, f[h]);
        if (GAIN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[h][j] *= g[h][j];
        } else if (gamma != nullptr && in) {
          const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma + 16 * u + 8 * half));
          const float4 g1 = __ldg(reinterpret_cast<const float4*>(gamma + 16 * u + 8 * half) + 1);
          f[h][0] *= g0.x, f[h][1] *= g0.y, f[h][2] *= g0.z, f[h][3] *= g0.w;
          f[h][4] *= g1.x, f[h][5] *= g1.y, f[h][6] *= g1.z, f[h][7] *= g1.w;
        }
        if (NORM)
#pragma unroll
          for (int j = 0; j < 8; ++j) f[h][j] *= rinv;
#pragma unroll
        for (int j = 0; j < 8; j += 2) a = fmax3(a, fabsf(f[h][j]), fabsf(f[h][j + 1]));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      const float scale = block_scale(a);
      const float inv = __frcp_rn(scale);
      uint2 c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        c[h] = make_uint2(
            cvt_e4m3x4(f[h][0] * inv, f[h][1] * inv, f[h][2] * inv, f[h][3] * inv),
            cvt_e4m3x4(f[h][4] * inv, f[h][5] * inv, f[h][6] * inv, f[h][7] * inv));
      if (in) {
        const uint2 lo = swap ? c[1] : c[0], hi = swap ? c[0] : c[1];
        __stcs(reinterpret_cast<uint4*>(codes + 16 * u), make_uint4(lo.x, lo.y, hi.x, hi.y));
        if ((lane & 7) == 0) scales[u >> 3] = scale;
      }
    };
    if (GAIN) {
#pragma unroll
      for (int i = 0; i < kHeldUnits / 32; ++i)
        if (32 * i < units) cast_unit(32 * i + lane, gain[i]);
      if (units > kHeldUnits) {
        float g[2][8] = {};
        const int u = kHeldUnits + lane;
        if (u < units)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4* at =
                reinterpret_cast<const float4*>(p.gamma + (unit + u) * 16 + 8 * (h ^ swap));
            const float4 a = __ldg(at), b = __ldg(at + 1);
            g[h][0] = a.x, g[h][1] = a.y, g[h][2] = a.z, g[h][3] = a.w;
            g[h][4] = b.x, g[h][5] = b.y, g[h][6] = b.z, g[h][7] = b.w;
          }
        cast_unit(u, g);
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < units; i += 32) cast_unit(i + lane, gain[0]);
    }
    fence_proxy_async_smem();   // the stage's reads come before the copy that refills it
    __syncwarp();
    if (!dead && n + kStages < mine) issue(n + kStages);
  }
}

// Weights in 128 x 128 blocks: one block per CTA, its 32 KB in the registers
// of 256 threads (four units each, eight threads along a row).
__global__ void __launch_bounds__(kCastThreads) blockcast_tiles_kernel(const CastParams p) {
  __shared__ float part[kCastWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tb = blockIdx.x / p.blocks;
  const int db = (int)(blockIdx.x - tb * p.blocks);
  const int u = 8 * db + (threadIdx.x & 7);
  grid_dependency_wait();
  allow_dependent_launch();
  uint4 x[4][2];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = tb * 128 + i * 32 + (threadIdx.x >> 3);
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (t < p.T && u < p.units) load16(x[i], p.x + t * p.D + 16 * u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[16];
    unpack16(x[i], f);
    a = fmaxf(a, absmax16(f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if (lane == 0) part[warp] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCastWarps; ++w) a = fmaxf(a, part[w]);
  const float scale = block_scale(a);
  const float inv = 1.0f / scale;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = tb * 128 + i * 32 + (threadIdx.x >> 3);
    if (t < p.T && u < p.units) {
      float f[16];
      unpack16(x[i], f);
      __stcs(reinterpret_cast<uint4*>(p.codes + t * p.D + 16 * u), codes16(f, inv));
    }
  }
  if (threadIdx.x == 0) p.scales[tb * p.blocks + db] = scale;
}

// The transpose in blocks of 128 tokens: a CTA takes 128 tokens x 64 columns.
// A thread holds four consecutive tokens of eight columns (four 16-byte
// loads; eight threads read the 128 bytes of a token), so the four codes of a
// column are one word of the transposed tile in shared memory, from where the
// codes leave in 16-byte pieces of a column's 128.  Pitch 33 words: the word
// reads of a column's pieces hit distinct banks.
constexpr int kTrCols = 64;
constexpr int kTrPitch = 33;

__global__ void __launch_bounds__(kCastThreads) blockcast_transpose_kernel(const CastParams p) {
  __shared__ uint32_t tile[kTrCols * kTrPitch];
  __shared__ float part[kCastWarps][kTrCols];
  __shared__ float inverse[kTrCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tb = blockIdx.y;
  const int c0 = (int)blockIdx.x * kTrCols;
  const int cg = lane & 7;                       // columns 8 cg .. 8 cg + 7
  const int tg = warp * 4 + (lane >> 3);         // tokens 4 tg .. 4 tg + 3
  const int col = c0 + 8 * cg;
  grid_dependency_wait();
  allow_dependent_launch();
  uint4 x[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t t = (int64_t)tb * 128 + 4 * tg + r;
    x[r] = make_uint4(0, 0, 0, 0);
    if (t < p.T && col < p.D) x[r] = __ldcs(reinterpret_cast<const uint4*>(p.x + t * p.D + col));
  }
  float f[4][8];
#pragma unroll
  for (int r = 0; r < 4; ++r) bf16x8_to_f32(x[r], f[r]);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a = fmaxf(fmaxf(fabsf(f[0][j]), fabsf(f[1][j])), fmaxf(fabsf(f[2][j]), fabsf(f[3][j])));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 8));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 16));
    if (lane < 8) part[warp][8 * cg + j] = a;
  }
  __syncthreads();
  if (threadIdx.x < kTrCols) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kCastWarps; ++w) a = fmaxf(a, part[w][threadIdx.x]);
    const float scale = block_scale(a);
    inverse[threadIdx.x] = 1.0f / scale;
    if (c0 + (int)threadIdx.x < p.D)
      p.scales[(int64_t)(c0 + threadIdx.x) * p.tblocks + tb] = scale;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float inv = inverse[8 * cg + j];
    tile[(8 * cg + j) * kTrPitch + tg] =
        cvt_e4m3x4(f[0][j] * inv, f[1][j] * inv, f[2][j] * inv, f[3][j] * inv);
  }
  __syncthreads();
  // 64 columns x 8 pieces of 16 codes, two per thread
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = threadIdx.x + k * kCastThreads;
    const int c = i >> 3, piece = i & 7;
    const int64_t t = (int64_t)tb * 128 + 16 * piece;
    if (c0 + c < p.D && t < p.pitch) {
      const uint32_t* w = tile + c * kTrPitch + 4 * piece;
      __stcs(reinterpret_cast<uint4*>(p.codes + (int64_t)(c0 + c) * p.pitch + t),
             make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

using CastKernel = void (*)(CastParams);

CastKernel pick_norm(int upt) {
  switch (upt) {
    case 1: return blockcast_rows_kernel<1, true>;
    case 2: return blockcast_rows_kernel<2, true>;
    case 4: return blockcast_rows_kernel<4, true>;
    default: return blockcast_rows_kernel<8, true>;
  }
}

CastKernel pick_plain(int upt) {
  switch (upt) {
    case 1: return blockcast_rows_kernel<1, false>;
    case 2: return blockcast_rows_kernel<2, false>;
    default: return blockcast_rows_kernel<4, false>;
  }
}

int launch(CastKernel kern, dim3 grid, const CastParams& p, cudaStream_t stream, bool pdl,
           size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kCastThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return fail_cuda(e, "launching the block-128 cast");
  return NTS_OK;
}

}  // namespace

int launch_blockcast(const BlockcastRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  CastParams p = {};
  p.x = static_cast<const __nv_bfloat16*>(rq.X);
  p.gamma = rq.gamma;
  p.codes = rq.codes;
  p.scales = rq.scales;
  p.rinv = rq.rinv;
  p.T = rq.T;
  p.D = (int)rq.D;
  p.units = p.D / 16;
  p.blocks = (int)((rq.D + 127) / 128);
  p.eps = rq.eps;
  p.inv_d = 1.0f / (float)p.D;
  const int64_t tblocks = (p.T + 127) / 128;
  if (rq.kind == kCastTiles && tblocks > 0x7fffffffll / p.blocks)
    return fail(NTS_ERR_UNSUPPORTED, "too many 128 x 128 blocks in one call");
  if (rq.kind == kCastTranspose && tblocks > 65535)
    return fail(NTS_ERR_UNSUPPORTED, "more than 65535 blocks of tokens");
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  note_launch(kCastUnit);

  if (rq.kind == kCastTiles) {
    log_launch("blockcast", "T=%lld D=%d 128x128", (long long)p.T, p.D);
    return launch(blockcast_tiles_kernel, dim3((unsigned)(tblocks * p.blocks)), p, stream,
                  tune.pdl != 0);
  }
  if (rq.kind == kCastTranspose) {
    p.pitch = (p.T + 15) / 16 * 16;
    p.tblocks = (int)tblocks;
    log_launch("blockcast_t", "T=%lld D=%d", (long long)p.T, p.D);
    return launch(blockcast_transpose_kernel,
                  dim3((unsigned)((rq.D + kTrCols - 1) / kTrCols), (unsigned)tblocks), p, stream,
                  tune.pdl != 0);
  }

  // Many rows: the ring.  Parts of rows below 2 KB cost more to hand out than to
  // load ([32768, 512] 12.1 us direct, 14.9 by the ring).
  const bool norm = rq.kind == kCastNorm;
  const bool flat = !norm && rq.D % 128 == 0;   // one long row: no block ends early
  const int64_t units = flat ? rq.T * (rq.D / 16) : p.units;
  if (tune.force_stages > 0 || (rq.T * rq.D >= (norm ? kNormRingValues : kRingValues) && units >= 64)) {
    p.ring_units = units;
    if (flat) p.T = 1;
    p.wpr = 1;
    if (norm)
      while (p.wpr < kCastWarps && p.units > p.wpr * kPartUnits) p.wpr *= 2;
    const int64_t per = norm ? (p.units + p.wpr - 1) / p.wpr : std::min<int64_t>(units, kHeldUnits);
    p.seg = (int)((per + 7) / 8 * 8);
    const int64_t segs = (units + p.seg - 1) / p.seg;
    if (!norm && segs >= (1ll << 31)) return fail(NTS_ERR_UNSUPPORTED, "matrix too large");
    p.segs = (int)segs;
    p.wait_limit_ns = tune.wait_limit_ns;
    p.missing_tx = tune.missing_tx;
    const size_t smem = (size_t)kCastWarps * kStages * p.seg * 32;
    const bool gain = norm && p.gamma != nullptr && p.seg <= kPartUnits;   // D <= 20480
    const CastKernel kern = gain   ? blockcast_ring_kernel<true, true>
                            : norm ? blockcast_ring_kernel<true, false>
                                   : blockcast_ring_kernel<false, false>;
    int per_sm = 0;
    int rc = prepare_kernel((const void*)kern, smem);
    if (rc == NTS_OK) rc = blocks_per_sm((const void*)kern, kCastThreads, smem, &per_sm);
    if (rc != NTS_OK) return rc;
    const int rpc = kCastWarps / p.wpr;
    const int64_t need = (p.T * (norm ? 1 : segs) + rpc - 1) / rpc;
    const unsigned grid = (unsigned)std::min<int64_t>(need, (int64_t)per_sm * dev.sm_count);
    log_launch(norm ? "rmsnorm_blockcast" : "blockcast", "T=%lld D=%d ring seg=%d wpr=%d grid=%u",
               (long long)rq.T, p.D, p.seg, p.wpr, grid);
    return launch(kern, dim3(grid), p, stream, tune.pdl != 0, smem);
  }

  int upt;
  int64_t ctas;
  if (norm) {
    // The fewest units per thread that still fill the GPU: more threads per
    // row while the rows alone leave SMs idle.
    p.wpr = 1;
    while (p.wpr < kCastWarps && p.wpr * 32 * 8 < p.units) p.wpr *= 2;
    while (p.wpr < kCastWarps && p.wpr * 32 < p.units && p.T * p.wpr < (int64_t)dev.sm_count * 32)
      p.wpr *= 2;
    const int per = (p.units + p.wpr * 32 - 1) / (p.wpr * 32);
    upt = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 8;
    const int rpc = kCastWarps / p.wpr;
    ctas = (p.T + rpc - 1) / rpc;
  } else {
    upt = p.units <= 32 ? 1 : p.units <= 64 ? 2 : 4;
    p.segs = (p.units + 32 * upt - 1) / (32 * upt);
    ctas = (p.T * p.segs + kCastWarps - 1) / kCastWarps;
  }
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, 1 << 24);
  log_launch(norm ? "rmsnorm_blockcast" : "blockcast",
             "T=%lld D=%d upt=%d wpr=%d segs=%d grid=%u", (long long)p.T, p.D, upt, p.wpr, p.segs,
             grid);
  return launch(norm ? pick_norm(upt) : pick_plain(upt), dim3(grid), p, stream,
                tune.pdl != 0);
}

int read_and_clear_cast_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_cast_status, sizeof(v));
  if (e != cudaSuccess) return fail_cuda(e, "reading the cast's status word");
  if (v != 0) e = cudaMemcpyToSymbol(g_cast_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return fail_cuda(e, "clearing the cast's status word");
  *out = v;
  return NTS_OK;
}

}  // namespace nts
