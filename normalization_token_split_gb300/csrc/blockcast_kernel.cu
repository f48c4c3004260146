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
// All of these are bound by HBM: 2 bytes read and 1 + 4/128 written per value.
#include <cuda_runtime.h>

#include <algorithm>

#include "nts_device.cuh"
#include "nts_internal.h"

namespace nts {

namespace {

constexpr int kCastThreads = 256;
constexpr int kCastWarps = kCastThreads / 32;

__device__ __forceinline__ float block_scale(float a) { return fmaxf(a, 0x1p-100f) / 448.0f; }

// 16 bf16 (two 16-byte loads; p is 16-byte aligned).
__device__ __forceinline__ void load16(uint4 (&v)[2], const __nv_bfloat16* p) {
  v[0] = __ldcs(reinterpret_cast<const uint4*>(p));
  v[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
}

__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float (&f)[16]) {
  float a[8], b[8];
  bf16x8_to_f32(v[0], a);
  bf16x8_to_f32(v[1], b);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = a[j];
    f[8 + j] = b[j];
  }
}

__device__ __forceinline__ float absmax16(const float (&f)[16]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2) m = fmax3(m, fabsf(f[j]), fabsf(f[j + 1]));
  return m;
}

__device__ __forceinline__ uint4 codes16(const float (&f)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = cvt_e4m3x4(f[4 * j] * inv, f[4 * j + 1] * inv, f[4 * j + 2] * inv, f[4 * j + 3] * inv);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

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

int launch(CastKernel kern, dim3 grid, const CastParams& p, cudaStream_t stream, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kCastThreads);
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
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
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

  if (rq.kind == kCastTiles) {
    if (tblocks > 0x7fffffffll / p.blocks)
      return fail(NTS_ERR_UNSUPPORTED, "too many 128 x 128 blocks in one call");
    log_launch("blockcast", "T=%lld D=%d 128x128", (long long)p.T, p.D);
    return launch(blockcast_tiles_kernel, dim3((unsigned)(tblocks * p.blocks)), p, stream,
                  tune.pdl != 0);
  }
  if (rq.kind == kCastTranspose) {
    if (tblocks > 65535) return fail(NTS_ERR_UNSUPPORTED, "more than 65535 blocks of tokens");
    p.pitch = (p.T + 15) / 16 * 16;
    p.tblocks = (int)tblocks;
    log_launch("blockcast_t", "T=%lld D=%d", (long long)p.T, p.D);
    return launch(blockcast_transpose_kernel,
                  dim3((unsigned)((rq.D + kTrCols - 1) / kTrCols), (unsigned)tblocks), p, stream,
                  tune.pdl != 0);
  }

  int upt;
  int64_t ctas;
  if (rq.kind == kCastNorm) {
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
  log_launch(rq.kind == kCastNorm ? "rmsnorm_blockcast" : "blockcast",
             "T=%lld D=%d upt=%d wpr=%d segs=%d grid=%u", (long long)p.T, p.D, upt, p.wpr, p.segs,
             grid);
  return launch(rq.kind == kCastNorm ? pick_norm(upt) : pick_plain(upt), dim3(grid), p, stream,
                tune.pdl != 0);
}

}  // namespace nts
