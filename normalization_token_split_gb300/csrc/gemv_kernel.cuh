// gemv_kernel.cuh -- the kernel of the products with 4-bit weights (gemv_launch.cu
// describes it); instantiated in gemv_e2m1.cu and gemv_int4.cu.
#pragma once

#include <cuda_runtime.h>

#include "block_device.cuh"
#include "gemv_internal.h"

namespace nts {

namespace {

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
template <int SIZE>
__device__ __forceinline__ void copy_async_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes),
               "n"(SIZE)
               : "memory");
}

// Eight codes as four pairs of fp16.  E2M1: pair j holds values 2j and 2j + 1, by the
// hardware's conversion.  int4: values j and j + 4, a code's four bits put under the
// exponent of 1024 (or 64, where they stand four bits higher) and the offset taken off.
template <bool INT4>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (INT4) {
    const uint32_t v = w >> 8;
    const uint32_t a = (w & 0x000F000Fu) ^ 0x64086408u, b = (w & 0x00F000F0u) ^ 0x54805480u;
    const uint32_t c = (v & 0x000F000Fu) ^ 0x64086408u, d = (v & 0x00F000F0u) ^ 0x54805480u;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[0]) : "r"(a), "r"(0xE408E408u));   // -1032
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[1]) : "r"(b), "r"(0xD480D480u));   // -72
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[2]) : "r"(c), "r"(0xE408E408u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[3]) : "r"(d), "r"(0xD480D480u));
  } else {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
  }
}

// Four 8 x 16-byte matrices, one 4-byte word of row g of each per lane (g, t); lanes
// 8 i .. 8 i + 7 give the rows' addresses of matrix i.
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}

// d = A B + c: rows g and g + 8 of A by lanes (g, t), column g of B.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// Eight values in pairs (0, 1), (2, 3), .. as (0, 4), (1, 5), ..
__device__ __forceinline__ void by_fours(uint32_t (&p)[4]) {
  const uint32_t a = __byte_perm(p[0], p[2], 0x5410), b = __byte_perm(p[0], p[2], 0x7632);
  const uint32_t c = __byte_perm(p[1], p[3], 0x5410), d = __byte_perm(p[1], p[3], 0x7632);
  p[0] = a, p[1] = b, p[2] = c, p[3] = d;
}

// A warp's chunk of A as B fragments: frag[sub-block of 32][tile of 8 rows], and per
// block of 128 and tile the factors of the lane's two columns of a product.  First the
// loads alone, as the rows lie in memory (eight values of a row to a lane), so that they
// go out before the copies of the weights; then what the products take.
template <int NT>
__device__ __forceinline__ void load_rows(const GemvParams& p, int m0, int k0,
                                          uint32_t (&frag)[kGemvChunk / 32][NT][4],
                                          float (&factor)[kGemvChunk / 128][NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int end = min(p.M, m0 + p.per);
  if (p.a_scales == nullptr) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int m = m0 + 8 * j + g;
      const __nv_bfloat16* row =
          static_cast<const __nv_bfloat16*>(p.a) + m * p.lda + k0 + 8 * t;
#pragma unroll
      for (int i = 0; i < kGemvChunk / 32; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (m < end && k0 + 32 * i < p.K) x = __ldg(reinterpret_cast<const uint4*>(row + 32 * i));
        frag[i][j][0] = x.x, frag[i][j][1] = x.y, frag[i][j][2] = x.z, frag[i][j][3] = x.w;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = m0 + 8 * j + g;
    const uint8_t* row = static_cast<const uint8_t*>(p.a) + m * p.lda + k0 + 8 * t;
#pragma unroll
    for (int i = 0; i < kGemvChunk / 32; ++i) {
      uint2 x = make_uint2(0, 0);
      if (m < end && k0 + 32 * i < p.K) x = __ldg(reinterpret_cast<const uint2*>(row + 32 * i));
      frag[i][j][0] = x.x, frag[i][j][1] = x.y;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int b = 0; b < kGemvChunk / 128; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = m0 + 8 * j + 2 * t + i, block = k0 / 128 + b;
        factor[b][j][i] =
            col < end && block < p.kb ? __ldg(p.a_scales + (int64_t)col * p.kb + block) : 0.f;
      }
}

template <bool INT4, int NT>
__device__ __forceinline__ void convert_bf16(uint32_t (&frag)[kGemvChunk / 32][NT][4],
                                             float (&factor)[kGemvChunk / 128][NT][2]) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int b = 0; b < kGemvChunk / 128; ++b) {
      uint32_t most2 = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) most2 = bf16x2_absmax(most2, frag[4 * b + i / 4][j][i % 4]);
      float most = bf16x2_hmax_abs(most2);
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // 2^f: the largest comes to [2^14, 2^15), as far as 2^f and 2^-f are normal.  128 of
      // them by codes of up to 8 come to 2^25 at most, so group scales of 2^102 fit before
      // 2^-f takes it off again.
      const int f = max(-113, min(126, 141 - (int)(__float_as_uint(most) >> 23)));
      const float up = __uint_as_float((uint32_t)(127 + f) << 23);
      const float down = __uint_as_float((uint32_t)(127 - f) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t(&q)[4] = frag[4 * b + i][j];
        float v[8];
        bf16x8_to_f32(make_uint4(q[0], q[1], q[2], q[3]), v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[e] = INT4 ? pack_f16x2(v[e] * up, v[e + 4] * up)
                      : pack_f16x2(v[2 * e] * up, v[2 * e + 1] * up);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)   // column 2t + i is row 2t + i of A, of lanes (2t + i, .)
        factor[b][j][i] = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4 * i);
    }
}

template <bool INT4, int NT>
__device__ __forceinline__ void convert_e4m3(uint32_t (&frag)[kGemvChunk / 32][NT][4]) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < kGemvChunk / 32; ++i) {
      uint32_t(&f)[4] = frag[i][j];
      f[3] = e4m3x2_to_f16x2(f[1] >> 16), f[2] = e4m3x2_to_f16x2(f[1]);
      f[1] = e4m3x2_to_f16x2(f[0] >> 16), f[0] = e4m3x2_to_f16x2(f[0]);
      if (INT4) by_fours(f);
    }
}

template <bool INT4, int G, int NT>
__global__ void __launch_bounds__(32 * kMaxGemvWarps, 1) gemv_kernel(const GemvParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kChunk = kGemvChunk, kStages = kGemvStages;
  constexpr int kSubs = kChunk / 32;             // 16-byte pieces of a row's chunk of codes
  constexpr int kPer = kChunk / G;               // scales of a row's chunk
  constexpr int kCodes = kGemvRows * kChunk / 2;
  constexpr int kCopies = kGemvRows * kSubs / 32;   // of 16 bytes, per lane and tile
  constexpr int kStep = 32 / kSubs;              // rows of one copy of the warp
  static_assert(kSubs == 8, "a row's chunk is a line of 128 bytes");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  // Shared memory: stages [warps][stages] of codes and scales of 32 rows, the warps' sums
  // of a batch of tiles [batch][warps][2 halves][NT][16 rows][8], and across the cluster
  // the sums of the slice [8 NT][32 tiles]
  constexpr int kOuts = 8 * NT * kGemvRows;
  unsigned char* ring = smem + warp * kStages * p.stage_bytes;
  float* red = reinterpret_cast<float*>(smem + p.warps * kStages * p.stage_bytes);
  float* total = red + p.batch * p.warps * kOuts;

  const int slice = blockIdx.x / p.cluster;
  const int rank = blockIdx.x - slice * p.cluster;
  const int n0 = (int)((int64_t)p.N * slice / p.slices);
  const int rows = (int)((int64_t)p.N * (slice + 1) / p.slices) - n0;
  const int tiles = (rows + kGemvRows - 1) / kGemvRows;
  const int m0 = blockIdx.y * p.per;
  const int chunk = rank * p.warps + warp;       // of K
  const int k0 = chunk * kChunk;
  const bool live = chunk < p.chunks;

  // One tile's codes and scales into a stage.  A row's pieces change places with the
  // row's number, so that the eight rows that a warp reads at once meet distinct banks.
  const int row0 = lane / kSubs, piece = lane % kSubs;
  const int64_t pitch = p.K / 2;
  const unsigned char* codes = p.w + (n0 + row0) * pitch + k0 / 2 + 16 * piece;
  const __nv_bfloat16* scales = p.s + (int64_t)(n0 + lane) * p.groups + chunk * kPer;
  const int bytes = k0 + 32 * piece < p.K ? 16 : 0;
  const uint32_t to = smem_addr(ring) + row0 * kSubs * 16 + (piece ^ row0) * 16;
  auto stage = [&](int tile, uint32_t at) {
    if (live && tile < tiles) {
      const int left = rows - kGemvRows * tile;
      const unsigned char* from = codes;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        // rows four apart differ in the third bit of what their pieces change by
        const uint32_t dst = (i % 2 ? to ^ 64u : to) + 512 * i;
        copy_async16(dst + at, from, row0 + i * kStep < left ? bytes : 0);
        from += kStep * pitch;
      }
      codes = from;
      const uint32_t into = smem_addr(ring) + at + kCodes;
      if (p.vector) {
        const int n = lane < left ? 2 * kPer : 0;
        if constexpr (kPer == 8)
          copy_async16(into + lane * p.scale_pitch, scales, n);
        else
          copy_async_small<2 * kPer>(into + lane * p.scale_pitch, scales, n);
        scales += (int64_t)kGemvRows * p.groups;
      } else {
        // words that hold them, from the word of the first; nothing beyond the last
        const int have = min(kPer, p.groups - chunk * kPer);
        for (int q = lane; q < kGemvRows * 8; q += 32) {
          const int row = q >> 3, word = q & 7;
          if (4 * word >= p.scale_pitch) continue;
          const int64_t first =
              (int64_t)(n0 + kGemvRows * tile + row) * p.groups + chunk * kPer;
          const int n = row < left
                            ? (int)max64(0, min64(4, 2 * (first + have) - (4 * (first / 2) + 4 * word)))
                            : 0;
          copy_async_small<4>(into + row * p.scale_pitch + 4 * word,
                              n > 0 ? p.s + 2 * (first / 2) + 2 * word : p.s, n);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  grid_dependency_wait();
  allow_dependent_launch();
  uint32_t frag[kSubs][NT][4];
  float factor[kChunk / 128][NT][2];
  load_rows<NT>(p, m0, k0, frag, factor);
#pragma unroll
  for (int s = 0; s < kStages; ++s) stage(s, s * p.stage_bytes);
  if (p.a_scales != nullptr)
    convert_e4m3<INT4, NT>(frag);
  else
    convert_bf16<INT4, NT>(frag, factor);

  const int summed = min(p.warps, p.chunks - rank * p.warps);   // warps with a chunk
  // Row and piece of the matrix rows whose addresses this lane gives: matrices 0 and 1
  // are rows 0 to 7 and 8 to 15 of an even sub-block, 2 and 3 of the odd one behind it.
  const uint32_t matrices =
      smem_addr(ring) + (lane & 15) * kSubs * 16 + ((lane >> 4) ^ (lane & 7)) * 16;
  // Halves of a tile and sub-blocks whose products are formed side by side: independent
  // sums for the tensor pipe, as far as registers go.
  constexpr int kHalves = NT == 1 ? 2 : 1;
  uint32_t at = 0;
  int slot = 0;   // of the batch
  for (int tile = 0; tile < tiles; ++tile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    if (live) {
#pragma unroll
      for (int half = 0; half < 2; half += kHalves) {
        if (kHalves == 1 && rows <= kGemvRows * tile + 16 * half) break;
        float acc[kHalves][NT][4];
#pragma unroll
        for (int b = 0; b < kChunk / 128; ++b) {
          constexpr int kGroups = 128 / G;
          // the block's scales of rows g and g + 8
          float sc[kHalves][2][kGroups];
#pragma unroll
          for (int h = 0; h < 2 * kHalves; ++h) {
            const int row = 16 * half + g + 8 * h;
            const unsigned char* from = ring + at + kCodes + row * p.scale_pitch;
            float(&v)[kGroups] = sc[h / 2][h % 2];
            if (p.vector) {
              if constexpr (kGroups == 4) {
                const uint2 w = lds64(from + 8 * b);
                v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
                v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
              } else if constexpr (kGroups == 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(from + 4 * b);
                v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xFFFF0000u);
              } else {
                v[0] = __uint_as_float(
                    (uint32_t)*reinterpret_cast<const uint16_t*>(from + 2 * b) << 16);
              }
            } else {
              const int odd = (int)(((int64_t)(n0 + kGemvRows * tile + row) * p.groups +
                                     chunk * kPer) & 1);
#pragma unroll
              for (int i = 0; i < kGroups; ++i)
                v[i] = __uint_as_float(
                    (uint32_t)reinterpret_cast<const uint16_t*>(from)[odd + kGroups * b + i] << 16);
            }
          }
          float d[kHalves][NT][4], c[kHalves][2][NT][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {   // pairs of sub-blocks
            uint32_t w[kHalves][4];
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              load_matrices(((matrices + at) ^ (16u * (4 * b + 2 * i))) +
                                (half + h) * (16 * kSubs * 16), w[h]);
            uint32_t lo[kHalves][2][4], hi[kHalves][2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int h = 0; h < kHalves; ++h) {
                decode8<INT4>(w[h][2 * s], lo[h][s]);
                decode8<INT4>(w[h][2 * s + 1], hi[h][s]);
              }
            const bool opens = G <= 64 || i == 0;   // the pair opens its group or groups
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                  for (int j = 0; j < NT; ++j) {
                    const uint32_t(&f)[4] = frag[4 * b + 2 * i + s][j];
                    const uint32_t(&l)[4] = lo[h][s], (&u)[4] = hi[h][s];
                    float(&x)[4] = c[h][s][j];
                    if (k == 0 && opens)
                      mma_f16(x, l[0], u[0], l[1], u[1], f[0], f[1], 0.f, 0.f, 0.f, 0.f);
                    else
                      mma_f16(x, l[2 * k], u[2 * k], l[2 * k + 1], u[2 * k + 1], f[2 * k],
                              f[2 * k + 1], x[0], x[1], x[2], x[3]);
                  }
            // groups that end here, into the block's sums
#pragma unroll
            for (int s = G == 32 ? 0 : 1; s < 2; ++s) {
              if (32 * (2 * i + s + 1) % G != 0) continue;
              const int grp = 32 * (2 * i + s) / G;
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float v = G == 32 ? c[h][s][j][e] : c[h][0][j][e] + c[h][1][j][e];
                    d[h][j][e] = grp == 0 ? v * sc[h][e >> 1][grp]
                                          : fmaf(v, sc[h][e >> 1][grp], d[h][j][e]);
                  }
            }
          }
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[h][j][e] = b == 0 ? d[h][j][e] * factor[b][j][e & 1]
                                      : fmaf(d[h][j][e], factor[b][j][e & 1], acc[h][j][e]);
        }
        float* mine = red + (slot * p.warps + warp) * kOuts + half * (kOuts / 2);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              *reinterpret_cast<float2*>(mine + h * (kOuts / 2) + (16 * j + g + 4 * e) * 8 + 2 * t) =
                  make_float2(acc[h][j][e], acc[h][j][e + 1]);
      }
    }
    __syncwarp();   // the stage is read by all before the next copy into it
    stage(tile + kStages, at);
    at += p.stage_bytes;
    if (at == (uint32_t)(kStages * p.stage_bytes)) at = 0;
    if (++slot < p.batch && tile + 1 < tiles) continue;

    // the batch's sums over the warps, four columns of a row of W at a time
    __syncthreads();
    for (int o = threadIdx.x; o < slot * (kOuts / 4); o += blockDim.x) {
      const int b = o / (kOuts / 4), q = o % (kOuts / 4);
      const int half = q / (kOuts / 8), f = q % (kOuts / 8);
      const int m = f / 32 * 8 + f % 2 * 4;
      const int r = kGemvRows * (tile + 1 - slot + b) + 16 * half + f % 32 / 2;
      if (m0 + m >= p.M || r >= rows) continue;
      const float4* from = reinterpret_cast<const float4*>(red + b * p.warps * kOuts) + q;
      float v[4] = {};
#pragma unroll 4
      for (int w = 0; w < summed; ++w) {
        const float4 x = from[w * (kOuts / 4)];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.cluster > 1) {
          total[(m + e) * kGemvRows * tiles + r] = v[e];
        } else if (m0 + m + e < p.M) {
          const int64_t out = (int64_t)(m0 + m + e) * p.N + n0 + r;
          if (p.fp32)
            static_cast<float*>(p.y)[out] = v[e];
          else
            static_cast<__nv_bfloat16*>(p.y)[out] = __float2bfloat16_rn(v[e]);
        }
      }
    }
    slot = 0;
    if (tile + 1 < tiles) __syncthreads();   // read by all before the next batch
  }
  if (p.cluster == 1) return;

  // The sums of the cluster's CTAs, in their order: each takes a share of the slice.
  cluster_arrive_release();
  cluster_wait_acquire();
  const int count = rows * 8 * NT;
  for (int i = rank * blockDim.x + threadIdx.x; i < count; i += p.cluster * blockDim.x) {
    // neighbouring threads take neighbouring columns of a row of Y
    const int m = i / rows, r = i - m * rows;
    if (m0 + m >= p.M) break;
    const uint32_t from = smem_addr(total + m * kGemvRows * tiles + r);
    float v = 0.f;
    for (int c = 0; c < p.cluster; ++c) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_to_rank(from, c)) : "memory");
      v += x;
    }
    const int64_t out = (int64_t)(m0 + m) * p.N + n0 + r;
    if (p.fp32)
      static_cast<float*>(p.y)[out] = v;
    else
      static_cast<__nv_bfloat16*>(p.y)[out] = __float2bfloat16_rn(v);
  }
  cluster_arrive_release();   // no CTA ends while another reads its sums
  cluster_wait_acquire();
}

template <bool INT4, int G>
GemvKernel pick_tiles(int nt) {
  return nt == 1 ? gemv_kernel<INT4, G, 1> : gemv_kernel<INT4, G, 2>;
}

}  // namespace

template <bool INT4>
GemvKernel pick_gemv(int group, int nt) {
  return group == 32   ? pick_tiles<INT4, 32>(nt)
         : group == 64 ? pick_tiles<INT4, 64>(nt)
                       : pick_tiles<INT4, 128>(nt);
}

}  // namespace nts
