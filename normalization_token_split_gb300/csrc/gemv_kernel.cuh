// gemv_kernel.cuh -- the kernel of the products with 4-bit weights (gemv_launch.cu
// describes it); instantiated in gemv_{bf16,e4m3}_{e2m1,int4}.cu.
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

// Eight codes in the operand type of the products.  fp16 (four pairs): E2M1's pair j
// holds values 2j and 2j + 1, by the hardware's conversion; int4's values j and j + 4, a
// code's four bits put under the exponent of 1024 (or 64, where they stand four bits
// higher) and the offset taken off.  E4M3 (two fours): the even values, then the odd
// ones.  E2M1's bits under E4M3's bias are the values times 2^-6, subnormal ones too;
// int4's plus eight, 0 to 15, are as bits of E4M3 themselves times 2^-9.
template <bool E4M3, bool INT4>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&p)[E4M3 ? 2 : 4]) {
  if constexpr (E4M3 && INT4) {
    p[0] = (w & 0x0F0F0F0Fu) ^ 0x08080808u;
    p[1] = (w >> 4 & 0x0F0F0F0Fu) ^ 0x08080808u;
  } else if constexpr (E4M3) {
    p[0] = (w << 2 & 0x1C1C1C1Cu) | (w << 4 & 0x80808080u);
    p[1] = (w >> 2 & 0x1C1C1C1Cu) | (w & 0x80808080u);
  } else if constexpr (INT4) {
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
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint64_t e4m3x4_sum(uint32_t v, uint64_t s) {
  s = f2_add(s, e4m3x2_to_f2((uint16_t)v));
  return f2_add(s, e4m3x2_to_f2((uint16_t)(v >> 16)));
}

// Registers of a lane's part of 32 values of one row of A.
__host__ __device__ constexpr int frag_of(bool e4m3) { return e4m3 ? 2 : 4; }

// A warp's chunk of A as B fragments: frag[sub-block of 32][tile of 8 rows], and per
// block of 128 and tile the factors of the lane's two columns of a product.
template <bool INT4, int NT>
__device__ __forceinline__ void load_bf16(const GemvParams& p, int m0, int k0,
                                          uint32_t (&frag)[chunk_of(false, NT) / 32][NT][4],
                                          float (&factor)[chunk_of(false, NT) / 128][NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int end = min(p.M, m0 + p.per);
  // every load is issued before the first is used
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < chunk_of(false, NT) / 32; ++i) {
      const int m = m0 + 8 * j + g, k = k0 + 32 * i;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (m < end && k < p.K)
        x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a) +
                                                 m * p.lda + k + 8 * t));
      frag[i][j][0] = x.x, frag[i][j][1] = x.y, frag[i][j][2] = x.z, frag[i][j][3] = x.w;
    }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int b = 0; b < chunk_of(false, NT) / 128; ++b) {
      uint32_t most2 = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) most2 = bf16x2_absmax(most2, frag[4 * b + i / 4][j][i % 4]);
      float most = bf16x2_hmax_abs(most2);
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // 2^f: the largest comes to [2^14, 2^15), as far as 2^f and 2^-f are normal
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

// int4: also eight times the sums of A over each group, times the 2^-9 of the codes, into
// sums[group of the chunk][8 NT]: what the products are too large by.
template <bool INT4, int G, int NT>
__device__ __forceinline__ void load_e4m3(const GemvParams& p, int m0, int k0,
                                          uint32_t (&frag)[chunk_of(true, NT) / 32][NT][2],
                                          float (&factor)[chunk_of(true, NT) / 128][NT][2],
                                          float* sums) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int end = min(p.M, m0 + p.per);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < chunk_of(true, NT) / 32; ++i) {
      const int m = m0 + 8 * j + g, k = k0 + 32 * i;
      uint2 x = make_uint2(0, 0);
      if (m < end && k < p.K)
        x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.a) + m * p.lda + k +
                                                 8 * t));
      frag[i][j][0] = x.x, frag[i][j][1] = x.y;
    }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < chunk_of(true, NT) / 32; ++i) {
      const uint2 x = make_uint2(frag[i][j][0], frag[i][j][1]);
      frag[i][j][0] = __byte_perm(x.x, x.y, 0x6420);
      frag[i][j][1] = __byte_perm(x.x, x.y, 0x7531);
      if constexpr (INT4) {
        sum = e4m3x4_sum(x.y, e4m3x4_sum(x.x, sum));
        if (32 * (i + 1) % G == 0) {
          float v = f2_lo(sum) + f2_hi(sum);
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
          if (t == 0) sums[32 * i / G * 8 * NT + 8 * j + g] = v * -0x1p-6f;
          sum = 0;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < chunk_of(true, NT) / 128; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = m0 + 8 * j + 2 * t + i, block = k0 / 128 + b;
        factor[b][j][i] =
            col < end && block < p.kb ? __ldg(p.a_scales + (int64_t)col * p.kb + block) : 0.f;
      }
  }
  if (INT4) __syncwarp();
}

template <bool E4M3, bool INT4, int G, int NT>
__global__ void __launch_bounds__(32 * kMaxGemvWarps, 1) gemv_kernel(const GemvParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kChunk = chunk_of(E4M3, NT), kStages = stages_of(E4M3, NT);
  constexpr int kSubs = kChunk / 32;             // 16-byte pieces of a row's chunk of codes
  constexpr int kPer = kChunk / G;               // scales of a row's chunk
  constexpr int kCodes = kGemvRows * kChunk / 2;
  constexpr int kCopies = kGemvRows * kSubs / 32;   // of 16 bytes, per lane and tile
  constexpr int kFrag = frag_of(E4M3);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * kStages * p.stage_bytes;
  // the warps' sums of a batch of tiles [batch][warps][NT][16 rows][8]; int4 by E4M3: the
  // groups' sums of A; across the cluster [8 NT][16 tiles]
  float* red = reinterpret_cast<float*>(smem + p.warps * kStages * p.stage_bytes);
  constexpr int kOuts = 8 * NT * kGemvRows;
  float* sums = red + p.batch * p.warps * kOuts + warp * (E4M3 && INT4 ? kPer * 8 * NT : 0);
  float* total = red + p.batch * p.warps * kOuts + p.warps * (E4M3 && INT4 ? kPer * 8 * NT : 0);

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
  constexpr int kStep = 32 / kSubs;              // rows of one copy of the warp
  const int turn = kSubs == 8 ? row0 : row0 >> 1 & 3;
  const int64_t pitch = p.K / 2;
  const unsigned char* codes = p.w + (n0 + row0) * pitch + k0 / 2 + 16 * piece;
  const __nv_bfloat16* scales = p.s + (int64_t)(n0 + lane) * p.groups + chunk * kPer;
  const int bytes = k0 + 32 * piece < p.K ? 16 : 0;
  const uint32_t to = smem_addr(ring) + row0 * kSubs * 16 + (piece ^ turn) * 16;
  auto stage = [&](int tile, uint32_t at) {
    if (live && tile < tiles) {
      const int left = rows - kGemvRows * tile;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        // with eight pieces a row, rows four apart differ in the turn's third bit
        const uint32_t dst = (kSubs == 8 && i % 2 ? to ^ 64u : to) + 512 * i;
        copy_async16(dst + at, codes + i * kStep * pitch, row0 + i * kStep < left ? bytes : 0);
      }
      codes += kGemvRows * pitch;
      if (p.vector) {
        if (lane < kGemvRows) {
          const uint32_t dst = smem_addr(ring) + at + kCodes + lane * p.scale_pitch;
          const int n = lane < left ? 2 * kPer : 0;
          if constexpr (kPer == 8)
            copy_async16(dst, scales, n);
          else if constexpr (kPer >= 2)
            copy_async_small<2 * kPer>(dst, scales, n);
        }
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
          copy_async_small<4>(smem_addr(ring) + at + kCodes + row * p.scale_pitch + 4 * word,
                              n > 0 ? p.s + 2 * (first / 2) + 2 * word : p.s, n);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  grid_dependency_wait();
  allow_dependent_launch();
  for (int s = 0; s < kStages; ++s) stage(s, s * p.stage_bytes);

  uint32_t frag[kSubs][NT][kFrag];
  float factor[kChunk / 128][NT][2];
  if constexpr (E4M3)
    load_e4m3<INT4, G, NT>(p, m0, k0, frag, factor, sums);
  else
    load_bf16<INT4, NT>(p, m0, k0, frag, factor);

  const int summed = min(p.warps, p.chunks - rank * p.warps);   // warps with a chunk
  // Row and piece of the matrix rows whose addresses this lane gives: matrices 0 and 1
  // are rows 0 to 7 and 8 to 15 of an even sub-block, 2 and 3 of the odd one behind it.
  const int mrow = lane & 15, mturn = kSubs == 8 ? lane & 7 : lane >> 1 & 3;
  const uint32_t matrices =
      smem_addr(ring) + mrow * kSubs * 16 + ((lane >> 4) ^ mturn) * 16;
  uint32_t at = 0;
  int slot = 0;   // of the batch
  for (int tile = 0; tile < tiles; ++tile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    float* mine = red + (slot * p.warps + warp) * kOuts;
    if (live) {
      const unsigned char* st = ring + at;   // the tile's stage
      // the scales of rows g and g + 8
      float sc[2][kPer];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned char* from = st + kCodes + (g + 8 * h) * p.scale_pitch;
        if (kPer >= 2 && p.vector) {
          uint32_t w[kPer >= 2 ? kPer / 2 : 1];
          if constexpr (kPer == 8) {
            const uint4 v = lds128(from);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else if constexpr (kPer == 4) {
            const uint2 v = lds64(from);
            w[0] = v.x, w[1] = v.y;
          } else {
            w[0] = *reinterpret_cast<const uint32_t*>(from);
          }
#pragma unroll
          for (int i = 0; i < kPer / 2; ++i) {
            sc[h][2 * i] = __uint_as_float(w[i] << 16);
            sc[h][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        } else {
          const int odd = (int)(((int64_t)(n0 + kGemvRows * tile + g + 8 * h) * p.groups +
                                 chunk * kPer) & 1);
          const uint16_t* v = reinterpret_cast<const uint16_t*>(from) + odd;
#pragma unroll
          for (int i = 0; i < kPer; ++i) sc[h][i] = __uint_as_float((uint32_t)v[i] << 16);
        }
      }
      uint32_t w[4];
      float acc[NT][4];
#pragma unroll
      for (int b = 0; b < kChunk / 128; ++b) {
        float d[NT][4], c[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int sub = 4 * b + i;
          if (i % 2 == 0) load_matrices((matrices + at) ^ (16u * sub), w);
          uint32_t lo[kFrag], hi[kFrag];
          decode8<E4M3, INT4>(w[i % 2 * 2], lo);
          decode8<E4M3, INT4>(w[i % 2 * 2 + 1], hi);
          const bool opens = 32 * i % G == 0, ends = 32 * (i + 1) % G == 0;
          const int grp = 32 * sub / G;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t(&f)[kFrag] = frag[sub][j];
            float(&cj)[4] = c[j];
            if constexpr (E4M3) {
              float2 x = make_float2(0.f, 0.f);
              if (INT4 && opens) x = *reinterpret_cast<const float2*>(sums + grp * 8 * NT + 8 * j + 2 * t);
              if (opens)
                mma_e4m3(cj, lo[0], hi[0], lo[1], hi[1], f[0], f[1], x.x, x.y, x.x, x.y);
              else
                mma_e4m3(cj, lo[0], hi[0], lo[1], hi[1], f[0], f[1], cj[0], cj[1], cj[2], cj[3]);
            } else {
              if (opens)
                mma_f16(cj, lo[0], hi[0], lo[1], hi[1], f[0], f[1], 0.f, 0.f, 0.f, 0.f);
              else
                mma_f16(cj, lo[0], hi[0], lo[1], hi[1], f[0], f[1], cj[0], cj[1], cj[2], cj[3]);
              mma_f16(cj, lo[2], hi[2], lo[3], hi[3], f[2], f[3], cj[0], cj[1], cj[2], cj[3]);
            }
            if (ends) {
              const bool begins = 32 * (i + 1) == G;   // the block's first group
#pragma unroll
              for (int e = 0; e < 4; ++e)
                d[j][e] = begins ? cj[e] * sc[e >> 1][grp] : fmaf(cj[e], sc[e >> 1][grp], d[j][e]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[j][e] = b == 0 ? d[j][e] * factor[b][j][e & 1]
                               : fmaf(d[j][e], factor[b][j][e & 1], acc[j][e]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(mine + (16 * j + g + 8 * h) * 8 + 2 * t) =
              make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
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
      const int m = q / 32 * 8 + q % 2 * 4, r = kGemvRows * (tile + 1 - slot + b) + q % 32 / 2;
      if (m0 + m >= p.M) continue;
      const float4* from = reinterpret_cast<const float4*>(red + b * p.warps * kOuts) + q;
      float v[4] = {};
#pragma unroll 4
      for (int w = 0; w < summed; ++w) {
        const float4 x = from[w * (kOuts / 4)];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (E4M3) v[e] *= INT4 ? 512.f : 64.f;   // of the codes' bits
        if (p.cluster > 1) {
          total[(m + e) * kGemvRows * tiles + r] = v[e];
        } else if (m0 + m + e < p.M && r < rows) {
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

template <bool E4M3, bool INT4, int G>
GemvKernel pick_tiles(int nt) {
  switch (nt) {
    case 1: return gemv_kernel<E4M3, INT4, G, 1>;
    case 2: return gemv_kernel<E4M3, INT4, G, 2>;
    default: return gemv_kernel<E4M3, INT4, G, 4>;
  }
}

}  // namespace

template <bool E4M3, bool INT4>
GemvKernel pick_gemv(int group, int nt) {
  return group == 32   ? pick_tiles<E4M3, INT4, 32>(nt)
         : group == 64 ? pick_tiles<E4M3, INT4, 64>(nt)
                       : pick_tiles<E4M3, INT4, 128>(nt);
}

}  // namespace nts
