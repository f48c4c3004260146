// gemv_kernel.cu -- products of few rows with weights of 4 bits that carry a bf16 scale
// per group of 32, 64 or 128 values along K, on one GB300.
//
//     Y[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] c[n][k],
//
// c the E2M1 or int4 value of a code, A in bf16, or E4M3 codes with an fp32 scale per 128
// values (the operand of nts_gemm_blockscaled).
//
// GB300 mapping: with few rows the weights' bytes are the whole cost (0.5 a weight, and
// 2 per group), so they go through once, at HBM's rate, and everything else has to fit
// beside them: about six issue slots for the two weights of a lane.  The products run on
// mma.sync (m16n8k16, fp16 in, fp32 sums), 16 weight rows against 8 rows of A at a time:
// a fifth of the tensor instructions' rate is enough, and their operands come from
// registers, where the codes are turned into fp16 (exactly).  A's rows are the narrow
// operand, so 1 to 8 of them cost the same.
// A warp owns a chunk of K: its part of A stays in registers as B fragments for the
// whole call, and it streams its chunk of one tile of 16 weight rows after the other
// through its own ring of shared memory (cp.async, no barrier and no other warp's copies
// to wait for).  The codes of a group lie in the four lanes of a quad, four bytes each,
// so a group's products end in one fragment, which the group's scale multiplies in fp32.
// A tile's sums over the warps' chunks meet in shared memory, in a fixed order; a longer
// K is split over the CTAs of a cluster, whose sums meet once at the end.
// A's values become fp16 without loss where it matters: E4M3 codes exactly; bf16 rows by
// a power of two per 128 values that puts the largest near 2^14, so a value is exact
// unless it is below 2^-31 of the largest beside it, and then off by at most 2^-39 of it,
// under the fp32 sums' own roundings.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_device.cuh"
#include "block_internal.h"

namespace nts {

namespace {

constexpr int kMaxGemvWarps = 16;
constexpr int kRows = 16;          // weight rows of a tile
constexpr int kRedPitch = 20;      // floats per row of A in a tile's sums: distinct banks

// k values of a warp's chunk, and the ring's stages.
__host__ __device__ constexpr int chunk_of(int nt) { return nt <= 2 ? 256 : 128; }
__host__ __device__ constexpr int stages_of(int nt) { return nt <= 2 ? 4 : 6; }

struct GemvParams {
  const void* a;
  const float* a_scales;     // E4M3 rows, or nullptr: bf16
  int64_t lda;
  const uint8_t* w;
  const __nv_bfloat16* s;
  void* y;
  int M, N, K;
  int groups;                // scales of a weight row
  int kb;                    // a_scales per row
  int chunks;                // chunks of K
  int warps;                 // per CTA
  int cluster;               // CTAs along K
  int slices;                // row slices (clusters along N)
  int per;                   // rows of A per slice of M (blockIdx.y)
  int vector;                // a chunk's scales of a row are one aligned copy
  int pitch;                 // bytes of a row's scales in a stage
  int fp32;
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int size, int bytes) {
  if (size == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
  else if (size == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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

// c += A B of one m16n8k16: rows g and g + 8 of A by lanes (g, t), column g of B.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The halves of two pairs, lo halves first.
__device__ __forceinline__ void by_fours(uint32_t (&p)[4]) {
  const uint32_t a = __byte_perm(p[0], p[2], 0x5410), b = __byte_perm(p[0], p[2], 0x7632);
  const uint32_t c = __byte_perm(p[1], p[3], 0x5410), d = __byte_perm(p[1], p[3], 0x7632);
  p[0] = a, p[1] = b, p[2] = c, p[3] = d;   // (0,4) (1,5) (2,6) (3,7)
}

// A warp's chunk of A as B fragments: frag[sub-block of 32][tile of 8 rows][pair], and
// per block of 128 and tile the factors of the lane's two columns of a product.
template <bool INT4, int NT>
__device__ __forceinline__ void load_rows(const GemvParams& p, int m0, int k0,
                                          uint32_t (&frag)[chunk_of(NT) / 32][NT][4],
                                          float (&factor)[chunk_of(NT) / 128][NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int end = min(p.M, m0 + p.per);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = m0 + 8 * j + g;
#pragma unroll
    for (int b = 0; b < chunk_of(NT) / 128; ++b) {
      if (p.a_scales != nullptr) {
        uint2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + 128 * b + 32 * i;
          x[i] = make_uint2(0, 0);
          if (m < end && k < p.K)
            x[i] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.a) +
                                                        m * p.lda + k + 8 * t));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t(&f)[4] = frag[4 * b + i][j];
          f[0] = e4m3x2_to_f16x2(x[i].x), f[1] = e4m3x2_to_f16x2(x[i].x >> 16);
          f[2] = e4m3x2_to_f16x2(x[i].y), f[3] = e4m3x2_to_f16x2(x[i].y >> 16);
          if (INT4) by_fours(f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = m0 + 8 * j + 2 * t + i, block = k0 / 128 + b;
          factor[b][j][i] = col < end && block < p.kb
                                ? __ldg(p.a_scales + (int64_t)col * p.kb + block)
                                : 0.f;
        }
      } else {
        uint4 x[4];
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + 128 * b + 32 * i;
          x[i] = make_uint4(0, 0, 0, 0);
          if (m < end && k < p.K)
            x[i] = __ldg(reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(p.a) + m * p.lda + k + 8 * t));
          float v[8];
          bf16x8_to_f32(x[i], v);
#pragma unroll
          for (int e = 0; e < 8; e += 2) most = fmax3(most, fabsf(v[e]), fabsf(v[e + 1]));
        }
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        // 2^f: the largest comes to [2^14, 2^15), as far as 2^f and 2^-f are normal
        const int f = max(-113, min(126, 141 - (int)(__float_as_uint(most) >> 23)));
        const float up = __uint_as_float((uint32_t)(127 + f) << 23);
        const float down = __uint_as_float((uint32_t)(127 - f) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[8];
          bf16x8_to_f32(x[i], v);
          uint32_t(&q)[4] = frag[4 * b + i][j];
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
  }
}

template <bool INT4, int G, int NT>
__global__ void __launch_bounds__(32 * kMaxGemvWarps, 1) gemv_kernel(const GemvParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kChunk = chunk_of(NT), kStages = stages_of(NT);
  constexpr int kSubs = kChunk / 32;             // 16-byte pieces of a row's chunk of codes
  constexpr int kPer = kChunk / G;               // scales of a row's chunk
  constexpr int kCodes = kRows * kChunk / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int stage_bytes = kCodes + kRows * p.pitch;
  unsigned char* ring = smem + warp * kStages * stage_bytes;
  // sums: [2][warps][8 NT][kRedPitch]; across the cluster [8 NT][16 tiles]
  float* red = reinterpret_cast<float*>(smem + p.warps * kStages * stage_bytes);
  constexpr int kRed = 8 * NT * kRedPitch;
  float* total = red + 2 * p.warps * kRed;

  const int slice = blockIdx.x / p.cluster;
  const int rank = blockIdx.x - slice * p.cluster;
  const int n0 = (int)((int64_t)p.N * slice / p.slices);
  const int n1 = (int)((int64_t)p.N * (slice + 1) / p.slices);
  const int tiles = (n1 - n0 + kRows - 1) / kRows;
  const int m0 = blockIdx.y * p.per;
  const int chunk = rank * p.warps + warp;       // of K
  const int k0 = chunk * kChunk;
  const bool live = chunk < p.chunks;
  grid_dependency_wait();
  allow_dependent_launch();

  // One tile's codes and scales into a stage.  A row's pieces change places with the
  // row's number, so that the eight rows that a warp reads at once meet distinct banks.
  auto stage = [&](int tile, int s) {
    if (live && tile < tiles) {
      const uint32_t dst = smem_addr(ring) + s * stage_bytes;
      const int first = n0 + kRows * tile;
#pragma unroll
      for (int i = 0; i < kRows * kSubs / 32; ++i) {
        const int q = 32 * i + lane, row = q / kSubs, piece = q % kSubs;
        const int turn = kSubs == 8 ? row & 7 : row >> 1 & 3;
        const bool in = first + row < n1 && k0 + 32 * piece < p.K;
        copy_async(dst + (row * kSubs + (piece ^ turn)) * 16,
                   in ? p.w + (int64_t)(first + row) * (p.K / 2) + k0 / 2 + 16 * piece : p.w, 16,
                   in ? 16 : 0);
      }
      const int have = min(kPer, p.groups - chunk * kPer);   // scales of a row here
      if (p.vector) {
        if (lane < kRows) {
          const bool in = first + lane < n1;
          copy_async(dst + kCodes + lane * p.pitch,
                     in ? p.s + (int64_t)(first + lane) * p.groups + chunk * kPer : p.s,
                     max(4, 2 * kPer), in ? 2 * have : 0);
        }
      } else {
        // words that hold them, from the word of the first; nothing beyond the last
        for (int q = lane; q < kRows * 8; q += 32) {
          const int row = q >> 3, word = q & 7;
          if (4 * word >= p.pitch) continue;
          const int64_t at = (int64_t)(first + row) * p.groups + chunk * kPer;
          const int bytes =
              first + row < n1 ? (int)max64(0, min64(4, 2 * (at + have) - (4 * (at / 2) + 4 * word))) : 0;
          copy_async(dst + kCodes + row * p.pitch + 4 * word,
                     bytes > 0 ? p.s + 2 * (at / 2) + 2 * word : p.s, 4, bytes);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s < kStages; ++s) stage(s, s);

  uint32_t frag[kSubs][NT][4];
  float factor[kChunk / 128][NT][2];
  load_rows<INT4, NT>(p, m0, k0, frag, factor);

  for (int tile = 0, s = 0; tile < tiles; ++tile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const int first = n0 + kRows * tile;
    float* mine = red + ((tile & 1) * p.warps + warp) * kRed;
    if (live) {
      const unsigned char* st = ring + s * stage_bytes;
      // the scales of rows g and g + 8
      float sc[2][kPer];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned char* at = st + kCodes + (g + 8 * h) * p.pitch;
        if (p.vector) {
          if constexpr (kPer == 8) {
            const uint4 v = lds128(at);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sc[h][2 * i] = __uint_as_float(w[i] << 16);
              sc[h][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
          } else if constexpr (kPer == 4) {
            const uint2 v = lds64(at);
            sc[h][0] = __uint_as_float(v.x << 16), sc[h][1] = __uint_as_float(v.x & 0xFFFF0000u);
            sc[h][2] = __uint_as_float(v.y << 16), sc[h][3] = __uint_as_float(v.y & 0xFFFF0000u);
          } else if constexpr (kPer == 2) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
            sc[h][0] = __uint_as_float(v << 16), sc[h][1] = __uint_as_float(v & 0xFFFF0000u);
          }
        } else {
          const int odd = (int)(((int64_t)(first + g + 8 * h) * p.groups + chunk * kPer) & 1);
          const uint16_t* v = reinterpret_cast<const uint16_t*>(at) + odd;
#pragma unroll
          for (int i = 0; i < kPer; ++i) sc[h][i] = __uint_as_float((uint32_t)v[i] << 16);
        }
      }
      float acc[NT][4] = {};
#pragma unroll
      for (int b = 0; b < kChunk / 128; ++b) {
        float d[NT][4] = {}, c[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int sub = 4 * b + i;
          const int turn = kSubs == 8 ? g : g >> 1 & 3;   // of row g + 8 too
          const unsigned char* at = st + (g * kSubs + (sub ^ turn)) * 16 + 4 * t;
          uint32_t lo[4], hi[4];
          decode8<INT4>(*reinterpret_cast<const uint32_t*>(at), lo);
          decode8<INT4>(*reinterpret_cast<const uint32_t*>(at + 8 * kSubs * 16), hi);
          const bool opens = 32 * i % G == 0, ends = 32 * (i + 1) % G == 0;
          const int grp = 32 * sub / G;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (opens) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
            const uint32_t(&f)[4] = frag[sub][j];
            mma16816(c[j], lo[0], hi[0], lo[1], hi[1], f[0], f[1]);
            mma16816(c[j], lo[2], hi[2], lo[3], hi[3], f[2], f[3]);
            if (ends) {
              d[j][0] = fmaf(c[j][0], sc[0][grp], d[j][0]);
              d[j][1] = fmaf(c[j][1], sc[0][grp], d[j][1]);
              d[j][2] = fmaf(c[j][2], sc[1][grp], d[j][2]);
              d[j][3] = fmaf(c[j][3], sc[1][grp], d[j][3]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(d[j][e], factor[b][j][e & 1], acc[j][e]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * t + (e & 1)) * kRedPitch + g + 8 * (e >> 1)] = acc[j][e];
    }
    __syncwarp();   // the stage is read by all before the next copy into it
    stage(tile + kStages, s);
    if (++s == kStages) s = 0;
    __syncthreads();   // the other buffer's readers are past this barrier
    const int warps = min(p.warps, p.chunks - rank * p.warps);
    for (int o = threadIdx.x; o < 8 * NT * kRows; o += blockDim.x) {
      const int m = o / kRows, r = o % kRows;
      const float* at = red + (tile & 1) * p.warps * kRed + m * kRedPitch + r;
      float v = 0.f;
#pragma unroll 4
      for (int w = 0; w < warps; ++w) v += at[w * kRed];
      if (p.cluster > 1) {
        total[m * kRows * tiles + kRows * tile + r] = v;
      } else if (m < p.per && m0 + m < p.M && first + r < n1) {
        const int64_t to = (int64_t)(m0 + m) * p.N + first + r;
        if (p.fp32)
          static_cast<float*>(p.y)[to] = v;
        else
          static_cast<__nv_bfloat16*>(p.y)[to] = __float2bfloat16_rn(v);
      }
    }
  }
  if (p.cluster == 1) return;

  // The sums of the cluster's CTAs, in their order: each takes a share of the slice.
  cluster_arrive_release();
  cluster_wait_acquire();
  const int count = (n1 - n0) * 8 * NT;
  for (int i = rank * blockDim.x + threadIdx.x; i < count; i += p.cluster * blockDim.x) {
    // neighbouring threads take neighbouring columns of a row of Y
    const int m = i / (n1 - n0), r = i - m * (n1 - n0);
    if (m >= p.per || m0 + m >= p.M) continue;
    const uint32_t at = smem_addr(total + m * kRows * tiles + r);
    float v = 0.f;
    for (int c = 0; c < p.cluster; ++c) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_to_rank(at, c)) : "memory");
      v += x;
    }
    const int64_t to = (int64_t)(m0 + m) * p.N + n0 + r;
    if (p.fp32)
      static_cast<float*>(p.y)[to] = v;
    else
      static_cast<__nv_bfloat16*>(p.y)[to] = __float2bfloat16_rn(v);
  }
  cluster_arrive_release();   // no CTA ends while another reads its sums
  cluster_wait_acquire();
}

using GemvKernel = void (*)(GemvParams);

template <bool INT4, int G>
GemvKernel pick_tiles(int nt) {
  switch (nt) {
    case 1: return gemv_kernel<INT4, G, 1>;
    case 2: return gemv_kernel<INT4, G, 2>;
    case 3: return gemv_kernel<INT4, G, 3>;
    default: return gemv_kernel<INT4, G, 4>;
  }
}

template <bool INT4>
GemvKernel pick_group(int group, int nt) {
  return group == 32   ? pick_tiles<INT4, 32>(nt)
         : group == 64 ? pick_tiles<INT4, 64>(nt)
                       : pick_tiles<INT4, 128>(nt);
}

}  // namespace

int launch_gemv(const GemvRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  GemvParams p = {};
  p.a = rq.A;
  p.a_scales = rq.a_scales;
  p.lda = rq.lda;
  p.w = static_cast<const uint8_t*>(rq.W);
  p.s = static_cast<const __nv_bfloat16*>(rq.w_scales);
  p.y = rq.Y;
  p.M = (int)rq.M;
  p.N = (int)rq.N;
  p.K = (int)rq.K;
  p.groups = (p.K + rq.group - 1) / rq.group;
  p.kb = (p.K + 127) / 128;
  p.fp32 = rq.fp32_out;
  // slices of A's rows, in even parts; a chunk is half as long from 17 rows on, and a
  // cluster holds 128 chunks
  const int slices_m = (p.M + 31) / 32 * (p.M > 16 && p.K > 16384 ? 2 : 1);
  p.per = ((p.M + slices_m - 1) / slices_m + 7) / 8 * 8;
  const int nt = p.per / 8;
  const int chunk = chunk_of(nt), stages = stages_of(nt);
  p.chunks = (p.K + chunk - 1) / chunk;
  p.cluster = (p.chunks + kMaxGemvWarps - 1) / kMaxGemvWarps;
  p.warps = (p.chunks + p.cluster - 1) / p.cluster;
  const int per_row = chunk / rq.group;
  p.vector = per_row >= 2 && p.groups % per_row == 0;
  p.pitch = p.vector ? 2 * per_row : (2 * per_row + 2 + 3) / 4 * 4;
  const GemvKernel kern = rq.int4 ? pick_group<true>(rq.group, nt) : pick_group<false>(rq.group, nt);

  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)(32 * p.warps));
  const size_t base = (size_t)p.warps * stages * (kRows * chunk / 2 + kRows * p.pitch) +
                      (size_t)2 * p.warps * 8 * nt * kRedPitch * sizeof(float);
  // slices: what the GPU holds at once; the sums of a slice across a cluster take
  // shared memory, so a long N takes more slices than that
  const size_t limit = (size_t)dev.max_smem_optin;
  int64_t fit = 0;
  cfg.dynamicSmemBytes = base;
  int rc = prepare_kernel((const void*)kern, p.cluster > 1 ? limit : base);
  if (rc != NTS_OK) return rc;
  if (p.cluster == 1) {
    int per_sm = 0;
    rc = blocks_per_sm((const void*)kern, cfg.blockDim.x, base, &per_sm);
    fit = (int64_t)dev.sm_count * per_sm;
  } else {
    // asked with a size of shared memory that names the cluster too: the answers are
    // kept by kernel, threads and size
    cudaLaunchAttribute size;
    size.id = cudaLaunchAttributeClusterDimension;
    size.val.clusterDim.x = p.cluster;
    size.val.clusterDim.y = size.val.clusterDim.z = 1;
    cfg.attrs = &size;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = limit - 16 * p.cluster;
    rc = max_active_clusters((const void*)kern, cfg, p.cluster, &fit);
    cfg.dynamicSmemBytes = base;
  }
  if (rc != NTS_OK) return rc;
  p.slices = (int)std::min<int64_t>(std::max<int64_t>(1, fit / slices_m), p.N);
  if (p.cluster > 1) {
    const int row = 8 * nt * (int)sizeof(float);
    const int most = (int)((limit - base) / row) / kRows * kRows;   // rows of a slice
    p.slices = std::max(p.slices, (p.N + most - 1) / most);
    while ((p.N + p.slices - 1) / p.slices > most) ++p.slices;
    const int rows = (p.N + p.slices - 1) / p.slices;
    cfg.dynamicSmemBytes = base + (size_t)((rows + kRows - 1) / kRows * kRows) * row;
  }
  cfg.gridDim = dim3((unsigned)(p.slices * p.cluster), (unsigned)slices_m);
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (p.cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = p.cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (tune.pdl) attr[n++] = pdl_attribute();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  log_launch("gemv_groupscaled",
             "M=%d N=%d K=%d group=%d int4=%d tiles of 8=%d warps=%d cluster=%d slices=%d smem=%zu",
             p.M, p.N, p.K, rq.group, rq.int4, nt, p.warps, p.cluster, p.slices,
             cfg.dynamicSmemBytes);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return fail_cuda(e, "launching the product with 4-bit weights");
  return NTS_OK;
}

}  // namespace nts
