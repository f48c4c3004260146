// gemv_internal.h -- what the launcher of the products with 4-bit weights and its kernels
// share.
#pragma once

#include <cuda.h>   // CUtensorMap
#include <cuda_bf16.h>

#include <cstdint>

#include "block_internal.h"

namespace nts {

constexpr int kMaxGemvWarps = 16;
constexpr int kGemvRows = 32;      // weight rows of a tile

constexpr int kGemvChunk = 256;    // k values of a warp's chunk
constexpr int kGemvStages = 2;     // tiles of a warp's ring

struct GemvParams {
  const void* a;
  const float* a_scales;     // E4M3 rows
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
  int vector;                // a chunk's (tiles: a K block's) scales of a row are one aligned piece
  int scale_pitch;           // bytes of a row's scales in a stage
  int stage_bytes;           // a multiple of 128
  int fp32;
  int batch;                 // tiles whose sums the warps keep between two barriers
  uint64_t wait_limit_ns;    // tile kernel
  uint32_t missing_tx;       // test hook: bytes expected on the first stage but never sent
};

using GemvKernel = void (*)(GemvParams);

// The kernel for a group size and a number of tiles of 8 rows (gemv_e2m1.cu, gemv_int4.cu).
template <bool INT4>
GemvKernel pick_gemv(int group, int nt);
extern template GemvKernel pick_gemv<false>(int, int);
extern template GemvKernel pick_gemv<true>(int, int);
// The tile kernel for a group size and a type of A, whose rows it copies by a tensor map,
// and its shared memory.
using GemvTileKernel = void (*)(CUtensorMap, GemvParams);
constexpr int kTileThreads = 608;
constexpr int kTileRows = 32;      // rows of A of a tile
template <bool INT4>
GemvTileKernel pick_gemv_tile(int group, bool e4m3, size_t* smem);
extern template GemvTileKernel pick_gemv_tile<false>(int, bool, size_t*);
extern template GemvTileKernel pick_gemv_tile<true>(int, bool, size_t*);
// Each unit's status word.
template <bool INT4>
int read_and_clear_gemv_unit(unsigned* out);
extern template int read_and_clear_gemv_unit<false>(unsigned*);
extern template int read_and_clear_gemv_unit<true>(unsigned*);

}  // namespace nts
