// gemv_launch.cu -- products of few rows with weights of 4 bits that carry a bf16 scale
// per group of 32, 64 or 128 values along K, on one GB300.
//
//     Y[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] c[n][k],
//
// c the E2M1 or int4 value of a code, A in bf16, or E4M3 codes with an fp32 scale per 128
// values (the operand of nts_gemm_blockscaled).
//
// GB300 mapping: with few rows the weights' bytes are the whole cost (0.5 a weight, and
// 2 per group), so they go through once and everything else has to fit beside them: about
// six issue slots for two weights of a lane at HBM's rate.  The products run on mma.sync
// (m16n8k16, fp16 in, fp32 sums), 16 weight rows against 8 rows of A at a time, whose
// operands are registers, where the codes are turned into fp16 (exactly); A's rows are
// the narrow operand, so 1 to 8 of them cost the same.  (tcgen05 reads the weights from
// shared memory: as bf16 they would pass through it five bytes a weight, above its rate
// at HBM's; it serves more rows, below.)  mma.sync on E4M3 operands is taken apart into
// fp16 products (25 issue cycles for a k of 32, 16 by fp16 ones; int8 65), so E4M3 rows
// become fp16 too.
// A warp owns a chunk of 256 values of K: its part of A stays in registers as B
// fragments for the whole call, and it streams its chunk of one tile of 32 weight rows
// after the other through its own ring of shared memory (cp.async: no barrier and no other
// warp's copies to wait for).  The codes of a group lie in the four lanes of a quad, four
// bytes each (a matrix load's layout), so a group's products end in one fragment, which
// the group's scale multiplies in fp32.  The warps' sums of a few tiles at a time meet in
// shared memory, in a fixed order; a K beyond 16 chunks is split over the CTAs of a
// cluster, whose sums meet once at the end.
// A's values become fp16 without loss where it matters: E4M3 codes exactly; bf16 rows by
// a power of two per 128 values that puts the largest near 2^14, so a value is exact
// unless it is below 2^-31 of the largest beside it, and then off by at most 2^-39 of it,
// under the fp32 sums' own roundings.
//
// Measured (us, back to back in a graph over more than L2; of the copy's rate): [1, 4096]
// x [12288, 4096] E2M1, groups of 32, 9.3 (0.45); groups of 128 8.1; int4, groups of 32,
// 11.5 (0.36); [1, 4096] x [4096, 4096] 5.0; [1, 16384] x [4096, 16384] 11.6 (0.48); [8,
// 16384] E4M3 x [5120, 16384] int4, groups of 128, 16.9; [8, 16384] x [16384, 16384] 32.3
// (0.69); [16, 5120] x [15360, 5120], groups of 64, 20.1 (0.31).  Of the 13000 cycles after
// the start of the first of these, 4000 pass before A and the first tile are there, 2100
// are a tile's 16 steps of 32 values (33 issue slots a step: eight conversions, two
// products, four scalings and the loads) and 1300 the last sums.  Boxes of 8 or 16 rows
// by TMA in place of cp.async took 10.8 and 9.4 us; tiles of 16 rows with a barrier each
// 11.2; the codes by 4-byte loads 11.6; 20 warps of 96 registers the same as 16 of 128.
//
// More than 16 rows and many weights take gemv_tile_kernel: 128 rows of W by 32 of A on
// tcgen05, so that a code is turned once for 32 rows.  A's rows come by TMA as they are,
// bf16 or E4M3; the codes become that type, exactly, in registers on their way to shared
// memory.  Two teams of four warps do that for alternate K blocks, a warp each issues the
// blocks' products (a group's into columns of tensor memory of its own), and two more
// teams read the groups' sums back and multiply them by the scales in fp32.  A last warp
// starts A's copies and asks L2 for the codes some blocks ahead.
// [32, 5120] x [15360, 5120], E2M1 with groups of 64: 24.5 us (33.5 in passes of 16 rows);
// groups of 32 27.4, by E4M3 rows 27.1 (33.4 and 33.7); int4, groups of 128: 23.1 (38.1).
// Weights of 8 bits (nts_gemm_blockscaled) take 15.5, and less than 4 bits from 9 rows on:
// [8, 16384] E4M3 x [16384, 16384] 43.0 and 32.6, 9 rows 43.0 and 48.3.
// A K block takes ~1000 cycles of an SM, ~600 of them the codes' (17 integer instructions
// for eight of them, two cycles each a warp) and, beside that, ~640 the shared memory's for
// the stores, copies and products.
// Other forms, when this one took 24.2: fp16 operands, which E2M1 codes become in a third
// of the instructions, but A's rows only by 8 more warps, 27.7; a third team for the codes
// 26.5; the sums of every block read by all eight warps 24.6.
#include <cuda_runtime.h>

#include <algorithm>

#include "gemv_internal.h"

namespace nts {

namespace {

// Tiles of a batch, by tiles of 8 rows of A: 4 KB of sums per warp.
constexpr int kBatch = 4;

template <typename Kernel, typename... Args>
int launch(Kernel kern, cudaLaunchConfig_t cfg, int cluster, cudaStream_t stream, bool pdl,
           const Args&... args) {
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return fail_cuda(e, "launching the product with 4-bit weights");
  return NTS_OK;
}

// Tiles of 128 rows of W by 32 of A, K split over a cluster of the size that has the
// tiles done first: rounds of the clusters that the GPU holds at once, each a share of the
// K blocks and about nine more to start and end.  [32, 4096] x [4096, 4096] 10.2 us with
// clusters of 4, of which 32 run at once, 23 with 8 and 15 with 2.
int launch_tiles(const GemvRequest& rq, GemvParams p, cudaStream_t stream, const DeviceInfo& dev,
                 const LaunchTuning& tune) {
  constexpr int kMost = 8;
  const int64_t tiles_n = (p.N + 127) / 128, tiles_m = (p.M + kTileRows - 1) / kTileRows;
  size_t smem = 0;
  const bool e4m3 = p.a_scales != nullptr;
  const GemvTileKernel kern =
      (rq.int4 ? pick_gemv_tile<true> : pick_gemv_tile<false>)(rq.group, e4m3, &smem);
  int rc = prepare_kernel((const void*)kern, smem + 16 * kMost);
  if (rc != NTS_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTileThreads);
  int64_t best = 0;
  for (int s = 1; s <= kMost && s <= p.kb; ++s) {
    int64_t fit = dev.sm_count;
    if (s > 1) {   // asked with a size of shared memory that names the cluster too, as below
      cudaLaunchAttribute size;
      size.id = cudaLaunchAttributeClusterDimension;
      size.val.clusterDim.x = s;
      size.val.clusterDim.y = size.val.clusterDim.z = 1;
      cfg.attrs = &size;
      cfg.numAttrs = 1;
      cfg.dynamicSmemBytes = smem + 16 * s;
      rc = max_active_clusters((const void*)kern, cfg, s, &fit);
      if (rc != NTS_OK) return rc;
    }
    const int64_t cost = (tiles_n * tiles_m + fit - 1) / fit * ((p.kb + s - 1) / s + 9);
    if (best == 0 || cost < best) {
      best = cost;
      p.cluster = s;
    }
  }
  if (tiles_n * p.cluster > 0x7fffffffll || tiles_m > 65535)
    return fail(NTS_ERR_UNSUPPORTED, "too many tiles in one call");
  p.vector = p.K % 128 == 0;
  CUtensorMap rows;
  rc = make_row_map(&rows, rq.A, !e4m3, p.M, p.K, p.lda, kTileRows);
  if (rc != NTS_OK) return rc;
  note_launch(kGemvUnit);
  cfg.gridDim = dim3((unsigned)(tiles_n * p.cluster), (unsigned)tiles_m);
  cfg.dynamicSmemBytes = smem;
  log_launch("gemv_groupscaled", "M=%d N=%d K=%d group=%d int4=%d tiles of 128 x 32 cluster=%d smem=%zu",
             p.M, p.N, p.K, rq.group, rq.int4, p.cluster, smem);
  return launch(kern, cfg, p.cluster, stream, tune.pdl != 0, rows, p);
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
  p.s = static_cast<const __nv_bfloat16*>(rq.w_scales);
  p.y = rq.Y;
  p.M = (int)rq.M;
  p.N = (int)rq.N;
  p.K = (int)rq.K;
  p.groups = (p.K + rq.group - 1) / rq.group;
  p.kb = (p.K + 127) / 128;
  p.fp32 = rq.fp32_out;
  p.w = static_cast<const uint8_t*>(rq.W);
  p.wait_limit_ns = tune.wait_limit_ns;
  p.missing_tx = tune.missing_tx;
  // Tiles instead of a second pass where the weights are many.  us, tiles / passes, E2M1
  // with groups of 32 and bf16 rows, A's rows x [N, K]:
  //   [4096, 4096]    16: 9.9 /  7.7   32: 10.3 / 10.3   64: 15.1 / 14.1
  //   [5120, 5120]    16: 13.7 / 10.9  32: 14.1 / 14.8   64: 27.0 / 23.8
  //   [15360, 5120]   16: 27.1 / 20.3  32: 27.5 / 33.4   64: 53.4 / 62.0
  //   [16384, 16384]                   32: 80.3 / 156
  //   [2048, 5120]                     32: 10.3 /  8.5  128: 17.2 / 21.0
  // The rule does not know how many rounds of tiles fill the SMs, and is behind where the
  // last round is nearly empty or the tiles are few: 48 x [12288, 4096] 43.6 / 25.6 and
  // 32: 23.4 / 20.1 (int4 with groups of 128 19.4 / 21.5), 32 x [1024, 32768] 24.4 / 19.5,
  // 48 x [15360, 5120] 53.0 / 48.3; nor how many passes a long A takes: 512 x [2048, 8192]
  // 84 / 141, where it takes passes.
  enum { kAuto, kPasses, kTiles };
  const int kind = tune.force_vpt <= kTiles ? tune.force_vpt : kAuto;   // debug: one of these
  if (kind == kTiles || (kind == kAuto && p.M > 16 && (int64_t)p.N * p.K > 4096 * 4096))
    return launch_tiles(rq, p, stream, dev, tune);
  // slices of A's rows, in even parts
  const int slices_m = (p.M + 15) / 16;
  const int nt = p.M <= 8 ? 1 : 2;
  p.per = 8 * nt;
  const int chunk = kGemvChunk, stages = kGemvStages;
  p.chunks = (p.K + chunk - 1) / chunk;
  p.cluster = (p.chunks + kMaxGemvWarps - 1) / kMaxGemvWarps;
  p.warps = (p.chunks + p.cluster - 1) / p.cluster;
  const int per_row = chunk / rq.group;
  p.vector = p.groups % per_row == 0;
  p.scale_pitch = p.vector ? 2 * per_row : (2 * per_row + 2 + 3) / 4 * 4;
  p.stage_bytes = (kGemvRows * (chunk / 2 + p.scale_pitch) + 127) / 128 * 128;
  const GemvKernel kern = (rq.int4 ? pick_gemv<true> : pick_gemv<false>)(rq.group, nt);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)(32 * p.warps));
  p.batch = kBatch / nt;
  const auto bytes = [&] {
    return (size_t)p.warps *
           (stages * p.stage_bytes + kGemvRows * p.batch * 8 * nt * sizeof(float));
  };
  size_t base = bytes();
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
  // More CTAs than SMs only where each still has a whole tile.
  fit = std::min<int64_t>(fit / slices_m, std::max(dev.sm_count, p.N / kGemvRows));
  p.slices = (int)std::min<int64_t>(std::max<int64_t>(1, fit), p.N);
  if (p.cluster > 1) {
    // the sums of a slice across the cluster: with shorter batches, or more slices
    const size_t row = 8 * nt * sizeof(float);
    const auto whole = [](int64_t n) { return (n + kGemvRows - 1) / kGemvRows * kGemvRows; };
    const size_t want = whole((p.N + p.slices - 1) / p.slices) * row;
    while (p.batch > 1 && bytes() + want > limit) p.batch /= 2;
    base = bytes();
    const int64_t most = (int64_t)((limit - base) / row) / kGemvRows * kGemvRows;
    p.slices = (int)std::max<int64_t>(p.slices, (p.N + most - 1) / most);
    cfg.dynamicSmemBytes = base + whole((p.N + p.slices - 1) / p.slices) * row;
  }
  cfg.gridDim = dim3((unsigned)(p.slices * p.cluster), (unsigned)slices_m);
  log_launch("gemv_groupscaled",
             "M=%d N=%d K=%d group=%d int4=%d tiles of 8=%d warps=%d cluster=%d slices=%d smem=%zu",
             p.M, p.N, p.K, rq.group, rq.int4, nt, p.warps, p.cluster, p.slices,
             cfg.dynamicSmemBytes);
  return launch(kern, cfg, p.cluster, stream, tune.pdl != 0, p);
}

int read_and_clear_gemv_status(unsigned* out) {
  unsigned a = 0, b = 0;
  int rc = read_and_clear_gemv_unit<false>(&a);
  if (rc == NTS_OK) rc = read_and_clear_gemv_unit<true>(&b);
  *out = a | b;
  return rc;
}

}  // namespace nts
