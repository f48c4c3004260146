// gemm_kernel.cu -- matrix product of E4M3 operands with one fp32 scale for
// each block of 128 values along K, on the tcgen05 tensor cores of one GB300:
//
//     Y[m, n] = sum over kb of sa[m, kb] sw[n', kb]
//                   sum over k in block kb of A[m, k] W[n, k],
//
// n' = n / 128 (weights in 128 x 128 blocks) or n (1 x 128 blocks).  The
// inner sums of 128 products are left to the matrix instructions (fp32
// accumulators in tensor memory); the scales differ from block to block, so
// each block's sums are read back, scaled and added in fp32 registers.  One
// rounding to the output type at the end.
//
// Both kernels are pipelines of specialised warps: one warp fills a ring of
// shared-memory stages by TMA (128 bytes of K per row, 128-byte swizzle),
// one issues the matrix instructions of a stage into one of several
// tensor-memory buffers, two stage the scales of eight K blocks at a time,
// and the epilogue warps drain the buffers into registers.  The whole warp
// walks a role's loop and one elected lane acts: loops of a single thread
// cost ~25 cycles a branch.  Every wait is bounded.
//
//  * wide_kernel: rows of A are the instruction's M and BN rows of W its N,
//    tiles walked by a persistent grid: 256 x 256 by a pair of CTAs, or 128 x
//    128 by one.  Each epilogue thread holds one row of A, so a K block's scale
//    is one number per thread; with a scale per row of W too it holds fragments.
//  * narrow_kernel, for few rows of A: 128 rows of W are the instruction's M
//    and up to TN rows of A its N, so that the tensor cores waste nothing on
//    absent rows and the call reads W once at HBM speed.  K is split over the
//    CTAs of a cluster, which add their sums in rank order through
//    distributed shared memory.
//
// Measured (us in a graph): [8192, 5120] x [15360, 5120] 494 at 2070 MHz, 2.6
// PFLOP/s; kept up for seconds, in a graph or by calls, 530 to 540, 2.4 PFLOP/s,
// as the power limit takes the clock to 1910 to 1940 MHz.  The tensor pipe is 57 %
// busy, as the sums of a K block of 256 x 256 x 128 are read back and scaled in
// ~900 cycles, and its matrix instructions take 512 (without the scaling fmas 415,
// without the matrix instructions 423, with half of the operand bytes 489).
// [4096, 4112] x [4096, 4112] with scales per row, fp32: 107, one more multiply per
// sum.  [333, 5120] x [5120, 5120] 15.8, 510 cycles per K block of 128 x 128 and 4
// us to start and end.  One row by [12288, 4096] 11.7: W at 0.97 of the copy's
// rate, and the same 4 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_internal.h"
#include "gemm_device.cuh"

namespace nts {

namespace {

// kStatusTimeout bits of these kernels.
__device__ unsigned int g_gemm_status;

constexpr int kChunk = 8;        // K blocks per piece of staged scales
constexpr int kPieces = 2;       // pieces in flight

struct GemmParams {
  const float* sa;       // [M, kblocks]
  const float* sw;       // [N / 128 or N, kblocks]
  void* y;               // bf16 or fp32 [M, N]
  int64_t M, N;
  int kblocks;
  int tiles_m, tiles_n;  // wide
  int fp32_out;
  uint64_t wait_limit_ns;
  uint32_t missing_tx;   // test hook: bytes expected on the first stage but never sent
};

// After a wait gave up: the copies in flight land (the last S of `issued`
// stages) and the matrix instructions in flight end, each within the limit,
// before shared and tensor memory are given back.  The second CTA of a pair
// has its copies counted on the first one's barriers; it gives them a
// millisecond, a thousand times what a copy takes.
template <int S, bool PAIR>
__device__ __forceinline__ void drain(uint32_t full, uint32_t done, int64_t issued,
                                      uint64_t limit_ns) {
  const bool first = !PAIR || cluster_ctarank() == 0;
  if (threadIdx.x == 0) {
    if (first)
      for (int64_t j = max64(0, issued - S); j < issued; ++j)
        (void)mbar_wait_bounded(full + 8 * (int)(j % S), (uint32_t)((j / S) & 1), limit_ns);
    else
      for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {
      }
  }
  if (first && threadIdx.x >> 5 == 1 && elect_one()) {   // the thread that issues them
    mma_commit<PAIR>(done);
    (void)mbar_wait_bounded(done, 0, limit_ns);
  }
}

// A lane's share of staging the scales of N rows, from row0 on (of `rows` there
// are), for one K block: rows sub + 8 i, each to its place (linear over sub and
// 8 i) after dst.  Zeros where there is no row, or !in.  The addresses go from
// row to row by one step: formed anew for each copy they took the two warps 220
// cycles a copy beside the epilogue's arithmetic, more than the K blocks take
// when W has a scale per row ([4096, 4112] x [4096, 4112] to fp32: 128 us then,
// 106 so).
template <int N, typename Place>
__device__ __forceinline__ void stage_scales(uint32_t dst, const float* scales, int64_t row0,
                                             int64_t rows, int64_t kb, int64_t kblocks, bool in,
                                             int sub, Place place) {
  const int left = in ? (int)min64(N, rows - row0) : 0;
  const float* src = sub < left ? scales + (row0 + sub) * kblocks + kb : scales;
  dst += 4 * place(sub);
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    if (N % 8 != 0 && sub >= N) break;
    const bool here = sub + i < left;
    copy_async_f32(dst + 4 * place(i), src, here);
    if (here) src += 8 * kblocks;
  }
}

// ---------------------------------------------------------------- wide

constexpr int kGroupM = 16;   // tiles of A walked before the next tile of W

// Rows of Y that do not start on 32-byte boundaries leave through a little
// shared memory, 32 rows x 8 columns a warp at a time, so that a warp stores 8
// neighbouring values of four rows: each thread storing its own row's values
// one by one touched 32 sectors a store ([2048, 1696] x [5881, 1696]: 139 us
// then, 42 now).
constexpr int kOutPitch = 9, kOutWarp = 32 * kOutPitch;   // floats

// BN = 256: a pair of CTAs works on 256 rows of A by 256 rows of W.  Each CTA
// holds its 128 rows of A and half of W's rows, so an SM stores and reads 32 KB
// per K block for 512 cycles of matrix instructions.  BN = 128: one CTA, 128
// rows of A, for products with too few tiles for the pairs.
//
// Eight epilogue warps: four (one per 32 rows) for each half of the columns,
// 32 columns at a time, the next 32 on their way while these are scaled and
// added -- across K blocks too.  At BN = 256 a thread holds 128 sums and 64
// loaded values, more than 384 threads have registers for: 168 at launch, then
// 72 in the four other warps and 216 in the epilogue's eight (128 * 72 + 256 *
// 216 = 384 * 168).
template <int BN, bool ROWS>
struct Wide {
  static constexpr bool kPair = BN == 256;
  static constexpr int kTileM = kPair ? 256 : 128;        // rows of A per tile
  static constexpr int kRowsW = kPair ? BN / 2 : BN;      // rows of W per CTA
  static constexpr int kCols = BN / 2;                    // columns per epilogue warp
  static constexpr int kThreads = 384;                    // TMA, MMA, 2 scale warps; epilogue
  static constexpr int kRegs = kPair ? 168 : 0, kRegsDown = 72, kRegsUp = 216;
  static constexpr uint32_t kA = 128 * 128;
  static constexpr uint32_t kStage = kA + kRowsW * 128;
  static constexpr int kStages = 196608 / (int)kStage;    // 6
  static constexpr int kHalves = kPair && !ROWS ? 2 : 1;  // accumulators per K block
  static constexpr int kBufCols = BN / kHalves;           // columns of an accumulator
  static constexpr int kRing = kPair ? 2 : 3;             // K blocks in tensor memory
  static constexpr int kBufs = kRing * kHalves;           // at most 512 columns in all
  static constexpr int kScales = 128 + (ROWS ? BN : 4);   // floats per K block
  static constexpr uint32_t kScaleOff = kStages * kStage;
  static constexpr uint32_t kOutOff = kScaleOff + kPieces * kChunk * kScales * 4;
  static constexpr uint32_t kBarOff = kOutOff + 8 * kOutWarp * 4;
  static constexpr uint32_t kBytes = kBarOff + 256;
  static constexpr uint32_t kLaunch = kBytes + 1024;      // the base is rounded up to 1024
};

__device__ __forceinline__ void tile_at(const GemmParams& p, int64_t tile, int* tm, int* tn) {
  const int64_t per_group = (int64_t)kGroupM * p.tiles_n;
  const int64_t g = tile / per_group;
  const int64_t in = tile - g * per_group;
  const int rows = (int)min64(kGroupM, p.tiles_m - g * kGroupM);
  *tn = (int)(in / rows);
  *tm = (int)(g * kGroupM + (in - (int64_t)*tn * rows));
}

// With a scale for each row of W too, a thread reads fragments of 16 rows by 32
// columns (tmem_load_fragments): 32 rows and COLS columns take 4 row scales and
// COLS / 4 column scales a thread, where a thread with a row of its own needs
// all COLS of them from shared memory ([4096, 4112] x [4096, 4112] to fp32:
// 123 us then, 106 now).  The scales lie in shared memory in the order in
// which a thread needs them, four at a time.
__device__ __forceinline__ int row_place(int r) {
  return (r & ~31) + (r & 7) * 4 + (r >> 3 & 3);
}
__device__ __forceinline__ int column_place(int r) {
  return (r & ~31) + (r >> 1 & 3) * 8 + (r >> 3 & 3) * 2 + (r & 1);
}

// VEC: rows of Y start on 32-byte boundaries (a template parameter: with both
// ways out in one kernel the aligned one was 4 % slower).
template <int BN, bool ROWS, bool VEC>
__global__ void __launch_bounds__(Wide<BN, ROWS>::kThreads, 1)
wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
            const GemmParams p) {
  using C = Wide<BN, ROWS>;
  constexpr int S = C::kStages, NB = C::kBufs, H = C::kHalves;
  constexpr bool PAIR = C::kPair;
  extern __shared__ unsigned char raw[];
  const uint32_t sbase = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* smem = raw + (sbase - smem_addr(raw));
  float* scales = reinterpret_cast<float*>(smem + C::kScaleOff);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t full = bars, empty = full + 8 * S, tfull = empty + 8 * S, tempty = tfull + 8 * NB,
                 sfull = tempty + 8 * NB, sempty = sfull + 8 * kPieces, done = sempty + 8 * kPieces,
                 slot = done + 8;
  volatile int* stop = reinterpret_cast<volatile int*>(smem + (slot + 4 - sbase));
  int64_t* issued = reinterpret_cast<int64_t*>(smem + (slot + 8 - sbase));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, (PAIR ? 16 : 8) / H);   // warps that drain it
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(sfull + 8 * i, 64);
      mbar_init(sempty + 8 * i, 8);
    }
    mbar_init(done, 1);
    *stop = 0;
    *issued = 0;
    fence_mbar_init();
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_w);
  }
  if (warp == 1) tmem_alloc<PAIR>(slot, 512);
  tcgen05_fence_before();
  __syncthreads();
  if (PAIR) {   // the other CTA's barriers are there before anything signals them
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - sbase));
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const int64_t first = PAIR ? cluster_id_x() : blockIdx.x;
  const int64_t step = PAIR ? num_clusters_x() : gridDim.x;
  const uint32_t stop_at = slot + 4;
  uint32_t late = 0;

  if (warp < 4) {
    if (PAIR) registers_down<C::kRegsDown>();
    const bool leader = elect_one();
    if (warp == 0) {
      RingSlot<S> st;
      int64_t n = 0;   // stages issued
      for (int64_t tile = first; tile < tiles && !late; tile += step) {
        int tm, tn;
        tile_at(p, tile, &tm, &tn);
        const int ya = tm * C::kTileM + rank * 128, yw = tn * BN + rank * (C::kRowsW / H);
        for (int k0 = 0; k0 < p.kblocks && !late; k0 += kChunk) {
          const int k1 = min(k0 + kChunk, p.kblocks);
          for (int kb = k0; kb < k1; ++kb, st.advance()) {
            const uint32_t at = sbase + st.i * C::kStage, bar = full + 8 * st.i;
            // a pair's copies all count on the first CTA's barrier
            const uint32_t counts = PAIR ? map_to_rank(bar, 0) : bar;
            bar_wait(empty + 8 * st.i, st.parity ^ 1u, p.wait_limit_ns, stop_at, late);
            // *stop too: the matrix warp frees stages for the rest of a turn after its own
            // wait gave up, whose full phase still has all its arrivals and misses bytes (a
            // pair's second CTA arrives nowhere: what it copies meanwhile, a turn at most,
            // takes the first one's byte count below zero, which a barrier has room for)
            late |= (uint32_t)*stop;
            n += late ^ 1u;
            if (leader && !late) {
              if (rank == 0)
                mbar_arrive_expect_tx(
                    bar, C::kStage * (PAIR ? 2 : 1) +
                             (tile == first && kb == 0 ? p.missing_tx : 0u));
              tma_load_2d<PAIR>(at, &map_a, kb * 128, ya, counts);
#pragma unroll
              for (int h = 0; h < H; ++h)
                tma_load_2d<PAIR>(at + C::kA + h * (C::kRowsW / H) * 128, &map_w, kb * 128,
                                  yw + h * C::kBufCols, counts);
            }
            __syncwarp();
          }
          late = any_late(late);
        }
      }
      if (leader) *issued = n;
    } else if (warp == 1 && rank == 0) {
      // One K block after the other, whatever tile it belongs to: every block
      // begins its sums anew.  S blocks a turn, so that slots, buffers and
      // descriptors are constants.
      constexpr uint32_t instr = e4m3_instr(C::kTileM, C::kBufCols);
      static_assert(S * H % NB == 0, "a turn goes round both rings");
      constexpr uint32_t flips = S * H / NB % 2;   // whether a turn flips the buffers' parity
      const uint32_t da = operand_desc(sbase), dw = operand_desc(sbase + C::kA);
      const int64_t blocks = first < tiles ? ((tiles - first + step - 1) / step) * p.kblocks : 0;
      uint32_t parity = 0, stored = 0, drained = 1;   // answers on what comes next
      for (int64_t n = 0; n < blocks && !late; n += S, parity ^= 1u) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if (n + i >= blocks) break;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            constexpr int kLast = S * H - 1;
            const int u = i * H + h, b = u % NB;
            bar_wait(tempty + 8 * b, (parity & flips) ^ (u / NB & 1) ^ 1u, p.wait_limit_ns,
                     stop_at, late, drained);
            if (h == 0)
              bar_wait(full + 8 * i, parity, p.wait_limit_ns, stop_at, late, stored);
            const int v = u == kLast ? 0 : u + 1;
            const uint32_t turn = u == kLast ? parity ^ 1u : parity;
            if (h == H - 1) stored = bar_test(full + 8 * (v / H), turn);
            drained = bar_test(tempty + 8 * (v % NB), (turn & flips) ^ (v / NB & 1) ^ 1u);
            tcgen05_fence_after();
            if (leader) {   // (a look at `late` here costs 2 % of a product)
              constexpr uint32_t kNext = C::kStage >> 4, kHalf = C::kRowsW / H * 128 >> 4;
              mma_block<PAIR>(tmem + b * C::kBufCols, da + i * kNext, dw + i * kNext + h * kHalf,
                              instr);
              mma_commit<PAIR>(tfull + 8 * b);
              if (h == H - 1) mma_commit<PAIR>(empty + 8 * i);
            }
            __syncwarp();
          }
        }
        late = any_late(late);
      }
    } else if (warp > 1) {
      // scale warps: lanes 8 r .. 8 r + 7 copy the eight scales of a row; of W
      // without ROWS, the eight of each 128-row block
      const int sub = (warp - 2) * 4 + (lane >> 3), kl = lane & 7;
      RingSlot<kPieces> pc;
      for (int64_t tile = first; tile < tiles && !late; tile += step) {
        int tm, tn;
        tile_at(p, tile, &tm, &tn);
        const int64_t m0 = (int64_t)tm * C::kTileM + rank * 128, n0 = (int64_t)tn * BN;
        for (int k0 = 0; k0 < p.kblocks && !late; k0 += kChunk) {
          bar_wait(sempty + 8 * pc.i, pc.parity ^ 1u, p.wait_limit_ns, stop_at, late);
          const uint32_t dst = sbase + C::kScaleOff + 4 * (pc.i * kChunk + kl) * C::kScales;
          const int64_t at = k0 + kl;
          const bool in = at < p.kblocks;
          stage_scales<128>(dst, p.sa, m0, p.M, at, p.kblocks, in, sub, [](int r) {
            return ROWS ? row_place(r) : r;
          });
          if constexpr (ROWS)
            stage_scales<BN>(dst + 4 * 128, p.sw, n0, p.N, at, p.kblocks, in, sub, column_place);
          else
            stage_scales<BN / 128>(dst + 4 * 128, p.sw, n0 / 128, (p.N + 127) / 128, at, p.kblocks,
                                   in, sub, [](int r) { return r; });
          copy_async_arrive(sfull + 8 * pc.i);
          pc.advance();
          late = any_late(late);
        }
      }
    }
  } else {
    if (PAIR) registers_up<C::kRegsUp>();
    constexpr int COLS = C::kCols;
    constexpr int LOADED = ROWS ? 16 : 32, STEPS = COLS * 32 / (32 * LOADED);   // even
    const int group = (warp - 4) >> 2;
    const int quarter = (warp & 3) * 32, row = quarter + lane;
    const uint32_t mine = tmem + ((uint32_t)quarter << 16) + COLS * group;
    const int wblock = ROWS ? COLS * group : COLS * group / 128;
    const uint32_t drained = PAIR ? map_to_rank(tempty, 0) : tempty;
    RingSlot<C::kRing> tb;   // this group's buffers, or both groups'
    RingSlot<kPieces> pc;
    uint32_t v[2][LOADED];
    auto bar_of = [&](int i) { return 8 * (H * i + (H == 2 ? group : 0)); };
    // step j of a block: its columns 32 j .. + 31; ROWS: its columns 32 (j / 2)
    // .. + 31, the upper 16 rows and then the lower
    auto load = [&](int j) {
      const uint32_t at = mine + tb.i * BN;
      if constexpr (ROWS)
        tmem_load_fragments(v[j & 1], at + 32 * (j >> 1) + ((uint32_t)(j & 1) << 20));
      else
        tmem_load(v[j & 1], at + 32 * j);
    };
    // the block in buffer tb is there: its first step is on its way
    auto begin = [&](uint32_t ready) {
      bar_wait(tfull + bar_of(tb.i), tb.parity, p.wait_limit_ns, stop_at, late, ready);
      __syncwarp();
      tcgen05_fence_after();
      load(0);
    };
    const float* sc = nullptr;   // the scales of the block to come
    // the scales of a block (ROWS: and of its first columns) are asked for a block
    // ahead: shared memory is busy
    float scale = 0.f;
    float4 rows4 = make_float4(0.f, 0.f, 0.f, 0.f), columns[2][2];
    auto ask_rows = [&] {
      if constexpr (ROWS)
        rows4 = *reinterpret_cast<const float4*>(sc + quarter + (lane >> 2) * 4);
      else
        scale = sc[row] * sc[128 + wblock];
    };
    auto ask_columns = [&](const float* of, int c) {   // ROWS: columns 32 c .. + 31
      const float4* w =
          reinterpret_cast<const float4*>(of + 128 + wblock + 32 * c + (lane & 3) * 8);
      columns[c & 1][0] = w[0];
      columns[c & 1][1] = w[1];
    };
    for (int64_t tile = first; tile < tiles && !late; tile += step) {
      int tm, tn;
      tile_at(p, tile, &tm, &tn);
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      bar_wait(sfull + 8 * pc.i, pc.parity, p.wait_limit_ns, stop_at, late);
      __syncwarp();
      sc = scales + pc.i * kChunk * C::kScales;
      ask_rows();
      if constexpr (ROWS) ask_columns(sc, 0);
      begin(0);
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const float s = scale;
        const float r4[4] = {rows4.x, rows4.y, rows4.z, rows4.w};
        const float* here = sc;
        const bool more = kb + 1 < p.kblocks, turn = (kb & (kChunk - 1)) == kChunk - 1;
        const int piece = pc.i;
        sc += C::kScales;
        if (turn || !more) {
          pc.advance();
          if (more) {
            bar_wait(sfull + 8 * pc.i, pc.parity, p.wait_limit_ns, stop_at, late);
            __syncwarp();
            sc = scales + pc.i * kChunk * C::kScales;
          }
        }
        if (more) ask_rows();
        uint32_t ready = 0;
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          tmem_wait(v[j & 1]);
          if (j + 1 < STEPS) {
            load(j + 1);
            if (j + 2 == STEPS) {
              RingSlot<C::kRing> nx = tb;
              nx.advance();
              ready = bar_test(tfull + bar_of(nx.i), nx.parity);
            }
          } else {   // all in registers: the buffer is free, the next block begins
            tcgen05_fence_before();
            arrive_if<PAIR>(drained + bar_of(tb.i), lane == 0);
            tb.advance();
            if (more) begin(ready);
          }
          const uint32_t* x = v[j & 1];
          float* a = acc + LOADED * j;
          if constexpr (ROWS) {
            const int c = j >> 1;
            const float4 w0 = columns[c & 1][0], w1 = columns[c & 1][1];
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            if ((j & 1) == 0) {
              if (c + 1 < COLS / 32)
                ask_columns(here, c + 1);
              else if (more)
                ask_columns(sc, 0);   // COLS / 32 is even
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              a[i] = fmaf(__uint_as_float(x[i]),
                          r4[2 * (j & 1) + (i >> 1 & 1)] * w[(i >> 2) * 2 + (i & 1)], a[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] = fmaf(__uint_as_float(x[i]), s, a[i]);
          }
        }
        if (turn || !more) {
          __syncwarp();
          arrive_if<false>(sempty + 8 * piece, lane == 0);
        }
      }
      late = any_late(late);
      if (late) break;
      const int64_t m0 = (int64_t)tm * C::kTileM + rank * 128 + (warp & 3) * 32;
      const int64_t n0 = (int64_t)tn * BN + COLS * group;
      const int rows = (int)min64(32, p.M - m0), cols = (int)min64(COLS, p.N - n0);   // may be <= 0
      float* yf = static_cast<float*>(p.y) + m0 * p.N + n0;
      __nv_bfloat16* yh = static_cast<__nv_bfloat16*>(p.y) + m0 * p.N + n0;
      if (VEC && ROWS) {
        // whole 32-byte pieces of a row (bf16: halves) by four lanes
#pragma unroll
        for (int i = 0; i < COLS; i += 2) {
          const int r = (i >> 4 & 1) * 16 + (i >> 1 & 1) * 8 + (lane >> 2);
          const int c = (i >> 5) * 32 + (i >> 2 & 3) * 8 + (lane & 3) * 2;
          if (r < rows && c < cols) {
            if (p.fp32_out)
              *reinterpret_cast<float2*>(yf + r * p.N + c) = make_float2(acc[i], acc[i + 1]);
            else
              *reinterpret_cast<uint32_t*>(yh + r * p.N + c) = pack_bf16x2_rn(acc[i], acc[i + 1]);
          }
        }
      } else if (VEC) {
        // N a multiple of 8 (fp32) or 16: whole 32-byte pieces
        if (lane < rows) {
          if (p.fp32_out) {
#pragma unroll
            for (int j = 0; j < COLS; j += 8) {
              const float* a = acc + j;
              if (j < cols)
                st_global_v8(yf + lane * p.N + j, __float_as_uint(a[0]), __float_as_uint(a[1]),
                             __float_as_uint(a[2]), __float_as_uint(a[3]), __float_as_uint(a[4]),
                             __float_as_uint(a[5]), __float_as_uint(a[6]), __float_as_uint(a[7]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < COLS; j += 16) {
              const float* a = acc + j;
              if (j < cols)
                st_global_v8(yh + lane * p.N + j, pack_bf16x2_rn(a[0], a[1]),
                             pack_bf16x2_rn(a[2], a[3]), pack_bf16x2_rn(a[4], a[5]),
                             pack_bf16x2_rn(a[6], a[7]), pack_bf16x2_rn(a[8], a[9]),
                             pack_bf16x2_rn(a[10], a[11]), pack_bf16x2_rn(a[12], a[13]),
                             pack_bf16x2_rn(a[14], a[15]));
            }
          }
        }
      } else {
        float* out = reinterpret_cast<float*>(smem + C::kOutOff) + (warp - 4) * kOutWarp;
        const int c = lane & 7;
#pragma unroll
        for (int j = 0; j < COLS; j += 8) {
          if (j >= cols) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (ROWS)   // fragment values of the upper rows, then of the lower
              out[((i >> 2) * 16 + (i >> 1 & 1) * 8 + (lane >> 2)) * kOutPitch + (lane & 3) * 2 +
                  (i & 1)] = acc[(j >> 5) * 32 + (i >> 2) * 16 + (j >> 3 & 3) * 4 + (i & 3)];
            else
              out[lane * kOutPitch + i] = acc[j + i];
          }
          __syncwarp();
          if (j + c < cols) {
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 4) {
              const int r = r0 + (lane >> 3);
              const float v = out[r * kOutPitch + c];
              const int64_t at = r * p.N + j + c;
              if (r < rows) {
                if (p.fp32_out)
                  yf[at] = v;
                else
                  yh[at] = __float2bfloat16_rn(v);
              }
            }
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (*stop) {   // some lane's wait expired
    if (threadIdx.x == 0) atomicOr(&g_gemm_status, kStatusTimeout);
    drain<S, PAIR>(full, done, *issued, p.wait_limit_ns);
    __syncthreads();
  }
  if (PAIR) {   // no CTA leaves while the other's instructions use its memory
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tcgen05_fence_after();
  if (warp == 1) tmem_free<PAIR>(tmem, 512);
}

// -------------------------------------------------------------- narrow

constexpr int kMostSplit = 8;         // CTAs of a cluster, which share a tile's K
constexpr int kNarrowThreads = 256;   // TMA, MMA, 2 scale warps, 4 epilogue warps

// A stage holds two K blocks: a role's waits and arrivals cost several hundred
// cycles whatever a stage holds, more than the copies and instructions of one
// block.  Two CTAs share an SM: its 512 columns of tensor memory, and shared
// memory for three stages each (TN = 16 with a scale per 128 rows of W) or two.
template <int TN, bool ROWS>
struct Narrow {
  static constexpr int kPer = 2;                          // K blocks per stage
  static constexpr uint32_t kBufCols = kPer * TN;
  static constexpr int kBufs = TN == 64 ? 2 : 4;
  static constexpr uint32_t kCols = kBufCols * kBufs;     // 128 or 256
  static constexpr uint32_t kW = 128 * 128, kA = TN * 128;
  static constexpr uint32_t kStage = kPer * (kW + kA);
  static constexpr int kScales = TN + (ROWS ? 128 : 4);
  static constexpr int kStages = (112640 - kPieces * kChunk * kScales * 4) / (int)kStage;
  static constexpr uint32_t kScaleOff = kStages * kStage;
  static constexpr uint32_t kBarOff = kScaleOff + kPieces * kChunk * kScales * 4;
  static constexpr uint32_t kBytes = kBarOff + 256;
  static constexpr uint32_t kLaunch = kBytes + 1024;
  static_assert(kLaunch <= 233472 / 2 - 1024, "two CTAs per SM");
  static_assert(kChunk % kPer == 0, "a stage's scales lie in one piece");
  static_assert(kScaleOff >= TN * 128 * 4, "the sums for the other CTAs fit the ring");
};

template <int TN, bool ROWS>
__global__ void __launch_bounds__(kNarrowThreads, 2)
narrow_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
              const GemmParams p) {
  using C = Narrow<TN, ROWS>;
  constexpr int S = C::kStages, NB = C::kBufs;
  extern __shared__ unsigned char raw[];
  const uint32_t sbase = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* smem = raw + (sbase - smem_addr(raw));
  float* scales = reinterpret_cast<float*>(smem + C::kScaleOff);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t full = bars, empty = full + 8 * S, tfull = empty + 8 * S, tempty = tfull + 8 * NB,
                 sfull = tempty + 8 * NB, sempty = sfull + 8 * kPieces, done = sempty + 8 * kPieces,
                 slot = done + 8;
  volatile int* stop = reinterpret_cast<volatile int*>(smem + (slot + 4 - sbase));
  int64_t* issued = reinterpret_cast<int64_t*>(smem + (slot + 8 - sbase));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // gridDim.x = tiles of W x CTAs of a cluster, gridDim.y = tiles of A
  int split;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
  const int rank = (int)cluster_ctarank();
  const int tn = (int)blockIdx.x / split;
  const int tm = (int)blockIdx.y;
  // this CTA's stages: pairs of K blocks; the last pair may lack its second
  // one, whose copies read zeros behind the matrices' end
  const int pairs = (p.kblocks + 1) / 2;
  const int u0 = pairs * rank / split, u1 = pairs * (rank + 1) / split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, 4);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(sfull + 8 * i, 64);
      mbar_init(sempty + 8 * i, 4);
    }
    mbar_init(done, 1);
    *stop = 0;
    *issued = 0;
    fence_mbar_init();
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_w);
  }
  if (warp == 1) tmem_alloc<false>(slot, C::kCols);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - sbase));
  grid_dependency_wait();
  allow_dependent_launch();

  const uint32_t stop_at = slot + 4;
  uint32_t late = 0;
  const bool leader = elect_one();
  float acc[TN];
  if (warp == 0) {
    RingSlot<S> st;
    for (int u = u0; u < u1 && !late; ++u, st.advance()) {
      const uint32_t at = sbase + st.i * C::kStage, bar = full + 8 * st.i;
      bar_wait(empty + 8 * st.i, st.parity ^ 1u, p.wait_limit_ns, stop_at, late);
      if (leader && !late) {   // a second arrival in a phase would be one too many
        mbar_arrive_expect_tx(bar, C::kStage + (u == u0 ? p.missing_tx : 0u));
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tma_load_2d<false>(at + i * C::kW, &map_w, (2 * u + i) * 128, tn * 128, bar);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tma_load_2d<false>(at + 2 * C::kW + i * C::kA, &map_a, (2 * u + i) * 128, tm * TN, bar);
        *issued = u + 1 - u0;
      }
      late = any_late(late);
    }
  } else if (warp == 1) {
    constexpr uint32_t instr = e4m3_instr(128, TN);
    RingSlot<S> st;
    RingSlot<NB> tb;
    for (int u = u0; u < u1 && !late; ++u, st.advance(), tb.advance()) {
      const uint32_t dw = operand_desc(sbase + st.i * C::kStage);
      const uint32_t da = operand_desc(sbase + st.i * C::kStage + 2 * C::kW);
      const uint32_t d = tmem + tb.i * C::kBufCols;
      const uint32_t release = empty + 8 * st.i, ready = tfull + 8 * tb.i;
      bar_wait(tempty + 8 * tb.i, tb.parity ^ 1u, p.wait_limit_ns, stop_at, late);
      bar_wait(full + 8 * st.i, st.parity, p.wait_limit_ns, stop_at, late);
      tcgen05_fence_after();
      if (leader && !late) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_block<false>(d + i * TN, dw + i * (C::kW >> 4), da + i * (C::kA >> 4), instr);
        mma_commit<false>(ready);
        mma_commit<false>(release);
      }
      late = any_late(late);
    }
  } else if (warp < 4) {
    const int sub = (warp - 2) * 4 + (lane >> 3), kl = lane & 7;
    RingSlot<kPieces> pc;
    for (int k0 = 2 * u0; k0 < 2 * u1 && !late; k0 += kChunk, pc.advance()) {
      bar_wait(sempty + 8 * pc.i, pc.parity ^ 1u, p.wait_limit_ns, stop_at, late);
      const uint32_t dst = sbase + C::kScaleOff + 4 * (pc.i * kChunk + kl) * C::kScales;
      const int64_t at = k0 + kl;
      const bool in = at < min(2 * u1, p.kblocks);
      const auto place = [](int r) { return r; };
      stage_scales<TN>(dst, p.sa, (int64_t)tm * TN, p.M, at, p.kblocks, in, sub, place);
      stage_scales<ROWS ? 128 : 1>(dst + 4 * TN, p.sw, (int64_t)tn * (ROWS ? 128 : 1),
                                   ROWS ? p.N : tn + 1, at, p.kblocks, in, sub, place);
      copy_async_arrive(sfull + 8 * pc.i);
      late = any_late(late);
    }
  } else {
    const int row = (warp & 3) * 32 + lane;   // of W
    const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[j] = 0.f;
    RingSlot<NB> tb;
    RingSlot<kPieces> pc;
    const float* sc = nullptr;
    for (int u = 0; u < u1 - u0 && !late; ++u, tb.advance(), sc += 2 * C::kScales) {
      constexpr int kTurn = kChunk / 2;   // stages per piece of scales
      if (u % kTurn == 0) {
        bar_wait(sfull + 8 * pc.i, pc.parity, p.wait_limit_ns, stop_at, late);
        sc = scales + pc.i * kChunk * C::kScales;
      }
      bar_wait(tfull + 8 * tb.i, tb.parity, p.wait_limit_ns, stop_at, late);
      late = any_late(late);
      __syncwarp();
      tcgen05_fence_after();
      const uint32_t at = tmem + tb.i * C::kBufCols + lanes;
      constexpr int STEPS = 2 * TN / 16;   // the two blocks' columns, 16 at a time
      uint32_t v[2][16];
      tmem_load(v[0], at);
      const float sw[2] = {sc[TN + (ROWS ? row : 0)], sc[C::kScales + TN + (ROWS ? row : 0)]};
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int half = j / (STEPS / 2), col = 16 * (j % (STEPS / 2));
        tmem_wait(v[j & 1]);
        if (j + 1 < STEPS) tmem_load(v[(j + 1) & 1], at + 16 * (j + 1));
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 s = *reinterpret_cast<const float4*>(sc + half * C::kScales + col + i);
          const uint32_t* x = &v[j & 1][i];
          float* a = acc + col + i;
          a[0] = fmaf(__uint_as_float(x[0]), sw[half] * s.x, a[0]);
          a[1] = fmaf(__uint_as_float(x[1]), sw[half] * s.y, a[1]);
          a[2] = fmaf(__uint_as_float(x[2]), sw[half] * s.z, a[2]);
          a[3] = fmaf(__uint_as_float(x[3]), sw[half] * s.w, a[3]);
        }
      }
      tcgen05_fence_before();
      __syncwarp();
      arrive_if<false>(tempty + 8 * tb.i, lane == 0);
      if (u % kTurn == kTurn - 1) {
        arrive_if<false>(sempty + 8 * pc.i, lane == 0);
        pc.advance();
      }
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (*stop) {   // some lane's wait expired
    if (threadIdx.x == 0) atomicOr(&g_gemm_status, kStatusTimeout);
    drain<S, false>(full, done, *issued, p.wait_limit_ns);
    __syncthreads();
  }
  tcgen05_fence_after();
  if (warp == 1) tmem_free<false>(tmem, C::kCols);

  // The sums of this CTA's K blocks to shared memory (the ring is drained),
  // then every CTA adds its share of the tile over the ranks, in their order.
  float* sums = reinterpret_cast<float*>(smem);   // [TN][128]
  if (warp >= 4) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < TN; ++j) sums[j * 128 + row] = acc[j];
  }
  cluster_arrive_release();
  cluster_wait_acquire();
  const int rows = (int)min64(TN, p.M - (int64_t)tm * TN);
  const bool whole = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
  for (int i = rank * kNarrowThreads + threadIdx.x; i < rows * 32; i += split * kNarrowThreads) {
    const int64_t m = (int64_t)tm * TN + (i >> 5), nn = (int64_t)tn * 128 + 4 * (i & 31);
    float4 x[kMostSplit];
#pragma unroll
    for (int r = 0; r < kMostSplit; ++r)
      if (r < split) x[r] = ld_cluster_f32x4(map_to_rank(sbase + 16 * i, (uint32_t)r));
    float v[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
    for (int r = 1; r < kMostSplit; ++r)
      if (r < split) v[0] += x[r].x, v[1] += x[r].y, v[2] += x[r].z, v[3] += x[r].w;
    float* yf = static_cast<float*>(p.y) + m * p.N + nn;
    __nv_bfloat16* yh = static_cast<__nv_bfloat16*>(p.y) + m * p.N + nn;
    if (whole) {
      if (nn < p.N) {
        if (p.fp32_out)
          *reinterpret_cast<float4*>(yf) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(yh) =
              make_uint2(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (nn + j < p.N) {
          if (p.fp32_out)
            yf[j] = v[j];
          else
            yh[j] = __float2bfloat16_rn(v[j]);
        }
    }
  }
  // no CTA leaves while another reads its sums
  cluster_arrive_release();
  cluster_wait_acquire();
}

// ----------------------------------------------------------------- host

using GemmKernel = void (*)(CUtensorMap, CUtensorMap, GemmParams);

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Map of an E4M3 matrix [rows, K], copied in boxes of box_rows x 128 bytes
// with the 128-byte swizzle; rows and columns outside read as zeros.
int make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int box_rows) {
  const EncodeTiled enc = encode_tiled();
  if (enc == nullptr) return fail(NTS_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                         strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NTS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return NTS_OK;
}

cudaLaunchAttribute cluster_attribute(int cluster) {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)cluster;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

int launch(GemmKernel kern, const GemmRequest& rq, const GemmParams& p, int box_a, int box_w,
           dim3 grid, int threads, int regs, size_t smem, int cluster, cudaStream_t stream,
           bool pdl) {
  CUtensorMap map_a, map_w;
  int rc = make_map(&map_a, rq.A, rq.M, rq.K, box_a);
  if (rc == NTS_OK) rc = make_map(&map_w, rq.W, rq.N, rq.K, box_w);
  if (rc == NTS_OK) rc = prepare_kernel((const void*)kern, smem);
  if (rc != NTS_OK) return rc;
  if (regs > 0) {   // the split of the registers presumes what the CTA is launched with
    int have = 0;
    rc = kernel_registers((const void*)kern, &have);
    if (rc != NTS_OK) return rc;
    if (have != regs)
      return fail(NTS_ERR_UNSUPPORTED, "the product's kernel was built with %d registers, not %d",
                  have, regs);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int na = 0;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  attr[na++] = cluster_attribute(cluster);
  if (pdl) attr[na++] = pdl_attribute();
  cfg.numAttrs = na;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, map_a, map_w, p);
  if (e != cudaSuccess) return fail_cuda(e, "launching the block-scaled product");
  return NTS_OK;
}

template <int TN>
int launch_narrow(const GemmRequest& rq, const GemmParams& p, cudaStream_t stream,
                  const DeviceInfo& dev, const LaunchTuning& tune) {
  const int64_t tiles_n = (p.N + 127) / 128, tiles_m = (p.M + TN - 1) / TN;
  int split = 1;
  while (split < kMostSplit && 4 * split <= p.kblocks && tiles_n * tiles_m * split <= dev.sm_count)
    split *= 2;
  const int64_t gx = tiles_n * split;
  if (gx > 0x7fffffffll || tiles_m > 65535)
    return fail(NTS_ERR_UNSUPPORTED, "too many tiles in one call");
  log_launch("gemm_blockscaled", "M=%lld N=%lld K=%lld narrow TN=%d split=%d", (long long)p.M,
             (long long)p.N, (long long)rq.K, TN, split);
  const dim3 grid((unsigned)gx, (unsigned)tiles_m);
  return rq.w_rows == 1
             ? launch(narrow_kernel<TN, true>, rq, p, TN, 128, grid, kNarrowThreads, 0,
                      Narrow<TN, true>::kLaunch, split, stream, tune.pdl != 0)
             : launch(narrow_kernel<TN, false>, rq, p, TN, 128, grid, kNarrowThreads, 0,
                      Narrow<TN, false>::kLaunch, split, stream, tune.pdl != 0);
}

template <int BN, bool ROWS>
int launch_wide(const GemmRequest& rq, GemmParams p, cudaStream_t stream, const DeviceInfo& dev,
                const LaunchTuning& tune) {
  using C = Wide<BN, ROWS>;
  p.tiles_m = (int)((p.M + C::kTileM - 1) / C::kTileM);
  p.tiles_n = (int)((p.N + BN - 1) / BN);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const int cluster = C::kPair ? 2 : 1;
  const int64_t row_bytes = p.N * (p.fp32_out ? 4 : 2);
  const bool vec = row_bytes % 32 == 0 && reinterpret_cast<uintptr_t>(p.y) % 32 == 0;
  const GemmKernel kern = vec ? wide_kernel<BN, ROWS, true> : wide_kernel<BN, ROWS, false>;
  int64_t most = dev.sm_count;
  if (C::kPair) {
    int rc = prepare_kernel((const void*)kern, C::kLaunch);
    if (rc != NTS_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = cluster_attribute(cluster);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kLaunch;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    rc = max_active_clusters((const void*)kern, cfg, cluster, &most);
    if (rc != NTS_OK) return rc;
  }
  const unsigned grid = (unsigned)(std::min(tiles, most) * cluster);
  log_launch("gemm_blockscaled", "M=%lld N=%lld K=%lld wide %dx%d grid=%u", (long long)p.M,
             (long long)p.N, (long long)rq.K, C::kTileM, BN, grid);
  return launch(kern, rq, p, 128, C::kRowsW / C::kHalves, dim3(grid), C::kThreads, C::kRegs,
                C::kLaunch, cluster, stream, tune.pdl != 0);
}

}  // namespace

int launch_gemm(const GemmRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  note_launch(kGemmUnit);
  GemmParams p = {};
  p.sa = rq.a_scales;
  p.sw = rq.w_scales;
  p.y = rq.Y;
  p.M = rq.M;
  p.N = rq.N;
  p.kblocks = (int)((rq.K + 127) / 128);
  p.fp32_out = rq.fp32_out;
  p.wait_limit_ns = tune.wait_limit_ns;
  p.missing_tx = tune.missing_tx;
  enum { kAuto, kNarrow, kWide, kPair };
  int kind = tune.force_vpt <= kPair ? tune.force_vpt : kAuto;   // debug: one of these
  if (kind == kAuto) {
    // Few tiles of 128 x 128: their K loops leave SMs idle, and narrow_kernel
    // splits K (us, narrow / one CTA, bf16 with 128-row scales, then fp32 with a
    // scale per row of W: [200, 4096] x [1024, 4096] 7.8 / 12.1, 8.1 / 16.1; [100,
    // 4096] x [4096, 4096] 9.7 / 12.5, 10.3 / 16.3; [128, 5120] x [5120, 5120], 40
    // tiles, 14.8 / 15.1, 17.1 / 20.2; [128, 5120] x [15360, 5120] 27.2 / 18.7,
    // 31.0 / 22.0).  Up to 64 rows of A it reads W with less waste and holds out
    // longer ([64, 5120] x [5120, 5120] 10.7 / 14.5, 11.9 / 19.2; [64, 5120] x
    // [15360, 5120] 18.8 / 17.8, 20.2 / 21.2), up to 32 always ([32, 5120] x [15360,
    // 5120] 17.1 / 17.4, 17.6 / 20.6).
    const int64_t ones = (p.M + 127) / 128 * ((p.N + 127) / 128);
    const int64_t pairs = (p.M + 255) / 256 * ((p.N + 255) / 256);
    const int64_t sms = dev.sm_count;
    if (p.M <= 32 || 4 * ones <= sms || (p.M <= 64 && 2 * ones <= sms)) {
      kind = kNarrow;
    } else {
      // A K block takes a pair ~1.5 times as long as one CTA, with either layout of
      // W's scales: by the rounds of tiles (us, one CTA / pair, bf16 with 128-row
      // scales, then fp32 with a scale per row, by [5120, 5120]: [333, 5120], one
      // round of each, 15.4 / 22.3, 20.6 / 32.8; [512, 5120], two and one, 27.6 /
      // 22.5, 38.1 / 32.7; [1024, 5120], three and two, 39.8 / 41.1, 55.7 / 61.9;
      // [2048, 5120], five and three, 64.4 / 60.1, 90.9 / 90.4).
      const int64_t rounds = (ones + sms - 1) / sms, rounds2 = (pairs + sms / 2 - 1) / (sms / 2);
      kind = 2 * rounds <= 3 * rounds2 ? kWide : kPair;
    }
  }
  if (kind == kNarrow) {
    if (p.M <= 16) return launch_narrow<16>(rq, p, stream, dev, tune);
    if (p.M <= 32) return launch_narrow<32>(rq, p, stream, dev, tune);
    return launch_narrow<64>(rq, p, stream, dev, tune);
  }
  if (kind == kPair)
    return rq.w_rows == 1 ? launch_wide<256, true>(rq, p, stream, dev, tune)
                          : launch_wide<256, false>(rq, p, stream, dev, tune);
  return rq.w_rows == 1 ? launch_wide<128, true>(rq, p, stream, dev, tune)
                        : launch_wide<128, false>(rq, p, stream, dev, tune);
}

int read_and_clear_gemm_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemm_status, sizeof(v));
  if (e != cudaSuccess) return fail_cuda(e, "reading the product's status word");
  if (v != 0) e = cudaMemcpyToSymbol(g_gemm_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return fail_cuda(e, "clearing the product's status word");
  *out = v;
  return NTS_OK;
}

}  // namespace nts
