// gemv_tile.cuh -- the kernel of the products of more than 16 rows with 4-bit weights
// (gemv_launch.cu describes it); instantiated in gemv_e2m1.cu and gemv_int4.cu.
#pragma once

#include "gemm_device.cuh"
#include "gemv_kernel.cuh"

namespace nts {

namespace {

// kStatusTimeout bits of these kernels.
__device__ unsigned int g_gemv_status;

constexpr int kTeam = 4;             // warps of a team: two for the codes, two for the sums
constexpr int kScalesAhead = 4;      // K blocks of a team
constexpr int kCodesAhead = 12;      // K blocks

template <int G, bool E4M3>
struct Tile {
  static constexpr int TN = kTileRows;
  static constexpr int kGroups = 128 / G;      // of a K block
  static constexpr int kByte = E4M3 ? 1 : 2;   // of an operand's value
  static constexpr uint32_t kA = 128 * 128 * kByte, kB = TN * 128 * kByte, kStage = kA + kB;
  // A team's stages, all that leave an SM one CTA of these kernels (more than that cost
  // L1: with all of an SM's shared memory asked for, 25.5 us in place of 24.5 below).
  static constexpr int kStages = E4M3 ? 4 : 2;
  static constexpr uint32_t kBufCols = kGroups * TN;
  static constexpr int kBufs = 2;              // of a team, in tensor memory
  static constexpr uint32_t kCols = 2 * kBufs * kBufCols;
  static constexpr uint32_t kFactorOff = 2 * kStages * kStage;
  static constexpr uint32_t kBarOff = kFactorOff + 2 * kTeam * 2 * TN * 4;
  static constexpr uint32_t kLaunch = kBarOff + 512 + 1024;
  static_assert(kCols >= 32 && kCols <= 512 && (kCols & (kCols - 1)) == 0, "tensor memory");
  static_assert(kStages * kStage >= TN * 128 * 4, "the sums for the other CTAs fit the ring");
  static_assert(kLaunch <= 232448 && kLaunch >= 160 * 1024, "one CTA per SM");
};

__device__ __forceinline__ uint32_t permute(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}

// Eight codes as bf16 (o[0..3], in pairs) or E4M3 (o[0..1]), in their order.  A byte
// permutation looks up four codes' bytes in a table of eight by the low three bits; by
// the fourth it repeats a byte's top bit, which makes 0x80 of a code without it and 0xFF
// of one with it.
template <bool INT4, bool E4M3>
__device__ __forceinline__ void decode8_natural(uint32_t w, uint32_t (&o)[4]) {
  if constexpr (INT4 && !E4M3) {
    // the code under 128's last places, its offset taken off
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = ((w >> 4 * j) & 0x000F000Fu) ^ 0x43084308u;
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(q[j]) : "r"(v), "r"(0xC308C308u));   // -136
    }
    o[0] = permute(q[0], q[1], 0x5410);
    o[1] = permute(q[2], q[3], 0x5410);
    o[2] = permute(q[0], q[1], 0x7632);
    o[3] = permute(q[2], q[3], 0x7632);
  } else {
    const uint32_t low3 = w & 0x77777777u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sel = low3 >> 16 * h;
      // per byte: the top seven bits set below a code with its fourth bit, else clear
      const uint32_t sign = permute(0x80808080u, 0x80808080u, w >> 16 * h) << 1;
      if constexpr (E4M3 && INT4) {
        const uint32_t pos = permute(0x44403800u, 0x4E4C4A48u, sel);   // 0 .. 7
        const uint32_t neg = permute(0xCACCCED0u, 0xB8C0C4C8u, sel);   // -8 .. -1
        o[h] = (pos & ~sign) | (neg & sign);   // the last place of all is clear
      } else if constexpr (E4M3) {
        o[h] = permute(0x3C383000u, 0x4C484440u, sel) | (sign & 0x80808080u);
      } else {
        const uint32_t lo = permute(0xC0800000u, 0xC0804000u, sel);
        const uint32_t hi = permute(0x3F3F3F00u, 0x40404040u, sel) | (sign & 0x80808080u);
        o[2 * h] = permute(lo, hi, 0x5140);
        o[2 * h + 1] = permute(lo, hi, 0x7362);
      }
    }
  }
}

// D (+)= A B^T over 32 bytes of K, E4M3 or bf16 operands; one thread.
template <bool E4M3>
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                         uint32_t add) {
  if constexpr (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "r"(kDescHigh), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "r"(kDescHigh), "r"(add)
        : "memory");
}

// 8 columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ uint4 ldg_codes(const unsigned char* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

template <bool INT4, int G, bool E4M3>
__global__ void __launch_bounds__(kTileThreads, 1)
gemv_tile_kernel(const __grid_constant__ CUtensorMap rows, const GemvParams p) {
  using C = Tile<G, E4M3>;
  constexpr int S = C::kStages, NB = C::kBufs, TN = C::TN;
  extern __shared__ unsigned char raw[];
  const uint32_t sbase = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* smem = raw + (sbase - smem_addr(raw));
  // per team: a stage's codes are turned, its rows of A are there, it is used up; a buffer
  // of tensor memory holds its sums, they are read
  const uint32_t full = sbase + C::kBarOff, bfull = full + 16 * S, empty = bfull + 16 * S,
                 tfull = empty + 16 * S, tempty = tfull + 16 * NB, done = tempty + 16 * NB,
                 slot = done + 16;
  volatile int* stop = reinterpret_cast<volatile int*>(smem + (slot + 4 - sbase));
  int* issued = reinterpret_cast<int*>(smem + (slot + 8 - sbase));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // gridDim.x = tiles of W x CTAs of a cluster, gridDim.y = tiles of A
  const int split = p.cluster;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = (int)blockIdx.x / split * 128, m0 = (int)blockIdx.y * TN;
  const int b0 = p.kb * rank / split, b1 = p.kb * (rank + 1) / split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S; ++i) {
      mbar_init(full + 8 * i, kTeam);
      mbar_init(bfull + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2 * NB; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, kTeam);
    }
    mbar_init(done, 1);
    mbar_init(done + 8, 1);
    *stop = 0;
    *issued = 0;
    fence_mbar_init();
    prefetch_tensor_map(&rows);
  }
  constexpr int kDrainAt = 2 * kTeam, kMmaAt = 2 * kDrainAt, kLoadAt = kMmaAt + 2;
  static_assert(kTileThreads == 32 * (kLoadAt + 1), "the roles' warps");
  // The wait for columns of tensor memory has no limit: a CTA of another kernel on this SM
  // may hold them, and while these are held here it may wait for them.  So a CTA holds
  // columns only while it waits for nothing outside itself, and whoever wants them gets
  // them: it takes them when the launch before is done, lets the next one in, which may
  // want columns too, when it has them, and gives them back before it meets its peers.
  // (Taken before the launch before is done: 24.3 us in place of 24.5.)
  grid_dependency_wait();
  if (warp == kMmaAt) tmem_alloc<false>(slot, C::kCols);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - sbase));
  allow_dependent_launch();

  const uint32_t stop_at = slot + 4;
  uint32_t late = 0;
  const bool leader = elect_one();
  float acc[TN];
  if (warp < kDrainAt) {
    // The teams take the K blocks in turn; a thread takes 32 codes of four rows.
    const int team = warp / kTeam;
    // Eight lanes store 16 bytes each without a conflict: with E4M3 two rows of four chunks,
    // with bf16 four rows, two chunks of one half of the block each.
    const int row = warp % kTeam * 8 + (E4M3 ? lane >> 2 : (lane >> 4) * 4 + (lane >> 1 & 3));
    const int part = E4M3 ? lane & 3 : (lane >> 2 & 2) | (lane & 1);
    const unsigned char* codes = p.w + (int64_t)(n0 + row) * (p.K / 2) + 16 * part;
    const int64_t down = 32 * (int64_t)(p.K / 2);
    uint4 w[2][4];
    auto load_codes = [&](int b, uint4 (&v)[4]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = make_uint4(0, 0, 0, 0);
        if (n0 + row + 32 * c < p.N && b < b1 && 128 * b + 32 * part < p.K)
          v[c] = ldg_codes(codes + 64 * (int64_t)b + c * down);
      }
    };
    load_codes(b0 + team, w[0]);
    load_codes(b0 + team + 2, w[1]);
    const uint32_t to = E4M3 ? row * 128 : (part >> 1) * (C::kA / 2) + row * 128;
    const uint32_t turn = E4M3 ? (uint32_t)((row & 7) ^ 2 * part)
                               : (uint32_t)((row & 7) ^ 4 * (part & 1));
    RingSlot<S> st;
    uint32_t ready = 0;
    for (int b = b0 + team; b < b1 && !late; b += 4) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (b + 2 * u >= b1) break;
        const int stage = team * S + st.i;
        const uint32_t at = sbase + stage * C::kStage + to;
        bar_wait(empty + 8 * stage, st.parity ^ 1u, p.wait_limit_ns, stop_at, late, ready);
        st.advance();
        ready = bar_test(empty + 8 * (team * S + st.i), st.parity ^ 1u);   // of the next one
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = w[u][c];
          uint32_t o[4][4];
          if constexpr (E4M3) {
            decode8_natural<INT4, E4M3>(v.x, o[0]);
            decode8_natural<INT4, E4M3>(v.y, o[1]);
            decode8_natural<INT4, E4M3>(v.z, o[2]);
            decode8_natural<INT4, E4M3>(v.w, o[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              sts128(at + c * 32 * 128 + (((uint32_t)i ^ turn) << 4), o[2 * i][0], o[2 * i][1],
                     o[2 * i + 1][0], o[2 * i + 1][1]);
          } else {
            decode8_natural<INT4, E4M3>(v.x, o[0]);
            decode8_natural<INT4, E4M3>(v.y, o[1]);
            decode8_natural<INT4, E4M3>(v.z, o[2]);
            decode8_natural<INT4, E4M3>(v.w, o[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts128(at + c * 32 * 128 + (((uint32_t)i ^ turn) << 4), o[i][0], o[i][1], o[i][2],
                     o[i][3]);
          }
        }
        load_codes(b + 2 * u + 4, w[u]);
        fence_proxy_async_smem();
        __syncwarp();
        arrive_if<false>(full + 8 * stage, lane == 0);
      }
      late = any_late(late);
    }
  } else if (warp < kMmaAt) {
    const int team = (warp - kDrainAt) / kTeam;
    const int row = (warp & 3) * 32 + lane;   // of W
    const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
    const __nv_bfloat16* scale = p.s + (int64_t)(n0 + row) * p.groups;
    const bool in = n0 + row < p.N;
    const float* factor = p.a_scales + (int64_t)(m0 + lane) * p.kb;   // E4M3
    const bool in_row = E4M3 && m0 + lane < p.M;
    float* factors = reinterpret_cast<float*>(smem + C::kFactorOff) + (warp - kDrainAt) * 2 * TN;
    static_assert(TN == 32, "a lane for each row of A");
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[j] = 0.f;
    constexpr int WORDS = (C::kGroups + 1) / 2;
    uint32_t next[kScalesAhead][WORDS];   // a block's scales
    float next_factor[kScalesAhead];
    auto load_scales = [&](int b, uint32_t (&v)[WORDS], float& f) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) v[i] = 0;
      if (E4M3) f = 0.f;
      if (b >= b1) return;
      if (in_row) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(f) : "l"(factor + b));
      if (!in) return;
      const __nv_bfloat16* at = scale + b * C::kGroups;
      if (p.vector && C::kGroups > 1) {   // they are one aligned word
        if constexpr (C::kGroups == 4)
          asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(at));
        else
          asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v[0]) : "l"(at));
        return;
      }
#pragma unroll
      for (int i = 0; i < C::kGroups; ++i) {
        if (b * C::kGroups + i >= p.groups) break;
        uint16_t s;
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(s) : "l"(at + i));
        v[i / 2] |= (uint32_t)s << 16 * (i & 1);
      }
    };
#pragma unroll
    for (int u = 0; u < kScalesAhead; ++u) load_scales(b0 + team + 2 * u, next[u], next_factor[u]);
    RingSlot<NB> tb;
    uint32_t ready = 0;
    for (int bb = b0 + team; bb < b1 && !late; bb += 2 * kScalesAhead) {
#pragma unroll
      for (int u = 0; u < kScalesAhead; ++u) {
        if (bb + 2 * u >= b1) break;
        float sc[C::kGroups];
#pragma unroll
        for (int i = 0; i < C::kGroups; ++i)
          sc[i] = __uint_as_float(i & 1 ? next[u][i / 2] & 0xFFFF0000u : next[u][i / 2] << 16);
        float* f = factors + (u & 1) * TN;
        if (E4M3) f[lane] = next_factor[u];
        load_scales(bb + 2 * (u + kScalesAhead), next[u], next_factor[u]);
        const int buf = team * NB + tb.i;
        bar_wait(tfull + 8 * buf, tb.parity, p.wait_limit_ns, stop_at, late, ready);
        __syncwarp();
        tcgen05_fence_after();
        const uint32_t at = tmem + buf * C::kBufCols + lanes;
        // the groups' sums of eight columns at a time, the next ones on their way (not where
        // the registers do not hold them)
        constexpr int kAhead = E4M3 && C::kGroups == 4 ? 0 : 1;
        uint32_t v[kAhead + 1][C::kGroups][8];
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) tmem_load(v[0][g], at + g * TN);
        tb.advance();
        ready = bar_test(tfull + 8 * (team * NB + tb.i), tb.parity);   // the next block's
#pragma unroll
        for (int c = 0; c < TN / 8; ++c) {
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g) {
            if (kAhead == 0 && c > 0) tmem_load(v[0][g], at + g * TN + 8 * c);
          }
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g) tmem_wait(v[c & kAhead][g]);
          if (kAhead == 1 && c + 1 < TN / 8) {
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g)
              tmem_load(v[(c + 1) & 1][g], at + g * TN + 8 * (c + 1));
          }
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            float s[4];
            if (E4M3) {
              const float4 s4 = *reinterpret_cast<const float4*>(f + 8 * c + i);
              s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& a = acc[8 * c + i + e];
              float d = E4M3 ? __uint_as_float(v[c & kAhead][0][i + e]) * sc[0]
                             : fmaf(__uint_as_float(v[c & kAhead][0][i + e]), sc[0], a);
#pragma unroll
              for (int g = 1; g < C::kGroups; ++g)
                d = fmaf(__uint_as_float(v[c & kAhead][g][i + e]), sc[g], d);
              a = E4M3 ? fmaf(d, s[e], a) : d;
            }
          }
        }
        tcgen05_fence_before();
        __syncwarp();
        arrive_if<false>(tempty + 8 * buf, lane == 0);
      }
      late = any_late(late);
    }
  } else if (warp < kLoadAt) {
    constexpr uint32_t instr = e4m3_instr(128, TN) | (E4M3 ? 0u : 1u << 7 | 1u << 10);
    const int team = warp - kMmaAt;
    RingSlot<S> st;
    RingSlot<NB> tb;
    for (int b = b0 + team; b < b1 && !late; b += 2, st.advance(), tb.advance()) {
      const int stage = team * S + st.i, buf = team * NB + tb.i;
      const uint32_t da = operand_desc(sbase + stage * C::kStage);
      const uint32_t db = operand_desc(sbase + stage * C::kStage + C::kA);
      const uint32_t d = tmem + buf * C::kBufCols;
      bar_wait(tempty + 8 * buf, tb.parity ^ 1u, p.wait_limit_ns, stop_at, late);
      bar_wait(bfull + 8 * stage, st.parity, p.wait_limit_ns, stop_at, late);
      bar_wait(full + 8 * stage, st.parity, p.wait_limit_ns, stop_at, late);
      tcgen05_fence_after();
      if (leader && !late) {
        constexpr int kPer = 32 / C::kByte;   // values of a step; four to 128 bytes
#pragma unroll
        for (int k = 0; k < 128 / kPer; ++k)
          mma_step<E4M3>(d + kPer * k / G * TN, da + (k >> 2) * (C::kA >> 5) + (k & 3) * 2,
                         db + (k >> 2) * (C::kB >> 5) + (k & 3) * 2, instr, kPer * k % G != 0);
        mma_commit<false>(tfull + 8 * buf);
        mma_commit<false>(empty + 8 * stage);
      }
      late = any_late(late);
    }
  } else {
    // Lines of codes (two K blocks) and of scales of four rows a lane, on their way to L2:
    // a load from there is covered by the two blocks that a team's threads hold ahead.
    auto prefetch = [&](int b) {
      constexpr int kPerLine = 64 / C::kGroups;   // K blocks of a line of scales
      const bool codes = b % 2 == 0 || b == b0, sc = b % kPerLine == 0 || b == b0;
      if (b >= b1 || !(codes || sc)) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + lane + 32 * i;
        if (n >= p.N) break;
        if (codes) prefetch_l2(p.w + n * (p.K / 2) + 64 * b);
        if (sc) prefetch_l2(p.s + n * p.groups + b * C::kGroups);
      }
    };
    for (int b = b0; b < b0 + kCodesAhead; ++b) prefetch(b);
    RingSlot<S> st;
    for (int b = b0; b < b1 && !late; ++b) {
      prefetch(b + kCodesAhead);
      const int stage = (b - b0 & 1) * S + st.i;
      const uint32_t at = sbase + stage * C::kStage + C::kA, bar = bfull + 8 * stage;
      bar_wait(empty + 8 * stage, st.parity ^ 1u, p.wait_limit_ns, stop_at, late);
      if (leader && !late) {   // a second arrival in a phase would be one too many
        mbar_arrive_expect_tx(bar, C::kB + (b == b0 ? p.missing_tx : 0u));
#pragma unroll
        for (int h = 0; h < C::kByte; ++h)
          tma_load_2d<false>(at + h * (C::kB / C::kByte), &rows, 128 * b + 64 * h, m0, bar);
        *issued = b + 1 - b0;
      }
      late = any_late(late);
      if (b - b0 & 1) st.advance();
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (*stop) {   // some lane's wait expired: copies and instructions in flight end
    if (threadIdx.x == 0) {
      atomicOr(&g_gemv_status, kStatusTimeout);
      for (int j = max(0, *issued - 2 * S); j < *issued; ++j)
        (void)mbar_wait_bounded(bfull + 8 * ((j & 1) * S + (j >> 1) % S),
                                (uint32_t)((j >> 1) / S & 1), p.wait_limit_ns);
    }
    if (warp >= kMmaAt && warp < kLoadAt && elect_one()) {   // the threads that issue them
      mma_commit<false>(done + 8 * (warp - kMmaAt));
      (void)mbar_wait_bounded(done + 8 * (warp - kMmaAt), 0, p.wait_limit_ns);
    }
    __syncthreads();
  }
  tcgen05_fence_after();
  if (warp == kMmaAt) tmem_free<false>(tmem, C::kCols);

  // The sums of this CTA's K blocks to shared memory (the operands are used up), then
  // every CTA of the cluster adds its share of the tile over the ranks and their teams, in
  // their order.
  float* sums = reinterpret_cast<float*>(smem);   // [team][row of A][128]
  if (warp >= kDrainAt && warp < kMmaAt) {
    float* out = sums + (warp - kDrainAt) / kTeam * TN * 128 + (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < TN; ++j) out[j * 128] = acc[j];
  }
  if (split > 1) {
    cluster_arrive_release();
    cluster_wait_acquire();
  } else {
    __syncthreads();
  }
  const int here = min(TN, p.M - m0), cols = min(128, p.N - n0);
  for (int i = rank * kTileThreads + threadIdx.x; i < here * 128; i += split * kTileThreads) {
    const int m = i >> 7, n = i & 127;
    if (n >= cols) continue;
    float v = 0.f;
    if (split > 1) {
      for (int r = 0; r < split; ++r) {
        const uint32_t from = map_to_rank(sbase + 4 * i, (uint32_t)r);
        float x, y;
        asm volatile("ld.shared::cluster.f32 %0, [%2];\n\tld.shared::cluster.f32 %1, [%2 + %3];"
                     : "=f"(x), "=f"(y)
                     : "r"(from), "n"(TN * 128 * 4)
                     : "memory");
        v += x + y;
      }
    } else {
      v = sums[i] + sums[i + TN * 128];
    }
    const int64_t out = (int64_t)(m0 + m) * p.N + n0 + n;
    if (p.fp32)
      static_cast<float*>(p.y)[out] = v;
    else
      static_cast<__nv_bfloat16*>(p.y)[out] = __float2bfloat16_rn(v);
  }
  if (split > 1) {   // no CTA leaves while another reads its sums
    cluster_arrive_release();
    cluster_wait_acquire();
  }
}

template <bool INT4, int G>
GemvTileKernel pick_tile(bool e4m3, size_t* smem) {
  *smem = e4m3 ? Tile<G, true>::kLaunch : Tile<G, false>::kLaunch;
  return e4m3 ? gemv_tile_kernel<INT4, G, true> : gemv_tile_kernel<INT4, G, false>;
}

}  // namespace

template <bool INT4>
GemvTileKernel pick_gemv_tile(int group, bool e4m3, size_t* smem) {
  return group == 32   ? pick_tile<INT4, 32>(e4m3, smem)
         : group == 64 ? pick_tile<INT4, 64>(e4m3, smem)
                       : pick_tile<INT4, 128>(e4m3, smem);
}

template <bool INT4>
int read_and_clear_gemv_unit(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemv_status, sizeof(v));
  if (e != cudaSuccess) return fail_cuda(e, "reading the 4-bit product's status word");
  if (v != 0) e = cudaMemcpyToSymbol(g_gemv_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return fail_cuda(e, "clearing the 4-bit product's status word");
  *out = v;
  return NTS_OK;
}

}  // namespace nts
