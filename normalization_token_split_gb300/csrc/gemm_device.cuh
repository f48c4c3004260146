// gemm_device.cuh -- inline-PTX building blocks of the block-scaled matrix
// product: tensor-map copies, tcgen05 matrix instructions with accumulators
// in tensor memory (TMEM), and waits that end when any role of the CTA gave up.
#pragma once

#include <cuda.h>   // CUtensorMap

#include "nts_device.cuh"

namespace nts {

// Whether a phase of `bar` is complete, without waiting.  While the matrix
// instructions and the copies keep shared memory busy, an answer takes ~170
// cycles (24 on an idle SM): asked for early, it is there when it is needed.
__device__ __forceinline__ uint32_t bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}

// A bounded wait for a phase of `bar`, at once over when `done` (an earlier
// answer of bar_test) is set.  It costs a satisfied wait two branches and no
// vote: a role's loop passes several for every K block, and at ~25 cycles a
// branch they decide how fast it turns.  A wait that expires (limit_ns, or
// another role of the CTA set *stop) sets *stop and `late`; once `late` is set
// the waits that follow return at once, so a role may look at it only now and
// then, as long as what it does meanwhile stays inside its own memory and arrives
// at no barrier that counts bytes: all arrivals of such a phase may be there
// while bytes are missing, and one more is a fault.  Every lane tries and reads
// the clock by itself, so `late` is a lane's own: a loop that holds instructions
// of the whole warp is left on any_late.  The clock is read only after many
// tries: a read takes longer than most waits.
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                         uint32_t stop, uint32_t& late, uint32_t done = 0) {
  asm volatile(
      "{\n\t"
      ".reg .pred p, q;\n\t"
      ".reg .u64 t0, t;\n\t"
      ".reg .u32 n;\n\t"
      "setp.ne.u32 q, %5, 0;\n\t"
      "@q bra DONE;\n\t"
      "mov.u32 n, 0;\n"
      "TRY:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 64;\n\t"
      "@q bra TRY;\n\t"
      "mov.u64 t0, %%globaltimer;\n"
      "SLOW:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.u32 n, [%4];\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra LATE;\n\t"
      "mov.u64 t, %%globaltimer;\n\t"
      "sub.u64 t, t, t0;\n\t"
      "setp.le.u64 q, t, %3;\n\t"
      "@q bra SLOW;\n"
      "LATE:\n\t"
      "mov.u32 %0, 1;\n\t"
      "st.volatile.shared.u32 [%4], 1;\n"
      "DONE:\n\t"
      "}"
      : "+r"(late)
      : "r"(bar), "r"(parity), "l"(limit_ns), "r"(stop), "r"(done | late)
      : "memory");
}

// Whether a wait of any lane of the warp expired (a place where its lanes meet
// again).  Lanes that left a role's loop by their own answers would meet the
// others' warp-wide instructions at another place.
__device__ __forceinline__ uint32_t any_late(uint32_t late) {
  return __any_sync(0xFFFFFFFFu, late != 0) != 0;
}

// Arrive on `bar` from the lanes with on != 0, without a branch.  CLUSTER: a
// barrier of a CTA of this cluster (an address of map_to_rank), without a
// cluster-wide release: what it orders are tensor-memory loads that their own
// wait has completed, and a release at cluster scope took ~1300 cycles.
template <bool CLUSTER>
__device__ __forceinline__ void arrive_if(uint32_t bar, bool on) {
  if (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"((uint32_t)on)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"((uint32_t)on)
        : "memory");
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A place in a ring of N barriers: the slot and the parity of its phase.
template <int N>
struct RingSlot {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance() {
    if (++i == N) {
      i = 0;
      parity ^= 1u;
    }
  }
};

// Moves registers between the warpgroups of a CTA: every warp of a group of
// four executes it.  The sum over the groups stays what the CTA was launched with.
template <int R>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// Box of a 2-D tensor map, element (x, y) first, into shared memory.  x in
// elements of one byte, a multiple of 16.  PAIR: `bar` may be the barrier of
// either CTA of a pair (a cluster address).
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Allocates `cols` columns of tensor memory (a power of two, 32 to 512) and
// writes their address to shared memory; one whole warp.  The same warp frees
// them.  PAIR: one warp of each CTA of the pair does so.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Descriptor of a shared-memory operand tile: rows of 128 bytes along K,
// 128-byte swizzle, groups of eight rows 1024 bytes apart; the tile starts on
// a 1024-byte boundary and a step of 32 values along K adds 32 bytes.  The
// upper word is the same for every tile; this is the lower one.
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t operand_desc(uint32_t addr) {
  return (addr & 0x3FFFFu) >> 4 | 1u << 16;
}

// Instruction descriptor for E4M3 x E4M3 -> fp32, both operands along K,
// m x n tile.
__host__ __device__ constexpr uint32_t e4m3_instr(int m, int n) {
  return 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// D = A B^T over one K block (128 values, four steps of which the first
// overwrites D); one thread; a and b are operand_desc words.  PAIR: the two
// CTAs' halves of A's rows (each CTA's shared memory) times both halves of B's
// rows (one in each CTA); each CTA's tensor memory takes its rows of D.  One
// asm block, so that no step's descriptors stay in registers.
template <bool PAIR>
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a, uint32_t b, uint32_t instr) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.u32 p, %4, %4;\n\t"
        "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "setp.eq.u32 p, %4, %4;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "r"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.u32 p, %4, %4;\n\t"
        "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "setp.eq.u32 p, %4, %4;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\t"
        "mov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "r"(kDescHigh)
        : "memory");
}

// Arrive on `bar` (PAIR: on that barrier in both CTAs) once every matrix
// instruction issued so far by this thread is complete.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// 16 or 32 columns of this warp's 32 lanes of tensor memory: one lane per thread.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[16], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15 "
               "}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                 "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
               "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
               "}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                 "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                 "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                 "=r"(r[30]), "=r"(r[31])
               : "r"(addr));
}

// 32 columns of 16 lanes (the lanes of `addr` on), as the fragments of a matrix
// product lie: r[4 g + 2 h + e] is lane 8 h + t / 4, column 8 g + 2 (t % 4) + e,
// for the warp's thread t.
__device__ __forceinline__ void tmem_load_fragments(uint32_t (&r)[16], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15 "
               "}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                 "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}

// Waits for this thread's tensor-memory loads; names their registers so that
// no use of them moves above the wait.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// One fp32 value from global into shared memory without waiting for it (zero
// when !in; nothing is read then).
__device__ __forceinline__ void copy_async_f32(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}

// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace nts
