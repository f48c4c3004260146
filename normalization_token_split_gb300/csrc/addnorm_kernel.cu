// addnorm_kernel.cu -- the addition of a layer's output to the residual stream with
// RMSNorm and the cast to E4M3 codes with a scale per 128 values in the same pass
// (nts_rmsnorm_blockcast with an addition in front), and its gradient, on one GB300.
//
// Forward, per row of D values:
//     h_j  = round(x_j + r_j) to the stream's type (bf16 or fp32),
//     rinv = 1 / sqrt((1/D) sum h^2 + eps),  w_j = (h_j gamma_j) rinv,
// and the scales and codes of w as nts_rmsnorm_blockcast forms them.  The statistic
// is that of the h that is stored, so the gradient needs nothing but h and rinv.
// Backward, with dy the gradient of w, u_j = dy_j gamma_j and e the gradient of h from
// the layers behind:
//     dh_j = rinv u_j - h_j rinv^3 (1/D) sum u h + e_j   (of x and of r alike),
//     dgamma_j = sum over rows of dy_j h_j rinv.
//
// GB300 mapping: both are bound by HBM (7 to 11 and 8 to 16 bytes per value, 7 and 11
// flops).  A thread owns 16 neighbouring values of a row, the same ones of every row it
// meets, so its gains and its sums for dgamma stay in registers; eight lanes hold a
// block of 128.  A warp copies its part of the next rows into its own stages of shared
// memory (cp.async: no thread waits for another warp's copies), and a row's warps
// meet once, for the sum.  Rows of more than kSliceUnits units are split over the CTAs
// of a cluster, whose warps write their sums into every CTA's shared memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_device.cuh"
#include "block_internal.h"

namespace nts {

namespace {

constexpr int kMaxRowThreads = 512;   // a CTA's part of a row, in units of 16 values
constexpr int kSliceUnits = 512;      // rows up to this take one CTA
constexpr int kGroupThreads = 256;    // narrower rows share a CTA of about this size
constexpr int kForwardStages = 3, kBackwardStages = 2;
constexpr int kMaxWarps = kMaxRowThreads / 32;

// Shared memory of a staged unit: a 16-byte gap keeps the eight lanes of a read phase
// in distinct banks.
constexpr int kUnit16 = 32 + 16, kUnit32 = 64 + 16;

struct AddNormParams {
  const __nv_bfloat16* a;     // x, or dy
  const void* r;              // the residual, or h
  const void* e;              // backward: gradient from behind, or nullptr
  const float* gamma;         // or nullptr: ones
  void* h;                    // forward: the sum; backward: dh
  __nv_bfloat16* dx;          // backward, fp32 stream: dh in bf16, or nullptr
  uint8_t* codes;
  float* scales;
  float* rinv;                // forward: written, or nullptr
  const float* rinv_in;       // backward
  float* partial;             // backward: [CTAs per slice][D] sums for dgamma, or nullptr
  int64_t T;
  int D, blocks;
  int slice;                  // units of a row per CTA, a multiple of 8
  int tpr;                    // threads per row (slice), whole warps
  int wide;                   // rows of h start on 32-byte boundaries
  float eps, inv_d;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copies the warp's 32 units of a row, PIECES 16-byte pieces each, neighbouring lanes
// taking neighbouring pieces; units from `units` on become zeros.
template <int PIECES>
__device__ __forceinline__ void stage_units(uint32_t dst, const unsigned char* src, int units) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int q = 32 * i + lane, u = q / PIECES;
    const bool in = u < units;
    cp_async16(dst + u * (16 * PIECES + 16) + (q % PIECES) * 16, in ? src + 16 * q : src, in);
  }
}

__device__ __forceinline__ void read_bf16(const unsigned char* at, uint64_t (&v)[8]) {
  const uint4 a = lds128(at), b = lds128(at + 16);
  v[0] = bf16x2_to_f2(a.x), v[1] = bf16x2_to_f2(a.y);
  v[2] = bf16x2_to_f2(a.z), v[3] = bf16x2_to_f2(a.w);
  v[4] = bf16x2_to_f2(b.x), v[5] = bf16x2_to_f2(b.y);
  v[6] = bf16x2_to_f2(b.z), v[7] = bf16x2_to_f2(b.w);
}

template <bool F32>
__device__ __forceinline__ void read_stream(const unsigned char* at, uint64_t (&v)[8]) {
  if (!F32) {
    read_bf16(at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 a = lds128(at + 16 * i);
    v[2 * i] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[2 * i + 1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
  }
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], int wide) {
  if (wide) {
    st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  } else {
    st_global_v4(p, w[0], w[1], w[2], w[3]);
    st_global_v4(static_cast<unsigned char*>(p) + 16, w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ void pack16(const uint64_t (&v)[8], uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2_rn(f2_lo(v[i]), f2_hi(v[i]));
}

template <bool F32>
__device__ __forceinline__ void store_stream(void* row, int64_t unit, const uint64_t (&v)[8],
                                             int wide) {
  if (!F32) {
    uint32_t w[8];
    pack16(v, w);
    store32(static_cast<__nv_bfloat16*>(row) + 16 * unit, w, wide);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = (uint32_t)v[4 * i + j];
      w[2 * j + 1] = (uint32_t)(v[4 * i + j] >> 32);
    }
    store32(static_cast<float*>(row) + 16 * unit + 8 * i, w, wide);
  }
}

// A thread's place in the grid: the rows its group takes, and its unit of each.
template <int C>
struct Place {
  int lane, warp;       // warp of the row's group in this CTA
  int group;            // group of the CTA (C == 1)
  int rank;             // CTA of the cluster
  int warps;            // warps per row in this CTA
  int unit;             // of the row
  int left;             // units of the warp: its first unit to the row's or slice's end
  bool in;
  int64_t first, step;  // rows
  __device__ __forceinline__ explicit Place(const AddNormParams& p) {
    lane = threadIdx.x & 31;
    group = C == 1 ? (int)threadIdx.x / p.tpr : 0;
    const int t = threadIdx.x - group * p.tpr;
    warp = t >> 5;
    warps = p.tpr >> 5;
    rank = C == 1 ? 0 : (int)cluster_ctarank();
    const int groups = C == 1 ? (int)blockDim.x / p.tpr : 1;
    const int64_t id = C == 1 ? blockIdx.x : blockIdx.x / C;
    first = id * groups + group;
    step = (int64_t)(gridDim.x / C) * groups;
    const int begin = rank * p.slice, end = min(begin + p.slice, p.D / 16);
    unit = begin + t;
    left = end - (begin + 32 * warp);
    in = unit < end;
  }
};

// The sum of v over a row: its warps (of every CTA of the cluster) write theirs into
// part[buf] and meet once.  The other buffer's readers are past that meeting.
template <int C>
__device__ __forceinline__ float row_sum(float v, const Place<C>& at, const AddNormParams& p,
                                         float* part, int buf) {
  v = warp_sum(v);
  if (C == 1) {
    if (at.warps == 1) return v;
    float* mine = part + buf * kMaxWarps + at.group * at.warps;
    if (at.lane == 0) mine[at.warp] = v;
    named_barrier(1 + at.group, p.tpr);
    v = 0.f;
    for (int w = 0; w < at.warps; ++w) v += mine[w];
    return v;
  }
  float* all = part + buf * C * kMaxWarps;
  if (at.lane < C)
    st_cluster_f32(map_to_rank(smem_addr(all + at.rank * at.warps + at.warp), at.lane), v);
  cluster_arrive_release();
  cluster_wait_acquire();
  v = 0.f;
  for (int w = 0; w < C * at.warps; ++w) v += all[w];
  return v;
}

template <int C>
__device__ __forceinline__ void start_cluster() {
  if (C > 1) {   // every CTA runs before another writes into its shared memory
    cluster_arrive_relaxed();
    cluster_wait_acquire();
  }
}

template <int C, bool F32>
__global__ void __launch_bounds__(kMaxRowThreads) add_rmsnorm_kernel(const AddNormParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[2 * C * kMaxWarps];
  constexpr int kUnitR = F32 ? kUnit32 : kUnit16, kSize = F32 ? 4 : 2;
  constexpr int kStage = 32 * (kUnit16 + kUnitR);   // of a warp
  const Place<C> at(p);
  unsigned char* ring = smem + (threadIdx.x >> 5) * kForwardStages * kStage;
  const unsigned char* a = reinterpret_cast<const unsigned char*>(p.a) + 32 * (int64_t)(at.unit - at.lane);
  const unsigned char* r =
      static_cast<const unsigned char*>(p.r) + 16 * kSize * (int64_t)(at.unit - at.lane);
  start_cluster<C>();
  grid_dependency_wait();
  allow_dependent_launch();

  auto stage = [&](int64_t row, int s) {
    if (row < p.T && at.left > 0) {
      const uint32_t dst = smem_addr(ring) + s * kStage;
      stage_units<2>(dst, a + row * p.D * 2, at.left);
      stage_units<kSize>(dst + 32 * kUnit16, r + row * p.D * kSize, at.left);
    }
    cp_async_commit();   // empty groups keep the count
  };
#pragma unroll
  for (int s = 0; s < kForwardStages; ++s) stage(at.first + s * at.step, s);

  float gain[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.gamma != nullptr && at.in)
      v = __ldg(reinterpret_cast<const float4*>(p.gamma + 16 * at.unit) + j);
    gain[4 * j] = v.x, gain[4 * j + 1] = v.y, gain[4 * j + 2] = v.z, gain[4 * j + 3] = v.w;
  }

  int s = 0, buf = 0;
  for (int64_t row = at.first; row < p.T; row += at.step) {
    cp_async_wait<kForwardStages - 1>();
    __syncwarp();   // the warp's copies are seen by all its lanes
    const unsigned char* st = ring + s * kStage;
    uint64_t h[8];
    {
      uint64_t x[8];
      read_bf16(st + at.lane * kUnit16, x);
      read_stream<F32>(st + 32 * kUnit16 + at.lane * kUnitR, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = f2_add(x[i], h[i]);
      if (!F32) {   // the stored sum
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = bf16x2_to_f2(pack_bf16x2_rn(f2_lo(h[i]), f2_hi(h[i])));
      }
      if (!at.in)   // what an idle lane's stage holds is not part of the row
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = 0;
    }
    __syncwarp();   // read by all before the next copy into the stage
    stage(row + kForwardStages * at.step, s);
    if (++s == kForwardStages) s = 0;
    if (at.in)
      store_stream<F32>(static_cast<unsigned char*>(p.h) + row * p.D * kSize, at.unit, h, p.wide);
    uint64_t q0 = 0, q1 = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      q0 = f2_fma(h[i], h[i], q0);
      q1 = f2_fma(h[i + 1], h[i + 1], q1);
    }
    q0 = f2_add(q0, q1);
    const float ss = row_sum<C>(f2_lo(q0) + f2_hi(q0), at, p, part, buf);
    buf ^= 1;
    const float rinv = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
    if (p.rinv != nullptr && at.unit == 0) p.rinv[row] = rinv;
    float w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[2 * i] = f2_lo(h[i]) * gain[2 * i] * rinv;
      w[2 * i + 1] = f2_hi(h[i]) * gain[2 * i + 1] * rinv;
    }
    float m = absmax16(w);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float scale = block_scale(m);
    const uint4 c = codes16(w, __frcp_rn(scale));
    if (at.in) {
      __stcs(reinterpret_cast<uint4*>(p.codes + row * p.D + 16 * at.unit), c);
      if ((at.lane & 7) == 0) p.scales[row * p.blocks + (at.unit >> 3)] = scale;
    }
  }
}

template <int C, bool F32>
__global__ void __launch_bounds__(kMaxRowThreads) add_rmsnorm_backward_kernel(const AddNormParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[2 * C * kMaxWarps];
  constexpr int kUnitR = F32 ? kUnit32 : kUnit16, kSize = F32 ? 4 : 2;
  constexpr int kStage = 32 * (kUnit16 + 2 * kUnitR);
  const Place<C> at(p);
  unsigned char* ring = smem + (threadIdx.x >> 5) * kBackwardStages * kStage;
  const int64_t u0 = at.unit - at.lane;
  const unsigned char* a = reinterpret_cast<const unsigned char*>(p.a) + 32 * u0;
  const unsigned char* r = static_cast<const unsigned char*>(p.r) + 16 * kSize * u0;
  const unsigned char* e = static_cast<const unsigned char*>(p.e) + 16 * kSize * u0;
  start_cluster<C>();
  grid_dependency_wait();
  allow_dependent_launch();

  auto stage = [&](int64_t row, int s) {
    if (row < p.T && at.left > 0) {
      const uint32_t dst = smem_addr(ring) + s * kStage;
      stage_units<2>(dst, a + row * p.D * 2, at.left);
      stage_units<kSize>(dst + 32 * kUnit16, r + row * p.D * kSize, at.left);
      if (p.e != nullptr)
        stage_units<kSize>(dst + 32 * (kUnit16 + kUnitR), e + row * p.D * kSize, at.left);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kBackwardStages; ++s) stage(at.first + s * at.step, s);

  uint64_t gain[8], sum[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.gamma != nullptr && at.in)
      v = __ldg(reinterpret_cast<const float4*>(p.gamma + 16 * at.unit) + j);
    gain[2 * j] = f2(v.x, v.y);
    gain[2 * j + 1] = f2(v.z, v.w);
    sum[2 * j] = sum[2 * j + 1] = 0;
  }
  float next = at.first < p.T ? __ldg(p.rinv_in + at.first) : 0.f;

  int s = 0, buf = 0;
  for (int64_t row = at.first; row < p.T; row += at.step) {
    const float rinv = next;
    if (row + at.step < p.T) next = __ldg(p.rinv_in + row + at.step);
    cp_async_wait<kBackwardStages - 1>();
    __syncwarp();
    const unsigned char* st = ring + s * kStage;
    uint64_t g[8], h[8];
    read_bf16(st + at.lane * kUnit16, g);
    read_stream<F32>(st + 32 * kUnit16 + at.lane * kUnitR, h);
    const uint64_t rr = f2(rinv, rinv);
    uint64_t q0 = 0, q1 = 0;
    if (at.in) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        sum[i] = f2_fma(g[i], f2_mul(h[i], rr), sum[i]);
        sum[i + 1] = f2_fma(g[i + 1], f2_mul(h[i + 1], rr), sum[i + 1]);
        q0 = f2_fma(f2_mul(g[i], gain[i]), h[i], q0);
        q1 = f2_fma(f2_mul(g[i + 1], gain[i + 1]), h[i + 1], q1);
      }
      q0 = f2_add(q0, q1);
    }
    const float uh = row_sum<C>(f2_lo(q0) + f2_hi(q0), at, p, part, buf);
    buf ^= 1;
    const float k = -(uh * p.inv_d * rinv) * (rinv * rinv);
    const uint64_t kk = f2(k, k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      h[i] = f2_fma(h[i], kk, f2_mul(f2_mul(g[i], gain[i]), rr));
    if (p.e != nullptr) {
      read_stream<F32>(st + 32 * (kUnit16 + kUnitR) + at.lane * kUnitR, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = f2_add(h[i], g[i]);
    }
    __syncwarp();
    stage(row + kBackwardStages * at.step, s);
    if (++s == kBackwardStages) s = 0;
    if (at.in) {
      store_stream<F32>(static_cast<unsigned char*>(p.h) + row * p.D * kSize, at.unit, h, p.wide);
      if (F32 && p.dx != nullptr) {
        uint32_t w[8];
        pack16(h, w);
        store32(p.dx + row * p.D + 16 * at.unit, w, p.wide);
      }
    }
  }
  if (p.partial == nullptr) return;

  // The CTA's row of sums: over its groups, in their order.
  if (C == 1 && blockDim.x > p.tpr) {
    cp_async_wait<0>();
    __syncthreads();   // every warp is done with its stages
    float* red = reinterpret_cast<float*>(smem);   // [groups][16 slice]
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.in)
        *reinterpret_cast<float2*>(red + (at.group * p.slice + at.unit) * 16 + 2 * i) =
            make_float2(f2_lo(sum[i]), f2_hi(sum[i]));
    __syncthreads();
    const int groups = blockDim.x / p.tpr;
    for (int j = threadIdx.x; j < p.D; j += blockDim.x) {
      float v = red[j];
      for (int g = 1; g < groups; ++g) v += red[g * p.slice * 16 + j];
      p.partial[(int64_t)blockIdx.x * p.D + j] = v;
    }
    return;
  }
  if (at.in)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t id = C == 1 ? blockIdx.x : blockIdx.x / C;
      *reinterpret_cast<float4*>(p.partial + id * p.D + 16 * at.unit + 4 * i) =
          make_float4(f2_lo(sum[2 * i]), f2_hi(sum[2 * i]), f2_lo(sum[2 * i + 1]),
                      f2_hi(sum[2 * i + 1]));
    }
}

// dgamma: the sum of the CTAs' rows, in a fixed order; block (32 columns) x (32
// threads, each with every 32nd row).
__global__ void __launch_bounds__(1024) gain_grad_kernel(const float* partial, int n, int D,
                                                         float* dgamma) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  grid_dependency_wait();
  allow_dependent_launch();
  float v = 0.f;
  if (col < D)
#pragma unroll 8
    for (int r = threadIdx.y; r < n; r += 32) v += __ldcg(partial + (int64_t)r * D + col);
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < D) dgamma[out] = v;
}

using AddNormKernel = void (*)(AddNormParams);

template <int C>
AddNormKernel pick(bool f32, bool backward) {
  if (backward) return f32 ? add_rmsnorm_backward_kernel<C, true> : add_rmsnorm_backward_kernel<C, false>;
  return f32 ? add_rmsnorm_kernel<C, true> : add_rmsnorm_kernel<C, false>;
}

template <typename... A>
int launch(void (*kern)(A...), cudaLaunchConfig_t cfg, int cluster, cudaStream_t stream, bool pdl,
           A... args) {
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
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
  if (err != cudaSuccess) return fail_cuda(err, "launching the residual addition with RMSNorm");
  return NTS_OK;
}

}  // namespace

int launch_addnorm(const AddNormRequest& rq, cudaStream_t stream, const LaunchTuning& tune) {
  if (const int injected = take_injected_failure()) return injected;
  const DeviceInfo& dev = device_info();
  if (!dev.ok) return fail(NTS_ERR_CUDA, "could not query the current device");
  const bool backward = rq.dgamma != nullptr || rq.rinv_in != nullptr;
  const bool f32 = rq.fp32 != 0;
  AddNormParams p = {};
  p.a = static_cast<const __nv_bfloat16*>(rq.a);
  p.r = rq.r;
  p.e = rq.e;
  p.gamma = rq.gamma;
  p.h = rq.h;
  p.dx = static_cast<__nv_bfloat16*>(rq.dx);
  p.codes = rq.codes;
  p.scales = rq.scales;
  p.rinv = rq.rinv;
  p.rinv_in = rq.rinv_in;
  p.T = rq.T;
  p.D = (int)rq.D;
  p.blocks = (int)((rq.D + 127) / 128);
  p.eps = rq.eps;
  p.inv_d = 1.0f / (float)p.D;
  p.wide = reinterpret_cast<uintptr_t>(rq.h) % 32 == 0 && reinterpret_cast<uintptr_t>(rq.dx) % 32 == 0;
  const int units = p.D / 16;
  int C = 1;
  while (units > C * kSliceUnits) C *= 2;
  p.slice = ((units + C - 1) / C + 7) / 8 * 8;
  p.tpr = (p.slice + 31) / 32 * 32;
  const int groups = C == 1 ? std::max(1, kGroupThreads / p.tpr) : 1;
  const AddNormKernel kern = C == 1   ? pick<1>(f32, backward)
                             : C == 2 ? pick<2>(f32, backward)
                                      : pick<4>(f32, backward);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)(groups * p.tpr));
  const int unit = kUnit16 + (backward ? 2 : 1) * (f32 ? kUnit32 : kUnit16);
  cfg.dynamicSmemBytes = (size_t)cfg.blockDim.x * unit * (backward ? kBackwardStages : kForwardStages);
  int rc = prepare_kernel((const void*)kern, cfg.dynamicSmemBytes);
  if (rc != NTS_OK) return rc;
  int64_t most = 0;
  if (C == 1) {
    int per_sm = 0;
    rc = blocks_per_sm((const void*)kern, cfg.blockDim.x, cfg.dynamicSmemBytes, &per_sm);
    most = (int64_t)per_sm * dev.sm_count;
  } else {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    rc = max_active_clusters((const void*)kern, cfg, C, &most);
  }
  if (rc != NTS_OK) return rc;
  if (backward) most = std::min<int64_t>(most, kNormPartials);
  const int64_t rows = std::min<int64_t>((p.T + groups - 1) / groups, most);   // CTAs or clusters
  cfg.gridDim = dim3((unsigned)(rows * C));
  if (rq.dgamma != nullptr) p.partial = rq.partial;
  log_launch(backward ? "add_rmsnorm_backward" : "add_rmsnorm_blockcast",
             "T=%lld D=%d fp32=%d cluster=%d threads=%u rows at once=%d smem=%zu grid=%u",
             (long long)p.T, p.D, (int)f32, C, cfg.blockDim.x, groups, cfg.dynamicSmemBytes,
             cfg.gridDim.x);
  rc = launch(kern, cfg, C, stream, tune.pdl != 0, p);
  if (rc != NTS_OK || rq.dgamma == nullptr) return rc;
  cudaLaunchConfig_t sum = {};
  sum.gridDim = dim3((unsigned)((p.D + 31) / 32));
  sum.blockDim = dim3(32, 32);
  return launch(gain_grad_kernel, sum, 1, stream, tune.pdl != 0, (const float*)p.partial, (int)rows,
                p.D, rq.dgamma);
}

}  // namespace nts
