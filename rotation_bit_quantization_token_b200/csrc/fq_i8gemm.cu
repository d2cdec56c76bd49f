// INT8 x INT8 product with a scale for each token and each channel, sm_100a.
//
//     C[t, o] = (sum_i a[t, i] w[o, i]) * a_scale[t] * w_scale[o]
//
// for activations a [T, L] as the per-token quantizer writes them (FQ_OUT_INT8) and weights
// w [O, L] with one scale per output channel. The sum is exact: kind::i8 MMAs accumulate in
// int32 and |sum| <= 65536 * 128 * 128 = 2^30. It is rounded once to float32, multiplied by
// the two scales in float32 and rounded once to the output type.
//
// Layout of the work: the weights' rows lie on the TMEM lanes (M = 128 channels), tokens
// along the MMA's N (kBT = 16 .. 256), K in stages of 128 codes (one 128-byte swizzle atom).
// With few tokens the product is bound by reading the weights once, so the tile has no more
// token columns than needed, and the CTAs of a cluster split K between them and add their
// int32 partial sums through distributed shared memory (exact, whatever the order). With
// many tokens each CTA walks over tiles and the accumulator is double buffered, so that the
// epilogue of one tile runs under the MMAs of the next. A lane holds one channel, so a
// warp's stores of one token are 32 neighbouring outputs.
// Roles, 256 threads: warp 0 TMA producer, warp 1 MMA issuer (owns TMEM), warps 4-7 epilogue.
// Every wait is bounded; on expiry the kernel sets a bit in the caller's status word.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fq_internal.h"
#include "fq_ptx.cuh"

namespace fq {
namespace {

using namespace ptx;

constexpr int kBO = 128;       // weight rows per tile (TMEM lanes)
constexpr int kBK = 128;       // codes per row and stage
constexpr int kThreads = 256;
constexpr int kWarpProducer = 0, kWarpMma = 1, kWarpEpi0 = 4;

enum : uint32_t { kStFull = 1u << 0, kStEmpty = 1u << 1, kStDFull = 1u << 2, kStDEmpty = 1u << 3, kStDrain = 1u << 4 };

template <int kBT>
struct Geo {
  static constexpr int kWBytes = kBO * kBK;
  static constexpr int kABytes = kBT * kBK;
  static constexpr int kStage = kWBytes + kABytes;
  // two CTAs per SM for the narrow tiles (about 100 KB each in flight), one for the wide ones
  static constexpr int kStages = kBT <= 16 ? 5 : (kBT <= 64 ? 4 : (kBT == 128 ? 6 : 4));
  static constexpr int kMinBlocks = kBT <= 64 ? 2 : 1;
  static constexpr int kBufs = 2;
  static constexpr uint32_t kCols = kBufs * kBT < 32 ? 32u : uint32_t(kBufs * kBT);
  static constexpr int kSmem = kStages * kStage + 1024 /*alignment*/ + 512 /*barriers*/;
  static_assert(kSmem <= 227 * 1024 && kCols <= 512, "resources");
  static_assert(kBT * kBO * 4 <= kStages * kStage, "partial sums fit the ring");
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t d_full[2], d_empty[2];
  uint32_t tmem_base;
  int abort;
};

struct Params {
  const float* a_scale;
  const float* w_scale;
  void* C;
  uint32_t* status;
  int64_t T, O;
  int tiles_o, num_tiles, nk, split;
};

template <typename Out>
__device__ __forceinline__ Out to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_out<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_remote(uint32_t saddr, uint32_t rank) {
  uint32_t ra;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
  return v;
}

template <int kBT, typename Out>
__global__ void __launch_bounds__(kThreads, Geo<kBT>::kMinBlocks)
i8gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const Params p) {
  using G = Geo<kBT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + G::kStages * G::kStage);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) |  // int32 sums of signed bytes
                              (uint32_t(kBT >> 3) << 17) | (uint32_t(kBO >> 4) << 24);

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->d_full[b], 1);
      mbar_init(&bars->d_empty[b], 4);
    }
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bars->tmem_base, G::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // split = 1: tiles blockIdx.x, + gridDim.x, ...; split > 1: one tile per cluster, the
  // cluster's CTA r taking the K stages [r nk / split, (r + 1) nk / split)
  const int rank = p.split > 1 ? int(cluster_rank()) : 0;
  const int first = p.split > 1 ? int(blockIdx.x) / p.split : int(blockIdx.x);
  const int step = p.split > 1 ? p.num_tiles : int(gridDim.x);
  const int n_local = first < p.num_tiles ? (p.num_tiles - 1 - first) / step + 1 : 0;
  const int k0 = int(int64_t(p.nk) * rank / p.split), k1 = int(int64_t(p.nk) * (rank + 1) / p.split);

  if (warp == kWarpProducer) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_local; ++i) {
        const int tile = first + i * step;
        const int o0 = (tile % p.tiles_o) * kBO, t0 = (tile / p.tiles_o) * kBT;
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int s = it % G::kStages;
          if (it >= G::kStages &&
              !wait_bounded(&bars->empty[s], ((it / G::kStages) - 1) & 1, &bars->abort, p.status, kStEmpty)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->full[s], G::kStage);
          const uint32_t dst = sbase + s * G::kStage;
          tma_load_2d(dst, &map_w, kb * kBK, o0, &bars->full[s]);
          tma_load_2d(dst + G::kWBytes, &map_a, kb * kBK, t0, &bars->full[s]);
        }
      }
      // every issued load has landed before the CTA may exit (or reuse the ring)
      for (int j = it > G::kStages ? it - G::kStages : 0; j < it; ++j) {
        const uint32_t b = smem_u32(&bars->full[j % G::kStages]);
        const uint64_t tz = globaltimer();
        while (!mbar_try_wait(b, (j / G::kStages) & 1)) {
          if (globaltimer() - tz > kTimeoutNs) {
            if (p.status != nullptr) atomicOr(p.status, kStDrain);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    const bool leader = elect_one();
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && i < n_local; ++i) {
      const int buf = i & 1;
      if (i >= 2 && !warp_wait(&bars->d_empty[buf], ((i >> 1) - 1) & 1, &bars->abort, p.status, kStDEmpty)) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % G::kStages;
        if (!warp_wait(&bars->full[s], (it / G::kStages) & 1, &bars->abort, p.status, kStFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t wd = sw128_desc(sbase + s * G::kStage);
          const uint64_t ad = sw128_desc(sbase + s * G::kStage + G::kWBytes);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_i8(tmem + uint32_t(buf * kBT), wd + uint64_t((k * 32) >> 4), ad + uint64_t((k * 32) >> 4), kIdesc,
                   (kb > k0 || k > 0) ? 1u : 0u);
          mma_commit(&bars->empty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) mma_commit(&bars->d_full[buf]);
      __syncwarp();
    }
    // the MMAs of every stage that was issued complete before TMEM is released: wait for the
    // last commit of each stage
    if (lane == 0) {
      for (int j = it > G::kStages ? it - G::kStages : 0; j < it; ++j) {
        const uint32_t b = smem_u32(&bars->empty[j % G::kStages]);
        const uint64_t tz = globaltimer();
        while (!mbar_try_wait(b, (j / G::kStages) & 1)) {
          if (globaltimer() - tz > kTimeoutNs) {
            if (p.status != nullptr) atomicOr(p.status, kStDrain);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= kWarpEpi0) {
    const int q = warp - kWarpEpi0;
    const uint32_t t_lane = tmem + (uint32_t(q * 32) << 16);
    constexpr int kChunk = kBT < 32 ? kBT : 32;
    for (int i = 0; i < n_local; ++i) {
      const int tile = first + i * step;
      const int buf = i & 1;
      const int64_t o = int64_t(tile % p.tiles_o) * kBO + q * 32 + lane;
      const int64_t t0 = int64_t(tile / p.tiles_o) * kBT;
      const bool ok = warp_wait(&bars->d_full[buf], (i >> 1) & 1, &bars->abort, p.status, kStDFull);
      if (ok) {
        tc_fence_after();
        const float ws = o < p.O ? __ldg(p.w_scale + o) : 0.0f;
#pragma unroll 1
        for (int c = 0; c < kBT / kChunk; ++c) {
          uint32_t r[kChunk];
          if constexpr (kChunk == 16) tmem_ld16(t_lane + uint32_t(buf * kBT + c * kChunk), r);
          else tmem_ld32(t_lane + uint32_t(buf * kBT + c * kChunk), r);
          const int64_t ts = t0 + c * kChunk + lane;
          const float as = (lane < kChunk && ts < p.T) ? __ldg(p.a_scale + ts) : 0.0f;
          tmem_wait_ld();
          if (p.split > 1) {
            // this CTA's partial sums, [token][channel], into its own (drained) ring: every
            // load of it has been read by an MMA that completed before d_full
            int* part = reinterpret_cast<int*>(smem) + (c * kChunk) * kBO + q * 32 + lane;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) part[e * kBO] = int(r[e]);
          } else {
            Out* dst = static_cast<Out*>(p.C) + (t0 + c * kChunk) * p.O + o;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
              const float f = float(int(r[e])) * __shfl_sync(0xffffffffu, as, e) * ws;
              if (t0 + c * kChunk + e < p.T && o < p.O) dst[int64_t(e) * p.O] = to_out<Out>(f);
            }
          }
        }
      }
      // the accumulator is free for the tile after next
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->d_empty[buf]);
      if (!ok) break;
    }
  }

  if (p.split > 1) {
    // each CTA adds up its share of the tokens from all CTAs of the cluster
    cluster_sync();
    const bool good = *reinterpret_cast<volatile int*>(&bars->abort) == 0;
    const int per = (kBT + p.split - 1) / p.split;
    const int64_t o = int64_t(first % p.tiles_o) * kBO + (threadIdx.x & (kBO - 1));
    const int64_t t0 = int64_t(first / p.tiles_o) * kBT;
    const float ws = o < p.O ? __ldg(p.w_scale + o) : 0.0f;
    for (int e = rank * per + int(threadIdx.x) / kBO; good && e < min(kBT, (rank + 1) * per); e += kThreads / kBO) {
      if (t0 + e >= p.T) break;
      const uint32_t at = sbase + uint32_t(e * kBO + (threadIdx.x & (kBO - 1))) * 4u;
      int sum = 0;
      for (int r = 0; r < p.split; ++r) sum += ld_remote(at, uint32_t(r));
      const float f = float(sum) * __ldg(p.a_scale + t0 + e) * ws;
      if (o < p.O) static_cast<Out*>(p.C)[(t0 + e) * p.O + o] = to_out<Out>(f);
    }
    cluster_sync();  // no CTA leaves while another reads its partial sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

template <int kBT, typename Out>
cudaError_t launch_t(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  using G = Geo<kBT>;
  CUtensorMap map_w, map_a;
  if (!encode_bytes_2d(&map_w, g.w, uint64_t(g.O), uint64_t(g.L), kBK, kBO) ||
      !encode_bytes_2d(&map_a, g.a, uint64_t(g.T), uint64_t(g.L), kBK, kBT))
    return cudaErrorInvalidValue;
  Params p{};
  p.a_scale = g.a_scale;
  p.w_scale = g.w_scale;
  p.C = g.C;
  p.status = g.status;
  p.T = g.T;
  p.O = g.O;
  p.tiles_o = int((g.O + kBO - 1) / kBO);
  p.num_tiles = p.tiles_o * int((g.T + kBT - 1) / kBT);
  p.nk = int((g.L + kBK - 1) / kBK);
  // split K until every SM has its CTAs, as long as each CTA keeps four stages of work
  int split = 1;
  while (split < 8 && p.num_tiles * split * 2 <= num_sms * G::kMinBlocks && p.nk >= split * 2 * 4) split *= 2;
  p.split = split;
  auto kern = i8gemm_kernel<kBT, Out>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kern), G::kSmem);
  if (e != cudaSuccess) return e;
  const int resident = num_sms * G::kMinBlocks;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(split > 1 ? p.num_tiles * split : (p.num_tiles < resident ? p.num_tiles : resident)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_a, p);
}

template <typename Out>
cudaError_t launch_out(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  if (g.T <= 16) return launch_t<16, Out>(g, num_sms, stream);
  if (g.T <= 32) return launch_t<32, Out>(g, num_sms, stream);
  if (g.T <= 64) return launch_t<64, Out>(g, num_sms, stream);
  if (g.T <= 128) return launch_t<128, Out>(g, num_sms, stream);
  return launch_t<256, Out>(g, num_sms, stream);
}

}  // namespace

cudaError_t launch_i8gemm(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  switch (g.out_type) {
    case FQ_BF16: return launch_out<__nv_bfloat16>(g, num_sms, stream);
    case FQ_FP16: return launch_out<__half>(g, num_sms, stream);
    default: return launch_out<float>(g, num_sms, stream);
  }
}

}  // namespace fq
