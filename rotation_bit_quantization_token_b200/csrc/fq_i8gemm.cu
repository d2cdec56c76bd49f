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
// token columns than needed, and the CTAs of a cluster split K between them and send their int32
// partial sums to the one that owns the token (exact, whatever the order). With
// many tokens each CTA walks over tiles and the accumulator is double buffered, so that the
// epilogue of one tile runs under the MMAs of the next. A lane holds one channel, so a
// warp's stores of one token are 32 neighbouring outputs.
// Roles, 256 threads: warp 0 TMA producer, warp 1 MMA issuer (owns TMEM), warps 4-7 epilogue.
// Large products take i8gemm_pair_kernel: pairs of CTAs share 256 x 256 tiles (cta_group::2), each
// loading 128 rows of both operands, 32 KB a stage instead of 48 for the same products. The single
// kernel runs at 757 clocks a stage there (63 bytes a clock and SM, what L2 delivers), where the
// MMAs need 512.
// 8192 x 4096 x 14336: 303 us, 3.2 POP/s in bursts (363 us repeated, at 1000 W); 1 x 14336 x 4096:
// 14.5 us, 4.1 TB/s. Every wait is bounded; on expiry the kernel sets a bit in the caller's status word, or
// in the library's own where the caller gives none.
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

enum : uint32_t { kStFull = 1u << 0, kStEmpty = 1u << 1, kStDFull = 1u << 2, kStDEmpty = 1u << 3, kStDrain = 1u << 4, kStIn = 1u << 5 };

// kSplit: the CTAs of a cluster share one tile's K
template <int kBT, bool kSplit>
struct Geo {
  static constexpr int kWBytes = kBO * kBK;
  static constexpr int kABytes = kBT * kBK;
  static constexpr int kStage = kWBytes + kABytes;
  // two CTAs per SM for the narrow tiles (about 100 KB each in flight), one for the wide ones
  static constexpr int kMinBlocks = kBT <= 64 ? 2 : 1;
  static constexpr int kStages = kBT <= 16 ? 5 : (kBT <= 32 ? 4 : (kBT == 64 ? (kSplit ? 3 : 4) : (kBT <= 192 ? (kSplit ? 4 : 5) : (kSplit ? 3 : 4))));
  static constexpr int kMaxSplit = kBT >= 192 ? 2 : (kBT == 64 ? 4 : 8);  // as the partial sums fit
  static constexpr int kBufs = kSplit ? 1 : 2;  // accumulators
  static constexpr uint32_t kCols = kBufs * kBT < 32 ? 32u : uint32_t(kBufs * (kBT == 192 ? 256 : kBT));  // a power of two
  // partial sums from the other CTAs of the cluster, [sender][channel][token of this CTA's share]; a
  // channel's row is 16 bytes longer than its tokens, so that neighbouring lanes read other banks
  static constexpr int in_bytes(int split) { return (split - 1) * kBO * (kBT / split + 4) * 4; }
  static constexpr int kInBytes = kSplit ? in_bytes(kMaxSplit) : 0;  // grows with the split
  // 32 outputs of up to 32 tokens for each epilogue warp (wide tiles only)
  static constexpr int kStaging = kBT >= 128 && !kSplit ? 4 * 32 * 32 * 4 : 0;
  static constexpr int kOffIn = kStages * kStage;
  static constexpr int kOffBars = kOffIn + kInBytes + kStaging;
  static constexpr int kSmem = kOffBars + 1024 /*alignment*/ + 512 /*barriers*/;
  static_assert(kSmem * kMinBlocks <= (227 - (kMinBlocks - 1)) * 1024 && kCols <= 512, "resources");
};

// The status word of calls without one, on each device (fq_int8_device_status).
__device__ uint32_t own_status;
__device__ __forceinline__ uint32_t* status_word(uint32_t* given) { return given != nullptr ? given : &own_status; }

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t d_full[2], d_empty[2];
  uint64_t in_full;  // the other CTAs' partial sums are there
  uint32_t tmem_base;
  int abort;
  int issued;                    // pairs: stages that this CTA's producer has loaded
  int other_abort, other_issued;  // pairs: the other CTA's at its end
};

struct Params {
  const float* a_scale;
  const float* w_scale;
  void* C;
  uint32_t* status;
  int64_t T, O;
  int tiles_o, num_tiles, nk, split;
  int vec;  // rows of C are 16-byte aligned
  int stall;          // test hook: see fq_int8_debug_arm_stall
  uint64_t limit_ns;  // of every bounded wait
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

// Four (two) words to another CTA's shared memory, counted by its barrier.
__device__ __forceinline__ void push4(uint32_t dst, const uint32_t* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(dst),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void push2(uint32_t dst, const uint32_t* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1,%2}, [%3];" ::"r"(dst), "r"(v[0]),
               "r"(v[1]), "r"(bar)
               : "memory");
}

// Scales and stores kChunk tokens (columns col .. of TMEM row t_col) of a warp's 32 channels. With
// `stage` (this warp's shared memory, kChunk * 32 outputs) the tokens' 32 outputs leave as 16-byte
// pieces; without it, or where the rows of C are not 16-byte aligned, one output per lane and store.
template <int kChunk, typename Out>
__device__ __forceinline__ void store_chunk(uint32_t t_col, const Params& p, int64_t t0, int64_t o0, float ws, int lane,
                                            uint8_t* stage, bool vec) {
  uint32_t r[kChunk];
  if constexpr (kChunk == 16) tmem_ld16(t_col, r);
  else tmem_ld32(t_col, r);
  const float as = (lane < kChunk && t0 + lane < p.T) ? __ldg(p.a_scale + t0 + lane) : 0.0f;
  tmem_wait_ld();
  const int n = int(min(p.T - t0, int64_t(kChunk)));  // tokens there (may be negative)
  Out y[kChunk];
#pragma unroll
  for (int e = 0; e < kChunk; ++e) y[e] = to_out<Out>(float(int(r[e])) * __shfl_sync(0xffffffffu, as, e) * ws);
  if (vec && stage != nullptr && o0 + 32 <= p.O) {
    Out* mine = reinterpret_cast<Out*>(stage);
    __syncwarp();  // the last chunk has been read
#pragma unroll
    for (int e = 0; e < kChunk; ++e) mine[e * 32 + lane] = y[e];
    __syncwarp();
    constexpr int kPieces = 32 * int(sizeof(Out)) / 16, kPer = 32 / kPieces;  // pieces of a token, tokens per store
    const int piece = lane % kPieces;
#pragma unroll
    for (int e = 0; e < kChunk; e += kPer) {
      const int t = e + lane / kPieces;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + t * 32 * int(sizeof(Out)) + piece * 16);
      if (t < n) *(reinterpret_cast<uint4*>(static_cast<Out*>(p.C) + (t0 + t) * p.O + o0) + piece) = v;
    }
  } else if (o0 + lane < p.O) {
    Out* dst = static_cast<Out*>(p.C) + t0 * p.O + o0 + lane;
#pragma unroll
    for (int e = 0; e < kChunk; ++e, dst += p.O)
      if (e < n) *dst = y[e];
  }
}

template <int kBT, typename Out, bool kSplit>
__global__ void __launch_bounds__(kThreads, Geo<kBT, kSplit>::kMinBlocks)
i8gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const Params p) {
  using G = Geo<kBT, kSplit>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t* const status = status_word(p.status);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + G::kOffBars);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) |  // int32 sums of signed bytes
                              (uint32_t(kBT >> 3) << 17) | (uint32_t(kBO >> 4) << 24);

  // not split: tiles blockIdx.x, + gridDim.x, ...; split: one tile per cluster, the cluster's CTA r
  // taking the K stages [r nk / split, (r + 1) nk / split)
  const int rank = kSplit ? int(cluster_rank()) : 0;
  const int first = kSplit ? int(blockIdx.x) / p.split : int(blockIdx.x);
  const int step = kSplit ? p.num_tiles : int(gridDim.x);
  const int n_local = first < p.num_tiles ? (p.num_tiles - 1 - first) / step + 1 : 0;
  const int k0 = kSplit ? p.nk * rank / p.split : 0, k1 = kSplit ? p.nk * (rank + 1) / p.split : p.nk;
  const int per = kSplit ? kBT / p.split : kBT;  // tokens of this CTA's share of the outputs
  auto load = [&](int tile, int kb, int s) {
    mbar_arrive_expect_tx(&bars->full[s], G::kStage);
    const uint32_t dst = sbase + s * G::kStage;
    tma_load_2d(dst, &map_w, kb * kBK, (tile % p.tiles_o) * kBO, &bars->full[s]);
    tma_load_2d(dst + G::kWBytes, &map_a, kb * kBK, (tile / p.tiles_o) * kBT, &bars->full[s]);
  };
  // the first round of loads goes out before the CTA has met: nothing else writes the ring
  const bool stall = p.stall != 0 && rank == 0;  // (test hook) this CTA issues no loads
  const int n_early = n_local > 0 && !stall ? min(k1 - k0, G::kStages) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->d_full[b], 1);
      mbar_init(&bars->d_empty[b], 4);
    }
    mbar_init(&bars->in_full, 1);
    bars->abort = 0;
    fence_barrier_init();
    fence_proxy_async();
    if constexpr (kSplit) mbar_arrive_expect_tx(&bars->in_full, uint32_t((p.split - 1) * per * kBO * 4));
    for (int s = 0; s < n_early; ++s) load(first, k0 + s, s);
  }
  if (warp == kWarpMma) tmem_alloc(&bars->tmem_base, G::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // the cluster meets before a partial sum is sent (its CTAs run and their barriers are there); the
  // arrival is here, the wait just before sending, long after the others have arrived
  if constexpr (kSplit) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  if constexpr (kSplit) {
    // every warp of every CTA waits (the producer and issuer after their loops), so none may be left out
    if (warp == 2 || warp == 3) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (warp == kWarpProducer) {
    if (lane == 0) {
      int it = n_early;
      bool ok = true;
      for (int i = 0; ok && !stall && i < n_local; ++i) {
        for (int kb = k0 + (i == 0 ? n_early : 0); kb < k1; ++kb, ++it) {
          const int s = it % G::kStages;
          if (it >= G::kStages &&
              !wait_bounded(&bars->empty[s], ((it / G::kStages) - 1) & 1, &bars->abort, status, kStEmpty, p.limit_ns)) {
            ok = false;
            break;
          }
          load(first + i * step, kb, s);
        }
      }
      // every issued load has landed before the CTA may exit (or reuse the ring)
      for (int j = it > G::kStages ? it - G::kStages : 0; j < it; ++j) {
        const uint32_t b = smem_u32(&bars->full[j % G::kStages]);
        const uint64_t tz = globaltimer();
        while (!mbar_try_wait(b, (j / G::kStages) & 1)) {
          if (globaltimer() - tz > p.limit_ns) {
            atomicOr(status, kStDrain);
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
      if (i >= 2 && !warp_wait(&bars->d_empty[buf], ((i >> 1) - 1) & 1, &bars->abort, status, kStDEmpty, p.limit_ns)) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % G::kStages;
        if (!warp_wait(&bars->full[s], (it / G::kStages) & 1, &bars->abort, status, kStFull, p.limit_ns)) {
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
          if (globaltimer() - tz > p.limit_ns) {
            atomicOr(status, kStDrain);
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
      const bool ok = warp_wait(&bars->d_full[buf], (i >> 1) & 1, &bars->abort, status, kStDFull, p.limit_ns);
      if (ok) {
        tc_fence_after();
        const float ws = o < p.O ? __ldg(p.w_scale + o) : 0.0f;
        const int64_t o0 = int64_t(tile % p.tiles_o) * kBO + q * 32;
        uint8_t* stage = G::kStaging > 0 ? smem + G::kOffIn + q * (G::kStaging / 4) : nullptr;
        if constexpr (kSplit) {
          asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
          // Partial sums go to the CTA that owns the token, four tokens of a channel at a time (the sum
          // of integers is exact in any order); then this CTA's own share is completed and stored. No
          // CTA reads another's memory, so each may leave when it is done: two cluster barriers around
          // remote reads took 4000 clocks more.
          constexpr bool kHalves = G::kMaxSplit == 2;  // shares of whole chunks, of any size
          static_assert(!kHalves || kBT % (2 * kChunk) == 0, "shares");
          const int per_log = kHalves ? 31 : 31 - __clz(per);
          const int ch = q * 32 + lane;
          const uint32_t in_base = sbase + G::kOffIn, in_bar = smem_u32(&bars->in_full);
#pragma unroll 1
          for (int c = 0; c < kBT / kChunk; ++c) {
            if constexpr (kHalves) {
              if ((c * kChunk >= kBT / 2) == rank) continue;
            } else {
              if ((c * kChunk) >> per_log == rank && (c * kChunk + kChunk - 1) >> per_log == rank) continue;
            }
            uint32_t r[kChunk];
            const uint32_t t_col = t_lane + uint32_t(c * kChunk);
            if constexpr (kChunk == 16) tmem_ld16(t_col, r);
            else tmem_ld32(t_col, r);
            tmem_wait_ld();
            if constexpr (kHalves) {
              // one remote address for the chunk (one for every four tokens: 333 x 4099 x 8192 26 us for 21)
              const int at = (ch * (kBT / 2 + 4) + c * kChunk - (1 - rank) * (kBT / 2)) * 4;
              const uint32_t to = remote_addr(in_base + uint32_t(at), uint32_t(1 - rank)), bar = remote_addr(in_bar, uint32_t(1 - rank));
#pragma unroll
              for (int e = 0; e < kChunk; e += 4) push4(to + uint32_t(e * 4), r + e, bar);
            } else if (per_log >= 2) {
#pragma unroll
              for (int e = 0; e < kChunk; e += 4) {
                const int t = c * kChunk + e, dest = t >> per_log;
                const int slot = rank - (rank > dest ? 1 : 0);
                if (dest != rank)
                  push4(remote_addr(in_base + uint32_t(((slot * kBO + ch) * (per + 4) + (t & (per - 1))) * 4), uint32_t(dest)), r + e,
                        remote_addr(in_bar, uint32_t(dest)));
              }
            } else {
#pragma unroll
              for (int e = 0; e < kChunk; e += 2) {
                const int dest = (c * kChunk + e) >> 1;
                const int slot = rank - (rank > dest ? 1 : 0);
                if (dest != rank)
                  push2(remote_addr(in_base + uint32_t((slot * kBO + ch) * (per + 4) * 4), uint32_t(dest)), r + e,
                        remote_addr(in_bar, uint32_t(dest)));
              }
            }
          }
          if (!warp_wait(&bars->in_full, 0, &bars->abort, status, kStIn, p.limit_ns)) break;
#pragma unroll 1
          for (int c = rank * per / kChunk; c * kChunk < (rank + 1) * per; ++c) {
            uint32_t r[kChunk];
            const uint32_t t_col = t_lane + uint32_t(c * kChunk);
            if constexpr (kChunk == 16) tmem_ld16(t_col, r);
            else tmem_ld32(t_col, r);
            const int64_t tc = t0 + c * kChunk;
            const float as = (lane < kChunk && tc + lane < p.T) ? __ldg(p.a_scale + tc + lane) : 0.0f;
            tmem_wait_ld();
            for (int slot = 0; slot < p.split - 1; ++slot) {
              const int* in = reinterpret_cast<const int*>(smem + G::kOffIn) + (slot * kBO + ch) * (per + 4) - rank * per;
              if (per_log >= 2) {
#pragma unroll
                for (int e = 0; e < kChunk; e += 4) {
                  if (!kHalves && (c * kChunk + e) >> per_log != rank) continue;
                  const int4 v = *reinterpret_cast<const int4*>(in + c * kChunk + e);
                  r[e] += uint32_t(v.x);
                  r[e + 1] += uint32_t(v.y);
                  r[e + 2] += uint32_t(v.z);
                  r[e + 3] += uint32_t(v.w);
                }
              } else {
#pragma unroll
                for (int e = 0; e < kChunk; e += 2) {
                  if ((c * kChunk + e) >> 1 != rank) continue;
                  r[e] += uint32_t(in[c * kChunk + e]);
                  r[e + 1] += uint32_t(in[c * kChunk + e + 1]);
                }
              }
            }
            const bool there = o < p.O;
            Out* dst = static_cast<Out*>(p.C) + tc * p.O + o;
#pragma unroll
            for (int e = 0; e < kChunk; ++e, dst += p.O) {
              const float f = float(int(r[e])) * __shfl_sync(0xffffffffu, as, e) * ws;
              if (there && (kHalves || (c * kChunk + e) >> per_log == rank) && tc + e < p.T) *dst = to_out<Out>(f);
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kBT / kChunk; ++c)
            if (t0 + c * kChunk < p.T)
              store_chunk<kChunk, Out>(t_lane + uint32_t(buf * kBT + c * kChunk), p, t0 + c * kChunk, o0, ws, lane, stage, p.vec != 0);
        }
      } else if constexpr (kSplit) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      }
      // the accumulator is free for the tile after next
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->d_empty[buf]);
      if (!ok) break;
    }
  }

  if constexpr (kSplit) {
    if (warp == kWarpProducer || warp == kWarpMma) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
  if constexpr (kSplit) {
    // A CTA that gave up may still be sent partial sums: it stays until the others have sent theirs
    // (or have left, which counts as arriving) and what is on its way has landed, or a limit. One
    // that did not give up has waited for all of its own.
    if (*reinterpret_cast<volatile int*>(&bars->abort) != 0) {
      cluster_sync();
      if (threadIdx.x == 0) {
        const uint64_t tz = globaltimer();
        while (!mbar_try_wait(smem_u32(&bars->in_full), 0) && globaltimer() - tz < p.limit_ns) {
        }
      }
    }
  }
}

template <typename Out>
Params params_of(const I8GemmParams& g) {
  Params p{};
  p.a_scale = g.a_scale;
  p.w_scale = g.w_scale;
  p.C = g.C;
  p.status = g.status;
  p.T = g.T;
  p.O = g.O;
  p.nk = int((g.L + kBK - 1) / kBK);
  p.vec = (reinterpret_cast<uintptr_t>(g.C) & 15u) == 0 && (g.O * int64_t(sizeof(Out))) % 16 == 0;
  p.stall = g.stall_ns != 0;
  p.limit_ns = g.stall_ns != 0 ? g.stall_ns : kTimeoutNs;
  return p;
}

// ---- pairs of CTAs ----
constexpr int kPairStages = 6, kPairStage = 2 * kBO * kBK;  // 128 rows of W and of A per CTA
constexpr int kPairT = 256, kPairO = 256;
constexpr int kPairStaging = 4 * 32 * 32 * 4;
constexpr int kPairSmem = kPairStages * kPairStage + kPairStaging + 1024 + 512;
static_assert(kPairSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t dst, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}
// arrives at the barrier's place in both CTAs of the pair
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}

template <typename Out>
__global__ void __launch_bounds__(kThreads, 1)
i8gemm_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint32_t* const status = status_word(p.status);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + kPairStages * kPairStage + kPairStaging);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kPairT >> 3) << 17) | (uint32_t(kPairO >> 4) << 24);
  const int first = int(blockIdx.x) / 2, step = int(gridDim.x) / 2;
  const int n_local = first < p.num_tiles ? (p.num_tiles - 1 - first) / step + 1 : 0;

  // full and d_empty are the first CTA's (it issues the MMAs); empty and d_full are told to both
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->d_full[b], 1);
      mbar_init(&bars->d_empty[b], 8);
    }
    bars->abort = 0;
    fence_barrier_init();
    fence_proxy_async();
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == kWarpProducer) {
    if (lane == 0) {
      int it = 0;
      bool ok = p.stall == 0 || rank == 0;  // (test hook) the second CTA issues no loads
      for (int i = 0; ok && i < n_local; ++i) {
        const int tile = first + i * step;
        const int o0 = (tile % p.tiles_o) * kPairO + int(rank) * kBO, t0 = (tile / p.tiles_o) * kPairT + int(rank) * kBO;
        for (int kb = 0; kb < p.nk; ++kb, ++it) {
          const int s = it % kPairStages;
          if (it >= kPairStages &&
              !wait_bounded(&bars->empty[s], ((it / kPairStages) - 1) & 1, &bars->abort, status, kStEmpty, p.limit_ns)) {
            ok = false;
            break;
          }
          // the first CTA's barrier counts the bytes of both
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * kPairStage);
          const uint32_t bar = remote_addr(smem_u32(&bars->full[s]), 0);
          const uint32_t dst = sbase + s * kPairStage;
          tma_load_pair(dst, &map_w, kb * kBK, o0, bar);
          tma_load_pair(dst + kPairStage / 2, &map_a, kb * kBK, t0, bar);
        }
      }
      bars->issued = it;
    }
    __syncwarp();
  } else if (warp == kWarpMma && rank == 0) {
    const bool leader = elect_one();
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && i < n_local; ++i) {
      const int buf = i & 1;
      if (i >= 2 && !warp_wait(&bars->d_empty[buf], ((i >> 1) - 1) & 1, &bars->abort, status, kStDEmpty, p.limit_ns)) break;
      tc_fence_after();
      for (int kb = 0; kb < p.nk; ++kb, ++it) {
        const int s = it % kPairStages;
        if (!warp_wait(&bars->full[s], (it / kPairStages) & 1, &bars->abort, status, kStFull, p.limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t wd = sw128_desc(sbase + s * kPairStage), ad = sw128_desc(sbase + s * kPairStage + kPairStage / 2);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_i8_pair(tmem + uint32_t(buf * kPairT), wd + uint64_t((k * 32) >> 4), ad + uint64_t((k * 32) >> 4), kIdesc,
                        (kb > 0 || k > 0) ? 1u : 0u);
          commit_pair(&bars->empty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) commit_pair(&bars->d_full[buf]);
      __syncwarp();
    }
    // every MMA issued here has completed before TMEM is released: the last commit of each stage
    if (lane == 0) {
      for (int j = it > kPairStages ? it - kPairStages : 0; j < it; ++j) {
        const uint32_t b = smem_u32(&bars->empty[j % kPairStages]);
        const uint64_t tz = globaltimer();
        while (!mbar_try_wait(b, (j / kPairStages) & 1)) {
          if (globaltimer() - tz > p.limit_ns) {
            atomicOr(status, kStDrain);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= kWarpEpi0) {
    const int q = warp - kWarpEpi0;
    const uint32_t t_lane = tmem + (uint32_t(q * 32) << 16);
    uint8_t* stage = smem + kPairStages * kPairStage + q * (kPairStaging / 4);
    for (int i = 0; i < n_local; ++i) {
      const int tile = first + i * step;
      const int buf = i & 1;
      const int64_t o0 = int64_t(tile % p.tiles_o) * kPairO + int64_t(rank) * kBO + q * 32;
      const int64_t t0 = int64_t(tile / p.tiles_o) * kPairT;
      const bool ok = warp_wait(&bars->d_full[buf], (i >> 1) & 1, &bars->abort, status, kStDFull, p.limit_ns);
      if (ok) {
        tc_fence_after();
        const float ws = o0 + lane < p.O ? __ldg(p.w_scale + o0 + lane) : 0.0f;
#pragma unroll 1
        for (int c = 0; c < kPairT / 32; ++c)
          if (t0 + c * 32 < p.T)
            store_chunk<32, Out>(t_lane + uint32_t(buf * kPairT + c * 32), p, t0 + c * 32, o0, ws, lane, stage, p.vec != 0);
      }
      // the accumulator is free for the tile after next
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = remote_addr(smem_u32(&bars->d_empty[buf]), 0);
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
      }
      if (!ok) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {  // how this CTA ended, for the other one
    st_cluster(remote_addr(smem_u32(&bars->other_abort), rank ^ 1u), bars->abort);
    st_cluster(remote_addr(smem_u32(&bars->other_issued), rank ^ 1u), bars->issued);
  }
  cluster_sync();  // neither leaves while the other's MMAs or arrivals may reach it
  if (bars->abort != 0 || bars->other_abort != 0) {
    // One of them gave up, so loads may be in flight (in a call that is in order every stage has been
    // multiplied). Both CTAs' loads are counted by the first one's barriers: it waits for the last
    // stages, or a limit, arming those that only the second CTA has loaded; then both leave.
    if (rank == 0 && threadIdx.x == 0) {
      for (int j = bars->issued; j < bars->other_issued; ++j)
        mbar_arrive_expect_tx(&bars->full[j % kPairStages], kPairStage);
      const int n = max(bars->issued, bars->other_issued);
      const uint64_t tz = globaltimer();
      for (int j = max(n - kPairStages, 0); j < n; ++j)
        while (!mbar_try_wait(smem_u32(&bars->full[j % kPairStages]), (j / kPairStages) & 1) &&
               globaltimer() - tz < p.limit_ns) {
        }
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <typename Out>
cudaError_t launch_pair(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  CUtensorMap map_w, map_a;
  if (!encode_bytes_2d(&map_w, g.w, uint64_t(g.O), uint64_t(g.L), kBK, kBO) ||
      !encode_bytes_2d(&map_a, g.a, uint64_t(g.T), uint64_t(g.L), kBK, kBO))
    return cudaErrorInvalidValue;
  Params p = params_of<Out>(g);
  p.tiles_o = int((g.O + kPairO - 1) / kPairO);
  p.num_tiles = p.tiles_o * int((g.T + kPairT - 1) / kPairT);
  p.split = 1;
  auto kern = i8gemm_pair_kernel<Out>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kern), kPairSmem);
  if (e != cudaSuccess) return e;
  const int pairs = p.num_tiles < num_sms / 2 ? p.num_tiles : num_sms / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_a, p);
}

template <int kBT, typename Out, bool kSplit>
cudaError_t launch_t(const I8GemmParams& g, int split, int num_sms, cudaStream_t stream) {
  using G = Geo<kBT, kSplit>;
  CUtensorMap map_w, map_a;
  if (!encode_bytes_2d(&map_w, g.w, uint64_t(g.O), uint64_t(g.L), kBK, kBO) ||
      !encode_bytes_2d(&map_a, g.a, uint64_t(g.T), uint64_t(g.L), kBK, kBT))
    return cudaErrorInvalidValue;
  Params p = params_of<Out>(g);
  p.tiles_o = int((g.O + kBO - 1) / kBO);
  p.num_tiles = p.tiles_o * int((g.T + kBT - 1) / kBT);
  p.split = split;
  auto kern = i8gemm_kernel<kBT, Out, kSplit>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kern), G::kSmem);
  if (e != cudaSuccess) return e;
  const int resident = num_sms * G::kMinBlocks;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(kSplit ? p.num_tiles * split : (p.num_tiles < resident ? p.num_tiles : resident)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kSplit ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_a, p);
}

template <int kBT, typename Out>
cudaError_t launch_tile(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  using G = Geo<kBT, true>;
  const int64_t tiles = ((g.O + kBO - 1) / kBO) * ((g.T + kBT - 1) / kBT), nk = (g.L + kBK - 1) / kBK;
  // Split K while that takes no SM a second CTA (1 x 14336 x 4096, 112 tiles: whole 14.5 us, in two
  // 15.4; 1 x 4096 x 4096, 32 tiles: whole 13.2, in four 8.5, in eight 10.3) and as long as each CTA keeps
  // four stages of work (4 x 2048 x 2048: 5.8 us with four, 6.6 with eight), or eight where the partial
  // sums are 96 KB or more (300 x 1024 x 1024: whole 8.7 us, in two 9.2; 512 x 1024 x 1024 9.9 and 11.0).
  constexpr int kLeast = kBT >= 192 ? 8 : 4;
  int split = 1;
  while (split < G::kMaxSplit && tiles * split * 2 <= num_sms && nk >= split * 2 * kLeast) split *= 2;
  return split > 1 ? launch_t<kBT, Out, true>(g, split, num_sms, stream) : launch_t<kBT, Out, false>(g, 1, num_sms, stream);
}

template <typename Out>
cudaError_t launch_out(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  // the narrowest tile that takes all tokens: 1 x 14336 x 4096 15 us with 16 columns, 20 with 64;
  // 16 x 6144 x 4096 10 and 13; 100 x 6144 x 4096 14 us with 128, 18 with 256
  if (g.T <= 16) return launch_tile<16, Out>(g, num_sms, stream);
  if (g.T <= 32) return launch_tile<32, Out>(g, num_sms, stream);
  if (g.T <= 64) return launch_tile<64, Out>(g, num_sms, stream);
  if (g.T <= 128) return launch_tile<128, Out>(g, num_sms, stream);
  // Pairs where their tiles take half of the machine or more (tiles of one CTA are then too many to be
  // split): 512 x 5120 x 14336 (40 tiles) 42.3 us, 51.8 with tiles of one CTA; 512 x 6144 x 4096 (48)
  // 19.0 and 20.3; 1024 x 6144 x 4096 (96) 28.5 and 32.4; with short rows 768 x 4096 x 1024 11.8 and 11.2.
  // Below it 333 x 4099 x 8192 (34) 26.5 and 21.4, split.
  const int64_t pairs = ((g.O + kPairO - 1) / kPairO) * ((g.T + kPairT - 1) / kPairT);
  if (pairs * 2 >= int64_t(num_sms / 2)) return launch_pair<Out>(g, num_sms, stream);
  // 192 token columns where that pads less than 256: 333 x 4099 x 8192 21.4 us for 25, 384 x 4096 x 14336
  // 30.1 for 36
  if ((g.T + 191) / 192 * 192 < (g.T + 255) / 256 * 256) return launch_tile<192, Out>(g, num_sms, stream);
  return launch_tile<256, Out>(g, num_sms, stream);
}

}  // namespace

cudaError_t i8gemm_status_word(uint32_t** word) {
  void* at = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&at, own_status);
  if (e == cudaSuccess) *word = static_cast<uint32_t*>(at);
  return e;
}

cudaError_t launch_i8gemm(const I8GemmParams& g, int num_sms, cudaStream_t stream) {
  switch (g.out_type) {
    case FQ_BF16: return launch_out<__nv_bfloat16>(g, num_sms, stream);
    case FQ_FP16: return launch_out<__half>(g, num_sms, stream);
    default: return launch_out<float>(g, num_sms, stream);
  }
}

}  // namespace fq
