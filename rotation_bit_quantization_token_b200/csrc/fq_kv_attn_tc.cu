// Attention over the 8-bit paged cache on the tensor cores (tcgen05): sequences with many rows,
// that is prompts and chunks of prompts.
//
// A row is a (new token, query head of the group) pair; one CTA takes two tiles of 128 rows of
// one sequence and key / value head, and a chunk of keys, 128 keys at a time:
//     S = Q K^T   (M = 128 rows, N = 128 keys, K = D; Q and K fp16 in shared memory)
//     P = exp2(S c - m c)                      (registers, one thread per row)
//     O += P V    (M = 128 rows, N = D, K = 128 keys; P fp16 in TMEM, V fp16 in shared memory)
// The two row tiles take turns: while one's softmax runs, the tensor cores do the other's
// products. Both share every converted tile of K and V.
//
// Codes reach the MMAs as fp16. A converter warpgroup moves the E4M3 bits into fp16 fields (every
// bit pattern gives a finite number, so stale bytes behind the last token cannot make a NaN) and
// multiplies by the page's power of two relative to the largest exponent among the sequence's
// pages, times 2^14: codes of pages down to 2^-38 of the largest keep all their bits. One power of
// two per row and one per output then undo all scaling: the score's factor c holds the softmax
// scale, log2 e, the q row's exponent and the keys' largest page exponent.
//
// Softmax. A thread owns one row (its TMEM lane), so no exchange is needed. The maximum that the
// exponents are taken against is only raised when a row exceeds it by 2^8 (the probabilities then
// stay below 2^8, within fp16, and relative rounding is the same): O and the sum are rescaled that
// rarely. Probabilities are rounded to fp16 (2^-11).
//
// Roles, 512 threads: warps 0-3 and 4-7 softmax of row tile 0 and 1 (and its output), 8-11
// converters, 12 TMA producer, 13 MMA issuer (owns TMEM). TMEM: O 2 x D columns, S 2 x 128 columns
// (P overwrites the first half of its S). Every wait is bounded.
#include <cstdint>

#include "fq_kv_common.cuh"

namespace fq {
namespace {

using namespace ptx;
using namespace kv;

constexpr int kThreads = 512;
constexpr int kKeys = 128;  // keys of a step
constexpr int kWarpConv0 = 8, kWarpProducer = 12, kWarpMma = 13;
// Register split (setmaxnreg): launched at 128 per thread; 2 softmax warpgroups, the converters, the rest
constexpr int kRegsSoftmax = 200, kRegsConv = 72, kRegsLow = 40;
static_assert(128 * (2 * kRegsSoftmax + kRegsConv + kRegsLow) <= kThreads * 128, "register split");

enum : uint32_t {
  kStRawFull = 1u << 0, kStRawEmpty = 1u << 1, kStKFull = 1u << 2, kStVFull = 1u << 3, kStKEmpty = 1u << 4,
  kStVEmpty = 1u << 5, kStSFull = 1u << 6, kStPFull = 1u << 7, kStOFull = 1u << 9, kStDrain = 1u << 10
};

template <int D>
struct Geo {
  static constexpr int kQBytes = 128 * D * 2;               // one row tile of Q
  static constexpr int kTile = kKeys * D * 2;               // a converted tile of K or V
  static constexpr int kRaw = kKeys * D;                    // its codes
  static constexpr int kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffRawK = kOffV + 2 * kTile;
  static constexpr int kOffRawV = kOffRawK + kRaw;
  static constexpr int kOffBars = kOffRawV + kRaw;
  static constexpr int kSmem = kOffBars + 1024 + 1024 /*alignment*/;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColO = 0, kColS = 2 * D, kCols = 512;
  static_assert(kColS + 256 <= kCols, "TMEM");
};

struct Bars {
  uint64_t raw_full[2], raw_empty[2];  // codes of K, of V
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int k_top, v_top;        // largest page exponents of the CTA's keys
  uint32_t valid[8];       // per step (mod 8): pages of the step that are there, one bit per 16 keys
  uint32_t factor[2][8];   // K, V: factor of each 16 keys of the step in the raw buffer, as half2
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int n>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}
// shared-memory descriptor with a leading-dimension offset (distance of the column atoms of an
// MN-major operand), 128-byte swizzle
__device__ __forceinline__ uint64_t desc_lbo(uint32_t saddr, uint32_t lbo) {
  const uint32_t lo = (saddr >> 4) | ((lbo >> 4) << 16);
  const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (uint64_t(hi) << 32) | lo;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kv_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const KvAttnParams p, const int row_tiles) {
  using G_ = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + G_::kOffBars);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps = p.c.page_size, H = p.c.kv_heads, G = p.q_heads / H;

  // the longest (last) row tiles first, so that the short ones fill the end of the launch
  int64_t idx = blockIdx.x;
  const int h = int(idx % H);
  idx /= H;
  const int b = int(idx % p.b.num_seqs);
  idx /= p.b.num_seqs;
  const int split = int(idx % p.tc_splits);
  const int tile = row_tiles - 1 - int(idx / p.tc_splits);

  const int64_t row0 = int64_t(tile) * kTcRows;
  const Rows s = sequence_rows(p, b, row0, kTcRows, G);
  if (tid == 0 && split == 0 && h == 0 && tile == 0 && p.status != nullptr && (!s.ok || s.n > p.max_q_len))
    atomicOr(p.status, FQ_KV_BAD_BATCH);
  const int rows = int(min(int64_t(kTcRows), s.n * G - row0));
  if (rows <= 0 || !takes_tc(p, s.n, G)) return;
  const int64_t c0 = int64_t(split) * p.tc_chunk;
  if (c0 >= s.end && split > 0) return;
  const int keys = int(min(int64_t(p.tc_chunk), s.end - c0));
  const bool whole = s.end <= p.tc_chunk;
  const int n_steps = (keys + kKeys - 1) / kKeys;
  const int n_tiles = rows > 128 ? 2 : 1;  // row tiles with rows
  const int* table = p.b.page_table + int64_t(b) * p.b.table_width + c0 / ps;
  const int n_pages = (keys + ps - 1) / ps;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], 4);
      mbar_init(&bars->k_full[i], 4);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], 4);
      mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_full[i], 1);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    bars->k_top = bars->v_top = kPageExpMin;
    fence_barrier_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bars->tmem_base, G_::kCols);
  __syncthreads();

  // ---- the largest page exponents, and Q ----
  {
    int kt = kPageExpMin, vt = kPageExpMin;
    for (int i = tid; i < n_pages; i += kThreads) {
      const int pg = __ldg(table + i);
      if (pg >= 0 && int64_t(pg) < p.c.num_pages) {
        kt = max(kt, page_exp(__ldg(p.c.k_scale + int64_t(pg) * H + h)));
        vt = max(vt, page_exp(__ldg(p.c.v_scale + int64_t(pg) * H + h)));
      } else if (p.status != nullptr) {
        atomicOr(p.status, FQ_KV_BAD_BATCH);
      }
    }
    kt = __reduce_max_sync(0xffffffffu, kt);
    vt = __reduce_max_sync(0xffffffffu, vt);
    if (lane == 0) {
      atomicMax(&bars->k_top, kt);
      atomicMax(&bars->v_top, vt);
    }
  }
  float c = 0.0f;   // factor of a score: z log2 e = S * c
  int64_t vis = 0;  // keys of the chunk that this thread's row sees
  if (warp < 8) {
    const int r = tid;  // row of the CTA, 0 .. 255
    const bool live = r < rows;
    const int64_t ri = row0 + r;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                          (live ? (s.t_first + ri / G) * p.q_stride + int64_t(h * G + ri % G) * D : 0);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (live) w = __ldg(reinterpret_cast<const uint4*>(src) + i);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack16(ww[e], p.fp16);
        amax = max3(amax, fabsf(f.x), fabsf(f.y));
      }
    }
    const int qe = row_exponent(amax);
    // the sign of the scale goes to Q (c stays positive, so a row's largest S is its largest
    // score); a zero scale makes Q zero
    const float f = p.scale == 0.0f ? 0.0f : (p.scale < 0.0f ? -exp2i(-qe) : exp2i(-qe));
    c = p.scale == 0.0f ? 1.0f : fabsf(p.scale) * kLog2e * exp2i(qe);
    const uint32_t dst = sbase + uint32_t((r >> 7) * G_::kQBytes + (r & 127) * 128);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (live) w = __ldg(reinterpret_cast<const uint4*>(src) + i);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        // elements 4j + 0, 2, 1, 3, the order of codes_lo and codes_hi
        const float2 a = unpack16(ww[e], p.fp16), d = unpack16(ww[e + 1], p.fp16);
        o[e] = h2(a.x * f, d.x * f);
        o[e + 1] = h2(a.y * f, d.y * f);
      }
      sts128(dst + uint32_t((i >> 3) * 16384) + uint32_t(((i & 7) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
    }
    int64_t v = s.len;
    if (p.causal) v = min(v, s.len - s.n + ri / G + 1);
    vis = live ? v - c0 : 0;
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int k_top = bars->k_top, v_top = bars->v_top;
  int* abort = &bars->abort;

  if (warp == kWarpProducer) {
    // ---------------- codes and page factors ----------------
    // Lane i < 8 looks after keys 16 i .. 16 i + 15 of every step: their page (two steps ahead)
    // and its scale bytes (one step ahead), so no load is waited for where it is used. The lane
    // whose keys begin a TMA box issues the box.
    setmaxnreg_dec<kRegsLow>();
    const int box = ps < kKeys ? ps : kKeys;
    auto page_of = [&](int j) {  // page of this lane's keys in step j, -1: none
      const int key = j * kKeys + lane * 16;
      if (lane >= 8 || j >= n_steps || key >= keys) return -1;
      const int pg = __ldg(table + key / ps);
      return pg >= 0 && int64_t(pg) < p.c.num_pages ? pg : -1;
    };
    auto bytes_of = [&](int pg) {
      if (pg < 0) return 0u;
      return uint32_t(__ldg(p.c.k_scale + int64_t(pg) * H + h)) | (uint32_t(__ldg(p.c.v_scale + int64_t(pg) * H + h)) << 8);
    };
    int pg0 = page_of(0), pg1 = page_of(1);
    uint32_t by0 = bytes_of(pg0);
    bool ok = true;
    int j = 0;
    for (; ok && j < n_steps; ++j) {
      const int pg2 = page_of(j + 2);
      const uint32_t by1 = bytes_of(pg1);
      const bool first_of_box = lane < 8 && (lane * 16) % box == 0 && pg0 >= 0;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, first_of_box));
      const uint32_t valid = __ballot_sync(0xffffffffu, pg0 >= 0);
      const int row = int(((int64_t(max(pg0, 0)) * H + h) * ps + (j * kKeys + lane * 16) % ps) * D / 128);
      // 2^(14 + exponent - top), zero below the range of fp16
      const int kd = 14 + page_exp(by0 & 0xFFu) - k_top, vd = 14 + page_exp(by0 >> 8) - v_top;
      const uint32_t kf = h2(exp2i(max(kd, -30)), exp2i(max(kd, -30))), vf = h2(exp2i(max(vd, -30)), exp2i(max(vd, -30)));
#pragma unroll
      for (int w = 0; ok && w < 2; ++w) {
        ok = j == 0 || warp_wait(&bars->raw_empty[w], (j - 1) & 1, abort, p.status, kStRawEmpty);
        if (!ok) break;
        if (lane < 8) bars->factor[w][lane] = w == 0 ? kf : vf;
        if (w == 0 && lane == 0) bars->valid[j & 7] = valid;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[w], boxes * uint32_t(box * D));
        __syncwarp();
        if (first_of_box)
          tma_load_2d(sbase + uint32_t((w == 0 ? G_::kOffRawK : G_::kOffRawV) + lane * 16 * D), w == 0 ? &map_k : &map_v, 0,
                      row, &bars->raw_full[w]);
        __syncwarp();
      }
      pg0 = pg1;
      pg1 = pg2;
      by0 = by1;
    }
    // the last copies have landed before the CTA may exit (each phase is also waited for by the
    // converters; after an abort they may have left)
    if (lane == 0 && j > 0) {
      for (int w = 0; w < 2; ++w) {
        const uint64_t t0 = globaltimer();
        while (!ok && !mbar_try_wait(smem_u32(&bars->raw_full[w]), (j - 1) & 1) && globaltimer() - t0 < kTimeoutNs / 4) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---------------- MMA issuer ----------------
    setmaxnreg_dec<kRegsLow>();
    const bool leader = elect_one();
    constexpr uint32_t kIdS = (1u << 4) | (uint32_t(kKeys >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) /*V is MN-major*/ | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    auto issue_s = [&](int w, int j) {
      const uint64_t q = sw128_desc(sbase + uint32_t(w * G_::kQBytes));
      const uint64_t k = sw128_desc(sbase + uint32_t(G_::kOffK + (j & 1) * G_::kTile));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = uint64_t(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
        mma_ss(tmem + G_::kColS + uint32_t(w * 128), q + off, k + off, kIdS, kk > 0 ? 1u : 0u);
      }
      mma_commit(&bars->s_full[w]);
    };
    bool ok = n_steps > 0 && warp_wait(&bars->k_full[0], 0, abort, p.status, kStKFull);
    if (ok) {
      tc_fence_after();
      if (leader) {
        for (int w = 0; w < n_tiles; ++w) issue_s(w, 0);
        mma_commit(&bars->k_empty[0]);
      }
      __syncwarp();
    }
    for (int j = 0; ok && j < n_steps; ++j) {
      const int st = j & 1;
      for (int w = 0; w < n_tiles; ++w) {
        ok = warp_wait(&bars->p_full[w], j & 1, abort, p.status, kStPFull);
        if (ok && w == 0) ok = warp_wait(&bars->v_full[st], (j >> 1) & 1, abort, p.status, kStVFull);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t v = desc_lbo(sbase + uint32_t(G_::kOffV + st * G_::kTile), 16384);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts(tmem + G_::kColO + uint32_t(w * D), tmem + G_::kColS + uint32_t(w * 128 + kk * 8),
                   v + uint64_t((kk * 2048) >> 4), kIdO, (j > 0 || kk > 0) ? 1u : 0u);
          if (w == n_tiles - 1) mma_commit(&bars->v_empty[st]);
          if (j == n_steps - 1) mma_commit(&bars->o_full[w]);
        }
        __syncwarp();
        if (j + 1 < n_steps) {
          if (w == 0) ok = warp_wait(&bars->k_full[st ^ 1], ((j + 1) >> 1) & 1, abort, p.status, kStKFull);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            issue_s(w, j + 1);
            if (w == n_tiles - 1) mma_commit(&bars->k_empty[st ^ 1]);
          }
          __syncwarp();
        }
      }
    }
    // every MMA issued here has completed before TMEM is released
    if (leader) mma_commit(&bars->mma_done);
    __syncwarp();
    if (lane == 0) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(smem_u32(&bars->mma_done), 0)) {
        if (globaltimer() - t0 > kTimeoutNs) {
          if (p.status != nullptr) atomicOr(p.status, kStDrain);
          break;
        }
      }
    }
    __syncwarp();
  } else if (warp >= kWarpConv0 && warp < kWarpConv0 + 4) {
    // ---------------- converters ----------------
    // Eight lanes of a warp take eight neighbouring keys and the same 16 codes of each: with the
    // 128-byte swizzle on both sides neither their reads nor their writes meet in a bank.
    setmaxnreg_dec<kRegsConv>();
    const int cw = warp - kWarpConv0;
    constexpr int kChunks = D / 16;  // 16-code chunks of a key
    constexpr int kIter = kKeys * kChunks / 128;
    bool ok = true;
    for (int j = 0; ok && j < n_steps; ++j) {
      const int st = j & 1;
#pragma unroll 1
      for (int w = 0; ok && w < 2; ++w) {
        ok = warp_wait(&bars->raw_full[w], j & 1, abort, p.status, kStRawFull);
        if (ok && j >= 2)
          ok = warp_wait(w == 0 ? &bars->k_empty[st] : &bars->v_empty[st], ((j >> 1) - 1) & 1, abort, p.status,
                         w == 0 ? kStKEmpty : kStVEmpty);
        if (!ok) break;
        const uint32_t raw = sbase + uint32_t(w == 0 ? G_::kOffRawK : G_::kOffRawV);
        const uint32_t dst = sbase + uint32_t((w == 0 ? G_::kOffK : G_::kOffV) + st * G_::kTile);
#pragma unroll
        for (int it = 0; it < kIter; ++it) {
          // groups of 8 keys x 4 chunks per warp and iteration
          const int unit = it * 4 + cw;
          const int key = (unit % 16) * 8 + (lane & 7);
          const int ch = (unit / 16) * 4 + (lane >> 3);
          const uint32_t o = uint32_t(key * D + ch * 16);
          const uint4 v = lds128(raw + (o ^ (((o >> 7) & 7u) << 4)));
          const uint32_t f = bars->factor[w][key >> 4];
          const uint32_t at = dst + uint32_t((ch >> 2) * 16384 + key * 128);
          const uint32_t c2 = uint32_t((ch & 3) * 2), k7 = uint32_t(key & 7);
          sts128(at + ((c2 ^ k7) << 4), hmul2(codes_lo(v.x), f), hmul2(codes_hi(v.x), f), hmul2(codes_lo(v.y), f),
                 hmul2(codes_hi(v.y), f));
          sts128(at + (((c2 + 1) ^ k7) << 4), hmul2(codes_lo(v.z), f), hmul2(codes_hi(v.z), f), hmul2(codes_lo(v.w), f),
                 hmul2(codes_hi(v.w), f));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->raw_empty[w]);
          mbar_arrive(w == 0 ? &bars->k_full[st] : &bars->v_full[st]);
        }
      }
    }
  } else if (warp < 8) {
    // ---------------- softmax and output of row tile w ----------------
    setmaxnreg_inc<kRegsSoftmax>();
    const int w = warp >> 2;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + G_::kColS + uint32_t(w * 128), t_o = t_lane + G_::kColO + uint32_t(w * D);
    if (p.scale != 0.0f) c = fmaxf(c * exp2i(k_top + 8 - 14), 1e-37f);  // positive: -inf * c is -inf
    float m = -INFINITY;  // the row's maximum that the exponents are taken against (of S)
    float2 l2 = make_float2(0.0f, 0.0f);
    bool ok = true;
    if (w < n_tiles) {
      for (int j = 0; j < n_steps; ++j) {
        ok = warp_wait(&bars->s_full[w], j & 1, abort, p.status, kStSFull);
        if (!ok) break;
        tc_fence_after();
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(t_s + uint32_t(i * 32), reinterpret_cast<uint32_t*>(x) + i * 32);
        tmem_wait_ld();
        const int left = int(min(vis - int64_t(j) * kKeys, int64_t(kKeys)));  // keys of the step that the row sees
        const uint32_t valid = bars->valid[j & 7];
        if (__any_sync(0xffffffffu, left < kKeys) || valid != 0xFFu) {
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (i >= left || ((valid >> (i / 16)) & 1u) == 0u) x[i] = -INFINITY;
        }
        float a0 = x[0], a1 = x[1], a2 = x[2], a3 = x[3];
#pragma unroll
        for (int i = 4; i < kKeys; i += 8) {
          a0 = max3(a0, x[i], x[i + 1]);
          a1 = max3(a1, x[i + 2], x[i + 3]);
          if (i + 4 < kKeys) {
            a2 = max3(a2, x[i + 4], x[i + 5]);
            a3 = max3(a3, x[i + 6], x[i + 7]);
          }
        }
        const float top = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
        // raise the maximum where the row is beyond it by 2^8 (or had none)
        const bool raise = top > m && !((top - m) * c <= 8.0f);
        if (__any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? (m == -INFINITY ? 0.0f : fast_exp2((m - top) * c)) : 1.0f;
          if (raise) m = top;
          l2.x *= alpha;
          l2.y *= alpha;
          if (j > 0) {
            // S(j) was issued after P V (j - 1) and has completed, so O is at rest
#pragma unroll
            for (int i = 0; i < D; i += 16) {
              uint32_t o[16];
              tmem_ld16(t_o + uint32_t(i), o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(t_o + uint32_t(i), o);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.0f : m;
        const float2 c2 = make_float2(c, c), n2 = make_float2(-mu * c, -mu * c);
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
        for (int i = 0; i < kKeys; i += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 u = __ffma2_rn(make_float2(x[i + e], x[i + e + 1]), c2, n2);
            float2 v = __ffma2_rn(make_float2(x[i + e + 2], x[i + e + 3]), c2, n2);
            u = make_float2(fast_exp2(u.x), fast_exp2(u.y));
            v = make_float2(fast_exp2(v.x), fast_exp2(v.y));
            sum0 = __fadd2_rn(sum0, u);
            sum1 = __fadd2_rn(sum1, v);
            pk[e / 2] = h2(u.x, u.y);
            pk[e / 2 + 1] = h2(v.x, v.y);
          }
          tmem_st16(t_s + uint32_t(i / 2), pk);
        }
        l2 = __fadd2_rn(l2, __fadd2_rn(sum0, sum1));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[w]);
      }
      if (ok && n_steps > 0) ok = warp_wait(&bars->o_full[w], 0, abort, p.status, kStOFull);
      if (ok) {
        tc_fence_after();
        const int r = tid;
        const bool live = r < rows;
        const int64_t ri = row0 + r;
        const int64_t row = (s.t_first + ri / G) * p.q_heads + h * G + ri % G;
        const float L = l2.x + l2.y;
        const float mz = m == -INFINITY ? -INFINITY : m * c;
        const float unit = exp2i(v_top + 8 - 14);
        const float inv = whole ? (L > 0.0f ? unit / L : 0.0f) : unit;
#pragma unroll
        for (int i = 0; i < D; i += 16) {
          uint32_t o[16];
          if (n_steps > 0) {
            tmem_ld16(t_o + uint32_t(i), o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          }
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {  // columns 0, 2, 1, 3 of every four
            y[e] = __uint_as_float(o[e]) * inv;
            y[e + 1] = __uint_as_float(o[e + 2]) * inv;
            y[e + 2] = __uint_as_float(o[e + 1]) * inv;
            y[e + 3] = __uint_as_float(o[e + 3]) * inv;
          }
          if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + i);
            dst[0] = make_uint4(pack16(y[0], y[1], p.fp16), pack16(y[2], y[3], p.fp16), pack16(y[4], y[5], p.fp16),
                                pack16(y[6], y[7], p.fp16));
            dst[1] = make_uint4(pack16(y[8], y[9], p.fp16), pack16(y[10], y[11], p.fp16), pack16(y[12], y[13], p.fp16),
                                pack16(y[14], y[15], p.fp16));
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(p.ws + (row * p.ws_splits + split) * (D + 4) + i);
#pragma unroll
            for (int e = 0; e < 16; e += 4) dst[e / 4] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        if (live && whole) {
          if (p.lse != nullptr) p.lse[row] = L > 0.0f ? (mz + log2f(L)) * kLn2 : -INFINITY;
        } else if (live) {
          float* dst = p.ws + (row * p.ws_splits + split) * (D + 4) + D;
          dst[0] = mz;
          dst[1] = L;
        }
      }
    }
  } else {
    setmaxnreg_dec<kRegsLow>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, G_::kCols);
  }
}

template <int D>
cudaError_t launch_tc(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  const uint64_t rows128 = uint64_t(p.c.num_pages) * p.c.kv_heads * p.c.page_size * D / 128;
  const int box = (p.c.page_size < kKeys ? p.c.page_size : kKeys) * D / 128;
  CUtensorMap map_k, map_v;
  if (!encode_bytes_2d(&map_k, p.c.k, rows128, 128, 128, uint32_t(box)) ||
      !encode_bytes_2d(&map_v, p.c.v, rows128, 128, 128, uint32_t(box)))
    return cudaErrorInvalidValue;
  auto kern = kv_attn_tc_kernel<D>;
  // setmaxnreg.inc draws on what the block was launched with
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != 128) return cudaErrorInvalidKernelImage;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(plan.tc_row_tiles) * p.c.kv_heads * plan.tc_splits * p.b.num_seqs;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  kern<<<unsigned(grid), kThreads, Geo<D>::kSmem, stream>>>(map_k, map_v, p, plan.tc_row_tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attn_tc(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  return p.c.head_dim == 128 ? launch_tc<128>(p, plan, stream) : launch_tc<64>(p, plan, stream);
}

}  // namespace fq
