// Attention over the 8-bit paged cache for sequences with few rows: decode steps.
//
// Rows are (new token, query head) pairs that share one key / value head (row r of a sequence: token
// r / G, head r % G of the group, G = q_heads / kv_heads), 8 or 16 of them per CTA, so a decode step
// reads each cached byte once for the whole group. The kernel is bound by reading the cache: 2 D
// bytes a token and head: 64 sequences of 500-16000 tokens, 8 heads of 128, take 173 us, 6.0 TB/s (189 us
// when repeated for long); one of 700 tokens takes 7.6 us, which is launch and latency.
//
// One CTA takes its rows and one chunk of keys; its four warps take tiles of 4096 / D keys in turn,
// each through a ring of its own (TMA boxes of 128-byte rows, swizzled; no barrier between the
// warps), with a running maximum, sum and output of its own; they are joined through shared memory
// at the end. The chunks of a longer sequence are joined by their cluster, each CTA reading a share of
// the others' results in shared memory, or, where they are too many, by a second kernel from partial
// results in the workspace.
//
// Products are mma.sync with the keys (then the output columns) on the M side and the rows on N: with
// 8 rows nothing is padded, and a thread holds a quarter of the output registers of the other
// orientation. S^T = K Q^T: a thread's words of K are codes of neighbouring d, which two conversions
// turn into one A fragment (the sum over d may run in any order, so q is held in the order that the
// words give). O^T += V^T P^T: P^T's fragments are those of S^T, transposed in registers (movmatrix);
// V^T's put two keys side by side, one byte permute for two codes.
//
// Numbers. A code becomes fp16 by the hardware conversion; keys behind the last token (or on a
// missing page) are zeroed in shared memory first, since stale bytes may be E4M3's NaN pattern. A row
// of q is scaled by the power of two that brings its largest magnitude into [2^14, 2^15) and
// converted to fp16: exact but for elements 2^-29 below the largest. The products are then exact in
// the fp32 sums of mma.sync, and the powers of two (q row, page of k) are applied to the score in
// float32. Probabilities are taken times 2^15 and rounded to fp16 for the second product: by 2^-11, or
// 2^-40 of the row's largest where they are below 2^-29 of it. The output accumulates
// in units of the page's own scale of v and moves to the next page's unit by a power of two, so that
// no page's scale has to fit beside another's in fp16: exponents lie in [-40, 40], so a unit changes
// by at most 2^80 and float32 holds all of it.
#include <cstdint>

#include "fq_kv_common.cuh"

namespace fq {
namespace {

using namespace ptx;
using namespace kv;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxChunkBytes = 4096 * 128;  // of K in one chunk (V as much again)
constexpr int kMaxCluster = 8;              // chunks that are joined in a cluster, at most
constexpr float kHeadroom = 15.0f;          // the largest probability is 2^15 before it is divided by the sum

enum : uint32_t { kStFull = 1u << 0 };

template <int D, int NT>
struct Geo {
  static constexpr int kRows = 8 * NT;                      // rows of a CTA
  static constexpr int kTileKeys = 4096 / D;                // keys of one warp's step
  static constexpr int kTileBytes = 4096;                   // codes of K (or V) of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kMinBlocks = NT == 1 ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kOStride = D + 4;                    // floats per row of a warp's output
  static constexpr int kJoinAt = kWarps * kRows * kOStride * 4;  // the CTA's own result, for its cluster
  static_assert(kJoinAt + kRows * kOStride * 4 <= kRing, "outputs fit the ring");
};

struct Shared {
  uint64_t full[kWarps][4];
  float m[kWarps][16], l[kWarps][16];
  int nan_from[128];  // per column: see hide_nans
  int nans;           // whether there is one
  int abort;
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// Byte offset of (key, byte d) in a tile of 128-byte swizzled rows (128 / D keys per row).
template <int D>
__device__ __forceinline__ uint32_t swz(int key, int d) {
  const uint32_t o = uint32_t(key * D + d);
  return o ^ (((o >> 7) & 7u) << 4);
}

// Words of the shared memory of a CTA of the cluster.
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Two E4M3 codes (the low and the high half of w) as two fp16 numbers each.
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Transposes the warp's 8 x 8 matrix of 16-bit elements (lane 4r + c holds row r, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// kOne: at most one query token a sequence, so all rows see the same keys (the code for others costs a
// decode batch 1.2 us of 173 although it is not reached)
template <int D, int NT, bool kOne>
__global__ void __launch_bounds__(kThreads, Geo<D, NT>::kMinBlocks)
kv_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const KvAttnParams p, const int row_tiles) {
  using G_ = Geo<D, NT>;
  constexpr int kTK = G_::kTileKeys, kRowsTile = G_::kRows;
  constexpr int kS = D / 16;      // k steps of q k^T, 16-column blocks of the output
  constexpr int kMT = kTK / 16;   // blocks of 16 keys of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared* sh = reinterpret_cast<Shared*>(smem + G_::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int H = p.c.kv_heads, G = p.q_heads / H;
  const int ps_log = 31 - __clz(p.c.page_size), ps = 1 << ps_log;

  grid_dependency_launch();
  unsigned idx = blockIdx.x;
  int split = 0;
  if (p.cluster) {  // the chunks of a row lie side by side
    split = int(idx % unsigned(p.splits));
    idx /= unsigned(p.splits);
  }
  const int tile = int(idx % unsigned(row_tiles));
  idx /= unsigned(row_tiles);
  const int h = int(idx % unsigned(H));
  idx /= unsigned(H);
  if (!p.cluster) {
    split = int(idx % unsigned(p.splits));
    idx /= unsigned(p.splits);
  }
  const int b = int(idx);

  const Rows s = sequence_rows(p, b, int64_t(tile) * kRowsTile, kRowsTile, G);
  if (tid == 0 && split == 0 && h == 0 && tile == 0 && p.status != nullptr && (!s.ok || s.n > p.max_q_len))
    atomicOr(p.status, FQ_KV_BAD_BATCH);
  const int row0 = tile * kRowsTile;
  const int rows = int(min(int64_t(kRowsTile), s.q * G - row0));
  if (rows <= 0 || takes_tc(p, s.q, G)) return;
  const int64_t c0 = int64_t(split) * p.chunk;  // first key of the chunk
  if (c0 >= s.end && split > 0) return;
  const int keys = int(min(int64_t(p.chunk), s.end - c0));
  const bool whole = s.end <= p.chunk;          // no other chunk: the result is final

  // ---- q on its way: this thread's elements t4 * D/4 .. + D/4 of row g (and g + 8) ----
  uint4 qw[NT][D / 32];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + g + 8 * n;
    const bool live = g + 8 * n < rows;
    const int64_t base = live ? (s.t_first + r / G) * p.q_stride + int64_t(h * G + r % G) * D + t4 * (D / 4) : 0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      qw[n][c] = live ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + base) + c) : make_uint4(0u, 0u, 0u, 0u);
  }

  // ---- page numbers of the chunk, barriers ----
  // scales beside them: (k exponent, v exponent) as bytes; a page outside the cache is -1
  int* s_page = reinterpret_cast<int*>(sh + 1);
  uint16_t* s_scale = reinterpret_cast<uint16_t*>(s_page + (p.chunk >> ps_log) + 1);
  const int n_pages = (keys + ps - 1) >> ps_log;
  if (tid < kWarps * G_::kStages) {
    mbar_init(&sh->full[tid / G_::kStages][tid % G_::kStages], 1);
    fence_barrier_init();
    fence_proxy_async();
  }
  if (tid == 0) sh->abort = sh->nans = 0;
  if (!kOne) sh->nan_from[tid] = kNoNan;
  const int* table = p.b.page_table + int64_t(b) * p.b.table_width + (c0 >> ps_log);
  for (int i = tid; i < n_pages; i += kThreads) {
    int pg = __ldg(table + i);
    if (pg < 0 || int64_t(pg) >= p.c.num_pages) {
      pg = -1;
      if (p.status != nullptr) atomicOr(p.status, FQ_KV_BAD_BATCH);
    }
    s_page[i] = pg;
  }
  __syncthreads();

  const int n_tiles = (keys + kTK - 1) / kTK;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * G_::kStages * G_::kStageBytes);
  const int box_log = min(ps_log, kTK == 32 ? 5 : 6);  // keys of one TMA box
  // Loads tile w of the chunk into a stage: lane 2i takes box i of K, lane 2i + 1 box i of V. Boxes
  // that start behind the last key, or whose page is missing, are left out.
  auto issue = [&](int w, int stage) {
    uint64_t* bar = &sh->full[warp][stage];
    const int at = w * kTK + ((lane >> 1) << box_log);
    int pg = -1;
    if (((lane >> 1) << box_log) < kTK && at < keys) pg = s_page[at >> ps_log];
    const uint32_t n = uint32_t(__popc(__ballot_sync(0xffffffffu, pg >= 0)));
    if (lane == 0) mbar_arrive_expect_tx(bar, n * uint32_t(D << box_log));
    __syncwarp();
    if (pg >= 0) {
      const int row = int((((int64_t(pg) * H + h) << ps_log) + (at & (ps - 1))) * D / 128);
      const uint32_t dst = ring + uint32_t(stage * G_::kStageBytes + (lane & 1) * G_::kTileBytes + ((lane >> 1) << box_log) * D);
      tma_load_2d(dst, (lane & 1) ? &map_v : &map_k, 0, row, bar);
    }
  };
#pragma unroll
  for (int st = 0; st < G_::kStages; ++st)
    if (warp + st * kWarps < n_tiles) issue(warp + st * kWarps, st);

  bool missing = false;  // a page of the chunk is not there
  for (int i = tid; i < n_pages; i += kThreads) {
    const int pg = s_page[i];
    int ke = 0, ve = 0;
    if (pg >= 0) {
      ke = page_exp(__ldg(p.c.k_scale + int64_t(pg) * H + h));
      ve = page_exp(__ldg(p.c.v_scale + int64_t(pg) * H + h));
    } else {
      missing = true;
    }
    s_scale[i] = uint16_t((ke + 127) | ((ve + 127) << 8));
  }

  // ---- q as fragments ----
  uint32_t qf[NT][kS][2];
  float rowf[NT][2];  // score factor of rows 2 t4, 2 t4 + 1 (+ 8)
  int vis[NT][2];     // keys of the chunk that they see
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + g + 8 * n;
    const bool live = g + 8 * n < rows;
    float x[D / 4];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint32_t ww[4] = {qw[n][c].x, qw[n][c].y, qw[n][c].z, qw[n][c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack16(ww[e], p.fp16);
        x[c * 8 + 2 * e] = f.x;
        x[c * 8 + 2 * e + 1] = f.y;
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int qe = row_exponent(amax);
    const float f = exp2i(-qe);
#pragma unroll
    for (int st = 0; st < kS; ++st) {
      qf[n][st][0] = h2(x[4 * st] * f, x[4 * st + 1] * f);
      qf[n][st][1] = h2(x[4 * st + 2] * f, x[4 * st + 3] * f);
    }
    int64_t v = s.len;
    if (p.causal) v = min(v, s.len - s.n + int64_t(r / G) + 1);
    const int see = live ? int(max(min(v - c0, int64_t(keys)), int64_t(0))) : 0;
    const float rf = p.scale * kLog2e * exp2i(qe);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // row 2 t4 + e belongs to the lanes of g = 2 t4 + e
      rowf[n][e] = __shfl_sync(0xffffffffu, rf, (2 * t4 + e) * 4);
      vis[n][e] = __shfl_sync(0xffffffffu, see, (2 * t4 + e) * 4);
    }
  }
  int all_see = keys;  // keys that every row sees
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (8 * n + 2 * t4 + e < rows) all_see = min(all_see, vis[n][e]);
  all_see = __reduce_min_sync(0xffffffffu, all_see);
  const bool uneven = !kOne && all_see < keys;  // a row does not see some of the keys
  missing = __syncthreads_or(missing);  // and the scales are there

  float o[kS][NT][4];
#pragma unroll
  for (int j = 0; j < kS; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][n][e] = 0.0f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[n][e] = -INFINITY;
      l[n][e] = 0.0f;
    }
  int unit = 0;        // exponent of the output's current unit
  bool first_unit = true;

  int stage = 0, phase = 0, in_flight = 0;
  for (int w = warp; w < n_tiles; w += kWarps) {
    if (!warp_wait(&sh->full[warp][stage], uint32_t(phase), &sh->abort, p.status, kStFull)) {
      // this warp's loads in flight land before its memory is used again (or a limit)
      for (; w < n_tiles && lane == 0; w += kWarps) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&sh->full[warp][stage]), uint32_t(phase)) && globaltimer() - t0 < kTimeoutNs / 4) {
        }
        if (++stage == G_::kStages) {
          stage = 0;
          phase ^= 1;
        }
        if (++in_flight == G_::kStages) break;
      }
      __syncwarp();
      break;
    }
    const uint32_t kbase = ring + uint32_t(stage * G_::kStageBytes), vbase = kbase + G_::kTileBytes;
    const int k0 = w * kTK;
    if (k0 + kTK > keys || missing) {
      // zero the keys that are not there
      for (int i = lane; i < kTK * (D / 16); i += 32) {
        const int key = i / (D / 16);
        if (k0 + key >= keys || s_page[(k0 + key) >> ps_log] < 0) {
          const uint32_t at = swz<D>(key, (i % (D / 16)) * 16);
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(kbase + at), "r"(0u) : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vbase + at), "r"(0u) : "memory");
        }
      }
      fence_proxy_async();  // the stage is written by TMA again later
      __syncwarp();
    }
    if (uneven && k0 + kTK > all_see) {
      for (int i = lane; i < kTK * (D / 16); i += 32) {
        const int key = i / (D / 16), d = (i % (D / 16)) * 16;
        uint4 v = lds128(vbase + swz<D>(key, d));
        if (has_nan(v)) {
          hide_nans(v, k0 + key, d, sh->nan_from);
          sh->nans = 1;
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(vbase + swz<D>(key, d)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
      }
      fence_proxy_async();
      __syncwarp();
    }

    // ---- scores ----
    float sc[kMT][NT][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 ka = lds128(kbase + swz<D>(mt * 16 + g, t4 * (D / 4) + c * 16));
        const uint4 kb = lds128(kbase + swz<D>(mt * 16 + g + 8, t4 * (D / 4) + c * 16));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a[4];
          cvt4(wa[e], a[0], a[2]);
          cvt4(wb[e], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(sc[mt][n], a, qf[n][c * 4 + e][0], qf[n][c * 4 + e][1]);
        }
      }
    }
    const bool masked = k0 + kTK > all_see || missing;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const int pg_i = min((k0 + mt * 16) >> ps_log, n_pages - 1);
      const float pf = exp2i(int(s_scale[pg_i] & 0xFFu) - 127);
      const bool there = !missing || s_page[pg_i] >= 0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = sc[mt][n][e] * (rowf[n][e & 1] * pf);
          sc[mt][n][e] = !masked || (there && k0 + mt * 16 + g + 8 * (e >> 1) < vis[n][e & 1]) ? v : -INFINITY;
        }
    }
    float alpha[NT][2], mu[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mt_max = fmaxf(sc[0][n][e], sc[0][n][e + 2]);
#pragma unroll
        for (int mt = 1; mt < kMT; ++mt) mt_max = fmaxf(mt_max, fmaxf(sc[mt][n][e], sc[mt][n][e + 2]));
        mt_max = fmaxf(mt_max, __shfl_xor_sync(0xffffffffu, mt_max, 4));
        mt_max = fmaxf(mt_max, __shfl_xor_sync(0xffffffffu, mt_max, 8));
        mt_max = fmaxf(mt_max, __shfl_xor_sync(0xffffffffu, mt_max, 16));
        // (rounded up: where scores are so large that 15 is lost beside them, nothing passes 2^15)
        const float mn = fmaxf(m[n][e], __fsub_ru(mt_max, kHeadroom));
        mu[n][e] = mn == -INFINITY ? 0.0f : mn;  // a row that has seen nothing yet
        alpha[n][e] = fast_exp2(m[n][e] - mu[n][e]);
        m[n][e] = mn;
        l[n][e] *= alpha[n][e];
      }

    // ---- probabilities and output, 16 keys at a time (within one page) ----
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const int pg_i = min((k0 + mt * 16) >> ps_log, n_pages - 1);
      const int ev = int(s_scale[pg_i] >> 8) - 127;
      if (ev != unit) {
        if (!first_unit) {
          const float u = exp2i(unit - ev);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            alpha[n][0] *= u;
            alpha[n][1] *= u;
          }
        }
        unit = ev;
      }
      first_unit = false;
      bool same = true;
#pragma unroll
      for (int n = 0; n < NT; ++n) same = same && alpha[n][0] == 1.0f && alpha[n][1] == 1.0f;
      if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int j = 0; j < kS; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[j][n][0] *= alpha[n][0];
            o[j][n][1] *= alpha[n][1];
            o[j][n][2] *= alpha[n][0];
            o[j][n][3] *= alpha[n][1];
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        alpha[n][0] = alpha[n][1] = 1.0f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float a = fast_exp2(sc[mt][n][2 * hh] - mu[n][0]), c = fast_exp2(sc[mt][n][2 * hh + 1] - mu[n][1]);
          l[n][0] += a;
          l[n][1] += c;
          pb[n][hh] = transpose8(h2(a, c));
        }
      }
      // this thread's keys 2 t4, + 1, + 8, + 9 and output columns g * D/8 .. + D/8
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = vbase + swz<D>(mt * 16 + 2 * t4 + (i & 1) + 8 * (i >> 1), g * (D / 8));
        if constexpr (D == 128) {
          const uint4 x = lds128(at);
          v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
        } else {
          const uint2 x = lds64(at);
          v[i][0] = x.x; v[i][1] = x.y;
        }
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t y[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) cvt4(v[i][c], y[i][0], y[i][1]);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const uint32_t a[4] = {__byte_perm(y[0][d], y[1][d], 0x5410), __byte_perm(y[0][d], y[1][d], 0x7632),
                                 __byte_perm(y[2][d], y[3][d], 0x5410), __byte_perm(y[2][d], y[3][d], 0x7632)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(o[c * 2 + d][n], a, pb[n][0], pb[n][1]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (w + G_::kStages * kWarps < n_tiles) issue(w + G_::kStages * kWarps, stage);
    if (++stage == G_::kStages) {
      stage = 0;
      phase ^= 1;
    }
  }

  // ---- join the warps ----
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
    }
  const float uf = exp2i(unit);  // out of the page's unit
  __syncthreads();               // every warp has left its ring
  float* so = reinterpret_cast<float*>(smem) + warp * kRowsTile * G_::kOStride;
#pragma unroll
  for (int j = 0; j < kS; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // block j's row g is output column g * D/8 + 2 j, its row g + 8 the next one
      float* x = so + (8 * n + 2 * t4) * G_::kOStride + g * (D / 8) + 2 * j;
      *reinterpret_cast<float2*>(x) = make_float2(o[j][n][0] * uf, o[j][n][2] * uf);
      *reinterpret_cast<float2*>(x + G_::kOStride) = make_float2(o[j][n][1] * uf, o[j][n][3] * uf);
    }
  if (g == 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sh->m[warp][8 * n + 2 * t4 + e] = m[n][e];
        sh->l[warp][8 * n + 2 * t4 + e] = l[n][e];
      }
  }
  __syncthreads();
  const bool meet = p.cluster && !whole;
  const bool gave_up = *reinterpret_cast<volatile int*>(&sh->abort) != 0;
  if (gave_up && !meet) return;
  constexpr int kTpr = kThreads / kRowsTile;  // threads per row
  constexpr int kPer = D / kTpr;              // columns of a thread
  const int r = tid / kTpr, d0 = (tid % kTpr) * kPer;
  if (r >= rows && !meet) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh->m[w][r]);
  const float Mu = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = fast_exp2(sh->m[w][r] - Mu);
    L += sh->l[w][r] * f;
    const float* x = reinterpret_cast<const float*>(smem) + (w * kRowsTile + r) * G_::kOStride + d0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += x[e] * f;
  }
  if (!kOne && sh->nans != 0) {
    int64_t v = s.len;
    if (p.causal) v = min(v, s.len - s.n + int64_t((row0 + r) / G) + 1);
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (sh->nan_from[d0 + e] < v - c0) acc[e] = NAN;
  }
  if (meet) {
    // A CTA that gave up takes part as well (the others read its memory; the result is undefined),
    // one without keys has left and is not read.
    float* own = reinterpret_cast<float*>(smem + G_::kJoinAt) + r * G_::kOStride;
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<float4*>(own + d0 + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    if (d0 == 0) *reinterpret_cast<float2*>(own + D) = make_float2(M, L);
    __syncwarp();
    cluster_sync();
    const int n = int((s.end + p.chunk - 1) / p.chunk);
    for (int i = split * kThreads + tid; i < rows * (D / 4); i += n * kThreads) {
      const int rr = i / (D / 4), col = i % (D / 4);
      const uint32_t at = smem_u32(smem) + uint32_t(G_::kJoinAt + rr * G_::kOStride * 4);
      float2 ml[kMaxCluster];
      float4 v[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        ml[c] = make_float2(-INFINITY, 0.0f);
        v[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < n) {
          const uint32_t from = remote_addr(at, uint32_t(c));
          ml[c] = ld_cluster2(from + D * 4);
          v[c] = ld_cluster4(from + col * 16);
        }
      }
      float Mc = -INFINITY, Lc = 0.0f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) Mc = fmaxf(Mc, ml[c].x);
      const float mu = Mc == -INFINITY ? 0.0f : Mc;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const float f = fast_exp2(ml[c].x - mu);
        Lc += ml[c].y * f;
        sum.x += v[c].x * f;
        sum.y += v[c].y * f;
        sum.z += v[c].z * f;
        sum.w += v[c].w * f;
      }
      // (a sum of zero is a row that sees no token; one that is not a number belongs to a NaN that it sees)
      const float inv = Lc != 0.0f ? 1.0f / Lc : 0.0f;
      const int64_t row = (s.t_first + (row0 + rr) / G) * p.q_heads + h * G + (row0 + rr) % G;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + 4 * col) =
          make_uint2(pack16(sum.x * inv, sum.y * inv, p.fp16), pack16(sum.z * inv, sum.w * inv, p.fp16));
      if (p.lse != nullptr && col == 0) p.lse[row] = Lc != 0.0f ? (mu + log2f(Lc)) * kLn2 : -INFINITY;
    }
    __syncwarp();
    cluster_sync();  // none leaves while its memory is read
    return;
  }
  const int64_t row = (s.t_first + (row0 + r) / G) * p.q_heads + h * G + (row0 + r) % G;
  if (whole) {
    const float inv = L != 0.0f ? 1.0f / L : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + d0);
#pragma unroll
    for (int e = 0; e < kPer / 2; e += 2)
      *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack16(acc[2 * e] * inv, acc[2 * e + 1] * inv, p.fp16),
                                                      pack16(acc[2 * e + 2] * inv, acc[2 * e + 3] * inv, p.fp16));
    if (p.lse != nullptr && d0 == 0) p.lse[row] = L != 0.0f ? (Mu + log2f(L)) * kLn2 : -INFINITY;
  } else {
    float* dst = p.ws + (row * p.ws_splits + split) * (D + 4);
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<float4*>(dst + d0 + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    if (d0 == 0) {
      dst[D] = M;
      dst[D + 1] = L;
    }
  }
}

// Joins the chunks of the rows that had more than one and no cluster. D / 4 threads lie side by side on a row's
// columns; kWide: a CTA takes one row, its groups of D / 4 threads different chunks of it (few rows
// with hundreds of chunks: a group alone took longer than the attention itself); else every group
// has a row of its own (many rows with a few chunks).
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads)
kv_attn_join_kernel(const KvAttnParams p, const int few) {
  constexpr int kCols = D / 4, kGroups = kThreads / kCols;
  const int tid = threadIdx.x;
  const int col = tid % kCols, grp = tid / kCols;
  int64_t row = kWide ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * kGroups + grp;
  const int G = p.q_heads / p.c.kv_heads;
  int64_t t = 0;
  int hq = 0, lo = 0;
  bool live = true;
  if (few > 0) {
    // only sequences of at most `few` rows can have chunks: row r of head h of sequence b
    const int64_t bh = row / few;
    const int r = int(row - bh * few), h = int(bh % p.c.kv_heads);
    live = bh / p.c.kv_heads < p.b.num_seqs;
    lo = live ? int(bh / p.c.kv_heads) : 0;
    hq = h * G + r % G;
    t = int64_t(__ldg(p.b.cu_new + lo)) + r / G;
    live = live && t >= 0 && t < p.T;
    row = t * p.q_heads + hq;
  } else {
    live = row < p.T * p.q_heads;
    t = row / p.q_heads;
    hq = int(row - t * p.q_heads);
    int hi = p.b.num_seqs - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.b.cu_new + mid) <= t) lo = mid;
      else hi = mid - 1;
    }
  }
  const int64_t i = t - __ldg(p.b.cu_new + lo);
  const int64_t n_new = int64_t(__ldg(p.b.cu_new + lo + 1)) - __ldg(p.b.cu_new + lo);
  const bool tc = takes_tc(p, min(n_new, int64_t(p.max_q_len)), G);
  const int tile_rows = tc ? kTcRows : p.tile_rows, chunk = tc ? p.tc_chunk : p.chunk;
  const Rows s = sequence_rows(p, lo, (i * G + hq % G) / tile_rows * tile_rows, tile_rows, G);
  live = live && i >= 0 && i < s.q && s.end > chunk && (tc || !p.cluster);
  // every thread waits, also where there is nothing to do: this kernel must not end before the
  // attention does, or what comes after it could start beside that
  grid_dependency_wait();
  if (!live) return;
  const int n = int((s.end + chunk - 1) / chunk);
  const float* src = p.ws + row * p.ws_splits * (D + 4);
  // a running maximum, as in the chunks themselves
  float M = -INFINITY, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int c = kWide ? grp : 0; c < n; c += kWide ? kGroups : 1) {
    const float* x = src + int64_t(c) * (D + 4);
    const float m = x[D], l = x[D + 1];
    const float4 v = *reinterpret_cast<const float4*>(x + 4 * col);
    const float mn = fmaxf(M, m), mu = mn == -INFINITY ? 0.0f : mn;
    const float f = fast_exp2(m - mu), g = fast_exp2(M - mu);
    M = mn;
    L = L * g + l * f;
    acc.x = acc.x * g + v.x * f;
    acc.y = acc.y * g + v.y * f;
    acc.z = acc.z * g + v.z * f;
    acc.w = acc.w * g + v.w * f;
  }
  if constexpr (kWide) {
    __shared__ float s_m[kGroups], s_l[kGroups];
    __shared__ float4 s_o[kGroups][kCols];
    if (col == 0) {
      s_m[grp] = M;
      s_l[grp] = L;
    }
    s_o[grp][col] = acc;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < kGroups; ++k) M = fmaxf(M, s_m[k]);
    const float mu = M == -INFINITY ? 0.0f : M;
    L = 0.0f;
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float4 v = s_o[k][col];
      const float f = fast_exp2(s_m[k] - mu);
      L += s_l[k] * f;
      acc.x += v.x * f;
      acc.y += v.y * f;
      acc.z += v.z * f;
      acc.w += v.w * f;
    }
  }
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + 4 * col) =
      make_uint2(pack16(acc.x * inv, acc.y * inv, p.fp16), pack16(acc.z * inv, acc.w * inv, p.fp16));
  if (p.lse != nullptr && col == 0) p.lse[row] = L != 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int D, int NT, bool kOne>
cudaError_t launch_rows(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  using G_ = Geo<D, NT>;
  const uint64_t rows128 = uint64_t(p.c.num_pages) * p.c.kv_heads * p.c.page_size * D / 128;
  const int box = (p.c.page_size < G_::kTileKeys ? p.c.page_size : G_::kTileKeys) * D / 128;
  CUtensorMap map_k, map_v;
  if (!encode_bytes_2d(&map_k, p.c.k, rows128, 128, 128, uint32_t(box)) ||
      !encode_bytes_2d(&map_v, p.c.v, rows128, 128, 128, uint32_t(box)))
    return cudaErrorInvalidValue;
  const int pages = p.chunk / p.c.page_size + 1;
  const int smem = G_::kRing + int(sizeof(Shared)) + pages * 6 + 16 + 1024;
  static std::atomic<uint64_t> done{0};
  const int most = G_::kRing + int(sizeof(Shared)) + (kMaxChunkBytes / D / 16 + 1) * 6 + 16 + 1024;
  const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kv_attn_kernel<D, NT, kOne>), most);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(plan.row_tiles) * p.c.kv_heads * plan.splits * p.b.num_seqs;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (!p.cluster) {
    kv_attn_kernel<D, NT, kOne><<<unsigned(grid), kThreads, smem, stream>>>(map_k, map_v, p, plan.row_tiles);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(plan.splits);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attn_kernel<D, NT, kOne>, map_k, map_v, p, plan.row_tiles);
}

template <int D>
cudaError_t launch_attn(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  if (plan.row_tiles > 0) {
    cudaError_t e;
    if (p.max_q_len == 1)
      e = p.tile_rows == 8 ? launch_rows<D, 1, true>(p, plan, stream) : launch_rows<D, 2, true>(p, plan, stream);
    else
      e = p.tile_rows == 8 ? launch_rows<D, 1, false>(p, plan, stream) : launch_rows<D, 2, false>(p, plan, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.ws_splits > 1) {
    // launched with the attention kernel still running (its blocks wait for it to complete)
    // beside prompts that are not split, only the few rows of the other sequences can be
    const int few = plan.tc_row_tiles > 0 && plan.tc_splits == 1 ? plan.row_tiles * plan.tile_rows : 0;
    const int64_t rows = few > 0 ? int64_t(p.b.num_seqs) * p.c.kv_heads * few : p.T * p.q_heads;
    // a row each where there are many chunks: one sequence of 65536 33 us, 52 with four rows a CTA; but
    // with 4 chunks of 64 sequences (6000 tokens) 133 us, 137.5 with a row each
    const bool wide = p.ws_splits > 8;
    const int64_t blocks = wide ? rows : (rows + kThreads / (D / 4) - 1) / (kThreads / (D / 4));
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D, true>, p, few)
                : cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D, false>, p, few);
  }
  return cudaSuccess;
}

// Keys of a chunk where max_len keys are to be `n` chunks.
int chunk_for(int64_t max_len, int64_t n, int64_t least) {
  const int64_t chunk = ((max_len + n - 1) / n + 127) / 128 * 128, most = 1 << 24;
  return int(chunk < least ? least : (chunk > most ? most : chunk));
}

}  // namespace

KvAttnPlan plan_kv_attn(const fq_kv_cache& c, const fq_kv_batch& b, int64_t T, int q_heads, int max_q_len,
                        int64_t max_seq_len, int num_sms) {
  KvAttnPlan plan{};
  const int G = q_heads / c.kv_heads;
  const int64_t rows = int64_t(max_q_len) * G;  // of one sequence, at most
  // Above 64 rows the tensor-core kernel; there the two are about even (64 sequences of 512 keys, 64
  // rows: 81 us here and 75 there; 8 of 16384: 190 and 180). With 128 rows this one takes twice as
  // long (156 us for 78; 360 for 159), with 32 that one does (43 for 75; 109 for 206).
  plan.tc_rows = 64;
  const int64_t few = b.num_seqs == 1 && rows > plan.tc_rows ? 0 : (rows < plan.tc_rows ? rows : plan.tc_rows);
  if (few == 0) plan.tc_rows = 0;  // one sequence: whatever its length, one kernel
  // 8 rows where that is all: 64 sequences of 6000, 8 rows, 133 us, 160 in CTAs of 16 rows; 16 sequences
  // of 4000, 16 rows, 35 us, 42.5 in CTAs of 8, which read the cache twice
  plan.tile_rows = few <= 8 ? 8 : 16;
  plan.row_tiles = int((few + plan.tile_rows - 1) / plan.tile_rows);
  plan.splits = plan.tc_splits = 1;
  plan.chunk = plan.tc_chunk = 0x7FFFFF80;
  if (plan.row_tiles > 0) {
    const int64_t ctas = int64_t(b.num_seqs) * c.kv_heads * plan.row_tiles;
    // One wave of CTAs (three or two on an SM) where that takes chunks of at most 1 MB (keys and
    // values): not a CTA more, since a second wave of a few costs a whole one (16 sequences of 8000
    // tokens, 8 heads: 48 us with 384 CTAs, 62 with 512). Else chunks of 0.5 MB (16 rows: 1 MB), so
    // that a ragged batch ends evenly: 64 sequences of 500-16000 tokens 197 us with chunks of 2 MB,
    // 174 with 1, 169 with 0.5, 172 with 0.25, where starts and ends of CTAs (3 us) begin to show.
    const int64_t wave = int64_t(plan.tile_rows == 8 ? 3 : 2) * num_sms, n = wave / ctas;
    const int64_t most = kMaxChunkBytes / c.head_dim;
    plan.chunk = chunk_for(max_seq_len, n > 1 ? n : 1, 256);
    if (n < 1 || plan.chunk > most) plan.chunk = int(plan.tile_rows == 8 ? most / 2 : most);
    plan.splits = int((max_seq_len + plan.chunk - 1) / plan.chunk);
    // Joined in a cluster: no workspace and no second kernel (4 us of host time), a sequence
    // of 700 tokens 7.7 us for 8.4, of 1500 7.8 for 9.7. In one wave only, since a cluster
    // waits for room for all its CTAs: 16 sequences of 16000 in 512 CTAs 116 us for 107.
    plan.cluster = plan.splits > 1 && plan.splits <= kMaxCluster && ctas * plan.splits <= wave;
  }
  if (rows > plan.tc_rows) {
    plan.tc_row_tiles = int((rows + kTcRows - 1) / kTcRows);
    // about one wave of CTAs, not two (512 new tokens of 8192 83 us, 118 with twice as many chunks; 4
    // times 256 of 4096 77 and 130), of 1024 keys or more (1000 new of 4000, two heads: 35 us, 54 with
    // 2048; 16 times 64 of 2000 the same). The token rows bound the CTAs that have work, whatever the
    // longest sequence.
    const int64_t ctas = (T * G + kTcRows - 1) / kTcRows * c.kv_heads, n = num_sms / ctas;
    plan.tc_chunk = chunk_for(max_seq_len, n > 1 ? n : 1, 1024);
    plan.tc_splits = int((max_seq_len + plan.tc_chunk - 1) / plan.tc_chunk);
  }
  plan.ws_splits = !plan.cluster && plan.splits > plan.tc_splits ? plan.splits : plan.tc_splits;
  // (sizes that no memory holds: more than any workspace has, not a number that wrapped)
  const int64_t rows_bytes = T * q_heads * int64_t(c.head_dim + 4) * 4;
  plan.ws_bytes = plan.ws_splits <= 1 ? 0 : (rows_bytes > INT64_MAX / plan.ws_splits ? INT64_MAX : rows_bytes * plan.ws_splits);
  return plan;
}

cudaError_t launch_kv_attn(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  if (plan.tc_row_tiles > 0) {
    const cudaError_t e = launch_kv_attn_tc(p, plan, stream);
    if (e != cudaSuccess) return e;
  }
  return p.c.head_dim == 128 ? launch_attn<128>(p, plan, stream) : launch_attn<64>(p, plan, stream);
}

}  // namespace fq
