// Attention over the 8-bit paged cache: softmax(scale q k^T) v, for any number of new tokens.
//
// Rows are (new token, query head) pairs that share one key / value head, packed 16 at a time
// (row r of a sequence: token r / G, head r % G of the group, G = q_heads / kv_heads), so a
// decode step reads each cached byte once for the whole group. With few rows the kernel is
// bound by reading the cache: 2 D bytes a token and head.
//
// One CTA takes 16 rows and one chunk of keys; its four warps take tiles of 32 keys in turn,
// each through a ring of its own (TMA boxes of 128-byte rows, swizzled; no barrier between the
// warps), with a running maximum, sum and output of its own; they are joined through shared
// memory at the end. A sequence longer than one chunk is joined by a second kernel from partial
// results in the workspace.
//
// Numbers. A code is converted to fp16 with integer operations (E4M3 bits moved into the fp16
// fields give code * 2^-8, subnormals included; every bit pattern gives a finite number, so
// stale bytes behind the last token cannot put a NaN into the sum). A row of q is scaled by the
// power of two that brings its largest magnitude into [2^14, 2^15) and converted to fp16: exact
// but for elements 2^-29 below the largest. The products are then exact in the fp32 sums of
// mma.sync, and the powers of two (q row, page of k, 2^8) are applied to the score in float32.
// Probabilities are rounded to fp16 (2^-11) for the second product. The output accumulates in
// units of the page's own scale of v and moves to the next page's unit by a power of two, so
// that no page's scale has to fit beside another's in fp16: exponents lie in [-40, 40], so a
// unit changes by at most 2^80 and float32 holds all of it.
#include <cstdint>

#include "fq_kv_common.cuh"

namespace fq {
namespace {

using namespace ptx;
using namespace kv;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTileKeys = 32;   // keys of one warp's step
constexpr int kRowsTile = 16;   // rows of a CTA
constexpr int kMaxChunk = 8192; // keys of a chunk (its page numbers sit in shared memory)
enum : uint32_t { kStFull = 1u << 0 };

template <int D>
struct Geo {
  static constexpr int kTileBytes = kTileKeys * D;          // codes of K (or V) of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kOStride = D + 4;                    // floats per row of a warp's output
  static_assert(kWarps * kRowsTile * kOStride * 4 <= kRing, "outputs fit the ring");
};

struct Shared {
  uint64_t full[kWarps][8];
  float m[kWarps][kRowsTile], l[kWarps][kRowsTile];
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

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
kv_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const KvAttnParams p, const int row_tiles) {
  using G_ = Geo<D>;
  constexpr int kS = D / 16;      // k steps of q k^T
  constexpr int kN = D / 8;       // 8-column blocks of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared* sh = reinterpret_cast<Shared*>(smem + G_::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int ps = p.c.page_size, H = p.c.kv_heads, G = p.q_heads / H;

  int64_t idx = blockIdx.x;
  const int tile = int(idx % row_tiles);
  idx /= row_tiles;
  const int h = int(idx % H);
  idx /= H;
  const int split = int(idx % p.splits);
  const int b = int(idx / p.splits);

  const Rows s = sequence_rows(p, b, int64_t(tile) * kRowsTile, kRowsTile, G);
  if (tid == 0 && split == 0 && h == 0 && tile == 0 && p.status != nullptr && (!s.ok || s.n > p.max_q_len))
    atomicOr(p.status, FQ_KV_BAD_BATCH);
  const int row0 = tile * kRowsTile;
  const int rows = int(min(int64_t(kRowsTile), s.n * G - row0));
  if (rows <= 0 || takes_tc(p, s.n, G)) return;
  const int64_t c0 = int64_t(split) * p.chunk;  // first key of the chunk
  if (c0 >= s.end && split > 0) return;
  const int keys = int(min(int64_t(p.chunk), s.end - c0));
  const bool whole = s.end <= p.chunk;          // no other chunk: the result is final

  // ---- page numbers of the chunk, barriers ----
  // scales beside them: (k exponent, v exponent) as bytes; a page outside the cache is -1
  int* s_page = reinterpret_cast<int*>(sh + 1);
  uint16_t* s_scale = reinterpret_cast<uint16_t*>(s_page + (p.chunk + ps - 1) / ps);
  const int n_pages = (keys + ps - 1) / ps;
  if (tid < kWarps * G_::kStages) mbar_init(&sh->full[tid / G_::kStages][tid % G_::kStages], 1);
  if (tid == 0) sh->abort = 0;
  const int* table = p.b.page_table + int64_t(b) * p.b.table_width + c0 / ps;
  for (int i = tid; i < n_pages; i += kThreads) {
    int pg = __ldg(table + i);
    if (pg < 0 || int64_t(pg) >= p.c.num_pages) {
      pg = -1;
      if (p.status != nullptr) atomicOr(p.status, FQ_KV_BAD_BATCH);
    }
    s_page[i] = pg;
  }
  if (tid == 0) {
    fence_barrier_init();
    fence_proxy_async();
  }
  __syncthreads();

  const int n_tiles = (keys + kTileKeys - 1) / kTileKeys;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * G_::kStages * G_::kStageBytes);
  const int box = ps < kTileKeys ? ps : kTileKeys;  // keys of one TMA box
  // loads tile w of the chunk into a stage (one lane); boxes that start behind the last key, or
  // whose page is missing, are left out: their keys are masked
  auto issue = [&](int w, int stage) {
    uint64_t* bar = &sh->full[warp][stage];
    const uint32_t dst = ring + uint32_t(stage * G_::kStageBytes);
    uint32_t bytes = 0;
    for (int k = 0; k < kTileKeys && w * kTileKeys + k < keys; k += box)
      if (s_page[(w * kTileKeys + k) / ps] >= 0) bytes += uint32_t(2 * box * D);
    mbar_arrive_expect_tx(bar, bytes);
    for (int k = 0; k < kTileKeys && w * kTileKeys + k < keys; k += box) {
      const int at = w * kTileKeys + k;
      const int pg = s_page[at / ps];
      if (pg < 0) continue;
      const int row = int(((int64_t(pg) * H + h) * ps + at % ps) * D / 128);
      tma_load_2d(dst + uint32_t(k * D), &map_k, 0, row, bar);
      tma_load_2d(dst + uint32_t(G_::kTileBytes + k * D), &map_v, 0, row, bar);
    }
  };
  if (lane == 0)
    for (int st = 0; st < G_::kStages; ++st)
      if (warp + st * kWarps < n_tiles) issue(warp + st * kWarps, st);

  for (int i = tid; i < n_pages; i += kThreads) {
    const int pg = s_page[i];
    int ke = 0, ve = 0;
    if (pg >= 0) {
      ke = page_exp(__ldg(p.c.k_scale + int64_t(pg) * H + h));
      ve = page_exp(__ldg(p.c.v_scale + int64_t(pg) * H + h));
    }
    s_scale[i] = uint16_t((ke + 127) | ((ve + 127) << 8));
  }

  // ---- q: this thread's elements of rows g and g + 8, t4 * D/4 .. + D/4 ----
  uint32_t qf[kS][4];
  float rowf[2];
  int64_t vis[2];  // keys of the chunk that the row sees
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = row0 + g + 8 * hh;
    const bool live = g + 8 * hh < rows;
    float x[D / 4];
    float amax = 0.0f;
    const int64_t base = live ? (s.t_first + r / G) * p.q_stride + int64_t(h * G + r % G) * D + t4 * (D / 4) : 0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (live) w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + base) + c);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
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
      qf[st][hh] = h2(x[4 * st] * f, x[4 * st + 2] * f);          // k pairs as codes_lo gives them
      qf[st][2 + hh] = h2(x[4 * st + 1] * f, x[4 * st + 3] * f);  // and codes_hi
    }
    rowf[hh] = p.scale * kLog2e * exp2i(qe);
    int64_t v = s.len;
    if (p.causal) v = min(v, s.len - s.n + int64_t(r / G) + 1);
    vis[hh] = live ? v - c0 : 0;
  }
  __syncthreads();  // scales

  float o[kN][4];
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  int unit = 0;        // exponent of the output's current unit
  bool first_unit = true;
  bool ok = true;

  int stage = 0, phase = 0;
  for (int w = warp; w < n_tiles; w += kWarps) {
    ok = warp_wait(&sh->full[warp][stage], uint32_t(phase), &sh->abort, p.status, kStFull);
    if (!ok) break;
    const uint32_t kbase = ring + uint32_t(stage * G_::kStageBytes), vbase = kbase + G_::kTileBytes;
    const int k0 = w * kTileKeys;

    // ---- scores ----
    float sc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.0f;
      const int key = j * 8 + g;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 v = lds128(kbase + swz<D>(key, t4 * (D / 4) + c * 16));
        const uint32_t ww[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_f16(sc[j], qf[c * 4 + e], codes_lo(ww[e]), codes_hi(ww[e]));
      }
    }
    float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pg_i = min((k0 + j * 8) / ps, n_pages - 1);
      const bool there = s_page[pg_i] >= 0;
      const float pf = exp2i(int(s_scale[pg_i] & 0xFFu) - 127 + 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int hh = e >> 1;
        const int64_t key = k0 + j * 8 + 2 * t4 + (e & 1);
        const float v = sc[j][e] * (rowf[hh] * pf);
        sc[j][e] = there && key < vis[hh] ? v : -INFINITY;
        mt[hh] = fmaxf(mt[hh], sc[j][e]);
      }
    }
    float alpha[2], mu[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      mt[hh] = fmaxf(mt[hh], __shfl_xor_sync(0xffffffffu, mt[hh], 1));
      mt[hh] = fmaxf(mt[hh], __shfl_xor_sync(0xffffffffu, mt[hh], 2));
      const float mn = fmaxf(m[hh], mt[hh]);
      mu[hh] = mn == -INFINITY ? 0.0f : mn;  // a row that has seen nothing yet
      alpha[hh] = fast_exp2(m[hh] - mu[hh]);
      m[hh] = mn;
      l[hh] *= alpha[hh];
    }
    uint32_t pr[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const float a = fast_exp2(sc[j][2 * hh] - mu[hh]), c = fast_exp2(sc[j][2 * hh + 1] - mu[hh]);
        l[hh] += a + c;
        pr[j][hh] = h2(a, c);
      }
    }

    // ---- output ----
    float f0 = alpha[0], f1 = alpha[1];
#pragma unroll
    for (int st = 0; st < 2; ++st) {  // 16 keys each, within one page
      const int pg_i = min((k0 + st * 16) / ps, n_pages - 1);
      const int ev = int(s_scale[pg_i] >> 8) - 127;
      if (ev != unit) {
        if (!first_unit) {
          const float u = exp2i(unit - ev);
          f0 *= u;
          f1 *= u;
        }
        unit = ev;
      }
      first_unit = false;
      if (__any_sync(0xffffffffu, f0 != 1.0f || f1 != 1.0f)) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      f0 = f1 = 1.0f;
      const uint32_t a[4] = {pr[2 * st][0], pr[2 * st][1], pr[2 * st + 1][0], pr[2 * st + 1][1]};
      // this thread's keys 2 t4, + 1, + 8, + 9 and output columns g * D/8 .. + D/8
      const int key = st * 16 + 2 * t4;
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = vbase + swz<D>(key + (i & 1) + 8 * (i >> 1), g * (D / 8));
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
        // byte d of two keys side by side in the high bytes of two halves
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t sel = uint32_t(d << 4) | uint32_t((4 + d) << 12);
          const uint32_t b0 = codes_hi(__byte_perm(v[0][c], v[1][c], sel));
          const uint32_t b1 = codes_hi(__byte_perm(v[2][c], v[3][c], sel));
          mma_f16(o[c * 4 + d], a, b0, b1);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && w + G_::kStages * kWarps < n_tiles) issue(w + G_::kStages * kWarps, stage);
    if (++stage == G_::kStages) {
      stage = 0;
      phase ^= 1;
    }
  }

  // ---- join the warps ----
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
  }
  const float uf = exp2i(unit + 8);  // out of the page's unit (and the codes' 2^-8)
  __syncthreads();                   // every warp has left its ring
  float* so = reinterpret_cast<float*>(smem) + warp * kRowsTile * G_::kOStride;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    // block j's column n of this thread's fragment is output column n * D/8 + j
    so[g * G_::kOStride + (2 * t4) * (D / 8) + j] = o[j][0] * uf;
    so[g * G_::kOStride + (2 * t4 + 1) * (D / 8) + j] = o[j][1] * uf;
    so[(g + 8) * G_::kOStride + (2 * t4) * (D / 8) + j] = o[j][2] * uf;
    so[(g + 8) * G_::kOStride + (2 * t4 + 1) * (D / 8) + j] = o[j][3] * uf;
  }
  if (t4 == 0) {
    sh->m[warp][g] = m[0];
    sh->m[warp][g + 8] = m[1];
    sh->l[warp][g] = l[0];
    sh->l[warp][g + 8] = l[1];
  }
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&sh->abort)) return;
  constexpr int kPer = D / 8;  // columns of a thread: 8 threads per row
  const int r = tid >> 3, d0 = (tid & 7) * kPer;
  if (r >= rows) return;
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
  const int64_t row = (s.t_first + (row0 + r) / G) * p.q_heads + h * G + (row0 + r) % G;
  if (whole) {
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) w[e] = pack16(acc[2 * e] * inv, acc[2 * e + 1] * inv, p.fp16);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + d0);
#pragma unroll
    for (int e = 0; e < kPer / 8; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    if (p.lse != nullptr && (tid & 7) == 0) p.lse[row] = L > 0.0f ? (Mu + log2f(L)) * kLn2 : -INFINITY;
  } else {
    float* dst = p.ws + (row * p.ws_splits + split) * (D + 4);
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<float4*>(dst + d0 + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    if ((tid & 7) == 0) {
      dst[D] = M;
      dst[D + 1] = L;
    }
  }
}

// Joins the chunks of the rows that had more than one: a warp per row.
template <int D>
__global__ void __launch_bounds__(128)
kv_attn_join_kernel(const KvAttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= p.T * p.q_heads) return;
  const int64_t t = row / p.q_heads;
  const int hq = int(row % p.q_heads);
  int lo = 0, hi = p.b.num_seqs - 1;  // the last sequence that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.b.cu_new + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const int G = p.q_heads / p.c.kv_heads;
  const int64_t i = t - __ldg(p.b.cu_new + lo);
  const int64_t n_new = int64_t(__ldg(p.b.cu_new + lo + 1)) - __ldg(p.b.cu_new + lo);
  const bool tc = takes_tc(p, n_new, G);
  const int tile_rows = tc ? kTcRows : kRowsTile, chunk = tc ? p.tc_chunk : p.chunk;
  const Rows s = sequence_rows(p, lo, (i * G + hq % G) / tile_rows * tile_rows, tile_rows, G);
  if (i < 0 || i >= s.n || i >= p.max_q_len || s.end <= chunk) return;
  const int n = int((s.end + chunk - 1) / chunk);
  const float* src = p.ws + row * p.ws_splits * (D + 4);
  float M = -INFINITY;
  for (int c = lane; c < n; c += 32) M = fmaxf(M, src[int64_t(c) * (D + 4) + D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float Mu = M == -INFINITY ? 0.0f : M;
  constexpr int E = D / 32;
  float L = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int c = 0; c < n; ++c) {
    const float* x = src + int64_t(c) * (D + 4);
    const float f = fast_exp2(x[D] - Mu);
    L += x[D + 1] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += x[lane * E + e] * f;
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  uint16_t* dst = static_cast<uint16_t*>(p.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack16(acc[e] * inv, acc[e + 1] * inv, p.fp16);
  if (p.lse != nullptr && lane == 0) p.lse[row] = L > 0.0f ? (Mu + log2f(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_attn(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  if (plan.row_tiles > 0) {
    const uint64_t rows128 = uint64_t(p.c.num_pages) * p.c.kv_heads * p.c.page_size * D / 128;
    const int box = (p.c.page_size < kTileKeys ? p.c.page_size : kTileKeys) * D / 128;
    CUtensorMap map_k, map_v;
    if (!encode_bytes_2d(&map_k, p.c.k, rows128, 128, 128, uint32_t(box)) ||
        !encode_bytes_2d(&map_v, p.c.v, rows128, 128, 128, uint32_t(box)))
      return cudaErrorInvalidValue;
    const int pages = (p.chunk + p.c.page_size - 1) / p.c.page_size;
    const int smem = Geo<D>::kRing + int(sizeof(Shared)) + pages * 6 + 16 + 1024;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = int64_t(plan.row_tiles) * p.c.kv_heads * plan.splits * p.b.num_seqs;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    kv_attn_kernel<D><<<unsigned(grid), kThreads, smem, stream>>>(map_k, map_v, p, plan.row_tiles);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.ws_splits > 1) {
    const int64_t blocks = (p.T * p.q_heads + 3) / 4;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    kv_attn_join_kernel<D><<<unsigned(blocks), 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

// Chunk of keys for `ctas` CTAs of one chunk each over max_len keys: chunks until there are
// `want` CTAs, of at least `least` keys.
int64_t chunk_for(int64_t max_len, int64_t ctas, int64_t want, int64_t least, int64_t most) {
  const int64_t n = (want + ctas - 1) / ctas;
  int64_t chunk = (max_len + n - 1) / n;
  chunk = (chunk + 127) / 128 * 128;
  return chunk < least ? least : (chunk > most ? most : chunk);
}

}  // namespace

KvAttnPlan plan_kv_attn(const fq_kv_cache& c, const fq_kv_batch& b, int64_t T, int q_heads, int max_q_len,
                        int64_t max_seq_len, int num_sms) {
  KvAttnPlan plan{};
  const int G = q_heads / c.kv_heads;
  const int64_t rows = int64_t(max_q_len) * G;  // of one sequence, at most
  plan.tc_rows = 64;
  const int64_t few = b.num_seqs == 1 && rows > plan.tc_rows ? 0 : (rows < plan.tc_rows ? rows : plan.tc_rows);
  if (few == 0) plan.tc_rows = 0;  // one sequence: whatever its length, one kernel
  plan.row_tiles = int((few + kRowsTile - 1) / kRowsTile);
  plan.splits = plan.tc_splits = 1;
  plan.chunk = plan.tc_chunk = 0x7FFFFF80;
  if (plan.row_tiles > 0) {
    const int64_t ctas = int64_t(b.num_seqs) * c.kv_heads * plan.row_tiles;
    plan.chunk = int(chunk_for(max_seq_len, ctas, 4 * int64_t(num_sms), 256, kMaxChunk));
    plan.splits = int((max_seq_len + plan.chunk - 1) / plan.chunk);
  }
  if (rows > plan.tc_rows) {
    plan.tc_row_tiles = int((rows + kTcRows - 1) / kTcRows);
    // the token rows bound the CTAs that have work, whatever the longest sequence
    const int64_t tiles = (T * G + kTcRows - 1) / kTcRows;
    plan.tc_chunk = int(chunk_for(max_seq_len, tiles * c.kv_heads, 2 * int64_t(num_sms), 1024, 1 << 24));
    plan.tc_splits = int((max_seq_len + plan.tc_chunk - 1) / plan.tc_chunk);
  }
  const int64_t slots = plan.splits > plan.tc_splits ? plan.splits : plan.tc_splits;
  plan.ws_bytes = slots > 1 ? T * q_heads * slots * int64_t(c.head_dim + 4) * 4 : 0;
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
