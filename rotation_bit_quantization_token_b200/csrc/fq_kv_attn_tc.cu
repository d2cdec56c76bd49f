// Attention over the 8-bit paged cache on the tensor cores (tcgen05): sequences with many rows,
// that is prompts and chunks of prompts.
//
// A row is a (new token, query head of the group) pair; one CTA takes two tiles of 128 rows of
// one sequence and key / value head, and a chunk of keys, 128 keys at a time:
//     S = Q K^T   (M = 128 rows, N = 128 keys, K = D; Q and K fp16 in shared memory)
//     P = exp2(S c - m)                        (registers, one thread per row)
//     O += P V    (M = 128 rows, N = D, K = 128 keys; P fp16 in TMEM, V fp16 in shared memory)
// The two row tiles take turns: while one's softmax runs, the tensor cores do the other's products.
// Both share every converted tile of K and V.
//
// Codes reach the MMAs as fp16, converted by a warpgroup that also multiplies by the page's power of
// two in the step's units, exactly: code * 2^e is an fp16 number for e in [-15, 7]. Where all pages of
// the CTA's keys lie within 2^15 of one another (their values; their keys), the largest one's are the
// units of every step. Else each step has its own: keys in units of its largest page, undone by the
// factor c of its scores (beside the softmax scale, log2 e and the q row's exponent); values in units
// that last as long as pages stay within [-15, 0] of it, and when they change, O is multiplied by the
// power of two between them. Pages of one step that lie further apart are taken in steps of their own,
// each over the same 128 keys with the other pages left out. (The producer is short of issue slots
// beside the softmax: with the units of every step worked out in every CTA the 8192-token prompt took
// 607 us, now 551.)
//
// Softmax. A thread owns one row (its TMEM lane), so no exchange is needed. What the exponents are taken
// against is only raised when a probability would pass 2^15.9 (within fp16); O and the sum are rescaled
// then. It is set so that the largest score has probability 2^12: the rounding to fp16 is 2^-11 of a
// probability, or 2^-37 of the row's largest for those below 2^-26 of it. (8192-token prompt: 552 us with 2^0
// for 2^12, where probabilities below 2^-14 of the largest lose bits and below 2^-25 vanish from O but not
// from the sum; 562 with 2^8, 573 with 2^14.)
//
// Roles, 512 threads: warp 0 MMA issuer (owns TMEM), 1 TMA producer, 4-7 and 8-11 softmax of row
// tile 0 and 1 (its Q before, its output after), 12-15 converters. The issuer comes first and waits as
// seldom as it can: its barrier operations queue behind the exponentials of its scheduler's softmax
// warps (about 200 clocks each), and a step of one row tile is a chain of softmax (2000 clocks), its
// hand-over, P V and S (1024), and their hand-over back; the two row tiles' chains overlap, about 2.2 us
// a step. TMEM: O 2 x D columns, S 2 x 128 columns (P overwrites the first half of its S).
// Every wait is bounded. A causal prompt of 8192 tokens, 32 heads of 128 on 8: 569 us, 0.97 PFLOP/s.
#include <cstdint>

#include "fq_kv_common.cuh"

namespace fq {
namespace {

using namespace ptx;
using namespace kv;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kKeys = 128;  // keys of a step
constexpr int kSorted = 256;  // sequences that are taken in order of length
constexpr int kWarpMma = 0, kWarpProducer = 1, kWarpSoft0 = 4, kWarpConv0 = 12;
// Register split (setmaxnreg): launched at 128 per thread; 2 softmax warpgroups, the converters, the rest
// (200, 72 and 40: 559 us for 551)
constexpr int kRegsLaunch = 128, kRegsSoftmax = 192, kRegsConv = 72, kRegsLow = 56;
static_assert(128 * (2 * kRegsSoftmax + kRegsConv + kRegsLow) <= kThreads * kRegsLaunch, "register split");

enum : uint32_t {
  kStRawFull = 1u << 0, kStRawEmpty = 1u << 1, kStKFull = 1u << 2, kStVFull = 1u << 3, kStTEmpty = 1u << 4,
    kStSFull = 1u << 6, kStPFull = 1u << 7, kStOFull = 1u << 9, kStDrain = 1u << 10
};

constexpr uint32_t kAllThere = (1u << (kKeys / 16)) - 1u;  // a step with all its pages
constexpr uint32_t kChange = 1u << 31, kLast = 1u << 30;
constexpr int kNoPage = -1000;  // no exponent
// Probabilities are taken times 2^kBase for a row's largest score when its reference was set, and the
// reference is set anew when one passes 2^kMost (fp16 ends at 2^16)
constexpr float kBase = 12.0f, kMost = 15.9f;
constexpr int kFarExp = 26;  // see units_of
// Scores beside which an exponent is lost: from 2^27 on, float32 has steps of 16 and more, which x c - m does
// not resolve (its product is not rounded). A row whose largest score is as large is computed in units of
// 2^k, in which it is below 2^27: scores that differ by a step of float32 still differ by 8 then, so that one takes
// all of the probability, or those that are equal share it.
__device__ __forceinline__ int units_of(float top) {  // k
  return max(0, int((__float_as_uint(top) >> 23) & 0xFFu) - 127 - kFarExp);
}

template <int D>
struct Geo {
  static constexpr int kQBytes = 128 * D * 2;               // one row tile of Q
  static constexpr int kTile = kKeys * D * 2;               // a converted tile of K or V
  static constexpr int kRaw = kKeys * D;                    // its codes
  static constexpr int kTiles = 3;                          // ring of converted tiles, K and V in turn
  static constexpr int kRaws = 4;                           // ring of code tiles
  static constexpr int kOffTile = 2 * kQBytes;
  static constexpr int kOffRaw = kOffTile + kTiles * kTile;
  static constexpr int kOffBars = kOffRaw + kRaws * kRaw;
  static constexpr int kSmem = kOffBars + 2048 + 1024 /*alignment*/;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColO = 0, kColS = 2 * D, kCols = 512;
  static_assert(kColS + 256 <= kCols, "TMEM");
};

// What the producer tells about a step that differs from the one before in more than its pages.
struct __align__(16) Step {
  int first;       // first key (of the chunk); else 128 further on
  float k_factor;  // 2^(exponent of the keys' unit - 6)
  int v_unit;      // exponent of the values' unit
};

struct Bars {
  // unit u = 2j is K of step j, u = 2j + 1 V of step j
  uint64_t raw_full[4], raw_empty[4];  // codes of unit u, slot u % 4
  uint64_t t_full[3], t_empty[3];      // converted tile of unit u, slot u % 3
  uint64_t s_full[2], p_full[2];     // row tile
  uint64_t o_full[2];                // row tile: O complete
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int4 range[8];                     // largest exponent and least (negated) of the pages' keys, and of their values, by scanning warp
  int8_t q_exp[kTcRows];   // exponents of Q's rows
  int sorted;
  // per step (mod 16; the producer is at most 4 + 3 steps ahead): the pages that are there, one bit per 16
  // keys, kChange where the step's other properties are to be read, kLast in the last step
  uint32_t valid[16];
  Step step[16];
  int8_t expo[4][8];       // per raw slot: exponent of each 16 keys in the step's units
  int nan_from[128];       // per column: see hide_nans
  int nans;                // whether there is one
};
static_assert(sizeof(Bars) <= 2048, "barrier block");

// One row tile's product under one election, the whole warp running the same code: descriptors then
// stay in uniform registers. (A leader branch with one instruction per MMA took about 110 clocks
// to issue each, twice what a 128 x 128 x 16 product needs.)
//
// S = Q K^T: D / 16 K steps, 32 bytes apart inside a 128-byte atom, atoms 128 rows of 128 bytes
// apart (2 and 1024 in the descriptors' 16-byte units); the first overwrites S.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred f, t, e;\n\t.reg .b32 r;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 f, %0, %0;\n\tsetp.eq.b32 t, %0, %0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
  if constexpr (D == 128)
    asm volatile(
        "{\n\t.reg .pred t, e;\n\t.reg .b32 r;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.eq.b32 t, %0, %0;\n\t"
        "add.s64 a0, %1, 1024;\n\tadd.s64 a1, %1, 1026;\n\tadd.s64 a2, %1, 1028;\n\tadd.s64 a3, %1, 1030;\n\t"
        "add.s64 b0, %2, 1024;\n\tadd.s64 b1, %2, 1026;\n\tadd.s64 b2, %2, 1028;\n\tadd.s64 b3, %2, 1030;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
}
// O += P V for kSteps * 16 keys (8 columns of P and 2048 bytes of V each); acc = 0: the first overwrites.
template <int kSteps>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred f, t, e;\n\t.reg .b32 r, a1;\n\t.reg .b64 b1;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
  if constexpr (kSteps > 2) mma_values<kSteps - 2>(d, a + 16, b + 256, idesc, 1u);
}
__device__ __forceinline__ void commit_e(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
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
// Four codes as fp16 (the codes' values), in order.
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t* y) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(y[0]), "=r"(y[1])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The scale bytes (as page_exp allows them) of the pages of a step's eight times 16 keys.
struct Pages {
  uint32_t k[2], v[2];
};
constexpr int kSpan = 15;  // exponents of a step's pages differ by this at most
__device__ __forceinline__ uint32_t bytes_of(uint32_t bits) {  // 0xFF for each of four bits
  return ((bits * 0x00204081u) & 0x01010101u) * 0xFFu;
}
__device__ __forceinline__ uint32_t top_byte(const uint32_t* w, uint32_t mask) {
  uint32_t x = __vmaxu4(w[0] & bytes_of(mask & 15u), w[1] & bytes_of(mask >> 4));
  x = __vmaxu4(x, x >> 16);
  return __vmaxu4(x, x >> 8) & 0xFFu;
}
__device__ __forceinline__ uint32_t least_byte(const uint32_t* w, uint32_t mask) {
  uint32_t x = __vminu4(w[0] | ~bytes_of(mask & 15u), w[1] | ~bytes_of(mask >> 4));
  x = __vminu4(x, x >> 16);
  return __vminu4(x, x >> 8) & 0xFFu;
}
// Which of the pages `left` (a bit each, not empty) a step takes: all of them where they lie within
// kSpan of one another, else the first and those within kSpan / 2 of it.
__device__ __forceinline__ uint32_t next_pages(const Pages& g, uint32_t left) {
  if (int(top_byte(g.k, left) - least_byte(g.k, left)) <= kSpan && int(top_byte(g.v, left) - least_byte(g.v, left)) <= kSpan)
    return left;
  const uint32_t first = left & (0u - left);
  const uint32_t k0 = top_byte(g.k, first) * 0x01010101u, v0 = top_byte(g.v, first) * 0x01010101u;
  uint32_t take = 0u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    constexpr uint32_t kNear = uint32_t(kSpan / 2) * 0x01010101u;
    uint32_t near = __vcmpleu4(__vabsdiffu4(g.k[i], k0), kNear) & __vcmpleu4(__vabsdiffu4(g.v[i], v0), kNear) & 0x08040201u;
    near |= near >> 16;
    near |= near >> 8;
    take |= (near & 15u) << (4 * i);
  }
  return take & left;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D, bool kF16>
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

  grid_dependency_launch();
  // heads, then chunks, then row tiles from the last (longest) to the first, then sequences from the
  // longest to the shortest (up to kSorted of them): the work that starts last is short, and the launch
  // ends evenly
  unsigned idx = blockIdx.x;
  const int h = int(idx % unsigned(H));
  idx /= unsigned(H);
  const int split = int(idx % unsigned(p.tc_splits));
  idx /= unsigned(p.tc_splits);
  const int tile = row_tiles - 1 - int(idx % unsigned(row_tiles));
  int b = int(idx / unsigned(row_tiles));
  if (p.b.num_seqs > 1 && p.b.num_seqs <= kSorted) {
    // the sequence of rank b: each of the first threads finds the rank of its own
    int* lens = reinterpret_cast<int*>(smem);  // (Q comes here later)
    if (tid < p.b.num_seqs) lens[tid] = __ldg(p.b.seq_lens + tid);
    __syncthreads();
    if (tid < p.b.num_seqs) {
      const int mine = lens[tid];
      int rank = 0;
      for (int i = 0; i < p.b.num_seqs; ++i) rank += lens[i] > mine || (lens[i] == mine && i < tid);
      if (rank == b) bars->sorted = tid;
    }
    __syncthreads();
    b = bars->sorted;
  }

  const int64_t row0 = int64_t(tile) * kTcRows;
  const Rows s = sequence_rows(p, b, row0, kTcRows, G);
  if (tid == 0 && split == 0 && h == 0 && tile == 0 && p.status != nullptr && (!s.ok || s.n > p.max_q_len))
    atomicOr(p.status, FQ_KV_BAD_BATCH);
  const int rows = int(min(int64_t(kTcRows), s.q * G - row0));
  if (rows <= 0 || !takes_tc(p, s.q, G)) return;
  const int64_t c0 = int64_t(split) * p.tc_chunk;
  if (c0 >= s.end && split > 0) return;
  const int keys = int(min(int64_t(p.tc_chunk), s.end - c0));
  const bool whole = s.end <= p.tc_chunk;
  // row r of the CTA: token tok0 + (rem0 + r) / G of the array, head (rem0 + r) % G of the group (a
  // row's own division is 32-bit)
  const int64_t i0 = quotient(row0, G);
  const unsigned rem0 = unsigned(row0 - i0 * G), Gu = unsigned(G);
  const int64_t tok0 = s.t_first + i0;
  const int n_windows = (keys + kKeys - 1) / kKeys;  // of 128 keys
  const int n_tiles = rows > 128 ? 2 : 1;  // row tiles with rows
  const int ps_log = 31 - __clz(ps);
  const int* table = p.b.page_table + int64_t(b) * p.b.table_width + (c0 >> ps_log);
  const int n_pages = (keys + ps - 1) >> ps_log;

  // The beginning of a CTA, by parts that run at the same time (11000 clocks to the first softmax, 13000
  // one after the other; an average CTA of an 8192-token prompt takes 145000): the producer sets up the
  // mbarriers and starts loading, warp 0 allocates TMEM, the softmax warps bring Q, the others count the
  // steps.
  if (warp == kWarpProducer && lane == 0) {
    for (int i = 0; i < G_::kRaws; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], 4);
    }
    for (int i = 0; i < G_::kTiles; ++i) {
      mbar_init(&bars->t_full[i], 4);
      mbar_init(&bars->t_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->o_full[i], 1);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) tmem_alloc(&bars->tmem_base, G_::kCols);
  if (warp >= kWarpConv0) {
    bars->nan_from[tid - kWarpConv0 * 32] = kNoNan;
    bars->nans = 0;
  }
  // ---- Q: kLpr lanes load a row, eight elements each; a softmax warp its own 32 rows ----
  constexpr int kLpr = D / 8, kRpi = 32 / kLpr;  // lanes per row, rows per instruction
  constexpr int kRowIter = 32 / kRpi;
  const int c8 = lane % kLpr, sub = lane / kLpr;
  int64_t my_row = 0;  // (token, head) index of this thread's row in q and out
  if (warp >= kWarpSoft0 && warp < kWarpSoft0 + 4 * n_tiles) {
    // (rows that are not there read the last one: loads under a condition were waited for one by one)
    const unsigned r = rem0 + unsigned(min(tid - kWarpSoft0 * 32, rows - 1)), ti = r / Gu, hi = r - ti * Gu;
    my_row = (tok0 + ti) * p.q_heads + h * G + int(hi);
    const uint16_t* mine = static_cast<const uint16_t*>(p.q) + (tok0 + ti) * p.q_stride + int64_t(h * G + int(hi)) * D;
    uint4 qv[kRowIter];
#pragma unroll
    for (int i = 0; i < kRowIter; ++i) {
      const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), i * kRpi + sub);
      qv[i] = __ldg(reinterpret_cast<const uint4*>(from) + c8);
    }
    // the sign of the scale goes to Q (c stays positive, so a row's largest S is its largest
    // score); a zero scale makes Q zero
    const float sign = p.scale == 0.0f ? 0.0f : (p.scale < 0.0f ? -1.0f : 1.0f);
    // eight rows' maxima together (their shuffles overlap; with all of them registers run out)
#pragma unroll
    for (int i0 = 0; i0 < kRowIter; i0 += 8) {
      uint32_t top[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;  // magnitudes compare as their bits do
        const uint4& x = qv[i0 + i];
        top[i] = __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
      }
#pragma unroll
      for (int o = kLpr / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (warp - kWarpSoft0) * 32 + (i0 + i) * kRpi + sub;
        const uint4& x = qv[i0 + i];
        const float2 x0 = unpack16(x.x, kF16), x1 = unpack16(x.y, kF16), x2 = unpack16(x.z, kF16), x3 = unpack16(x.w, kF16);
        const int qe = row_exponent(unpack16(max(top[i] & 0xFFFFu, top[i] >> 16), kF16).x);
        const float f = r < rows ? sign * exp2i(-qe) : 0.0f;
        const uint32_t dst = sbase + uint32_t((r >> 7) * G_::kQBytes + (c8 >> 3) * 16384 + (r & 127) * 128);
        sts128(dst + uint32_t(((c8 & 7) ^ (r & 7)) << 4), h2(x0.x * f, x0.y * f), h2(x1.x * f, x1.y * f),
               h2(x2.x * f, x2.y * f), h2(x3.x * f, x3.y * f));
        if (c8 == 0) bars->q_exp[r] = int8_t(qe);
      }
    }
    fence_proxy_async();
  }

  // ---- the range of the page exponents, four pages of a thread at a time ----
  constexpr int kScanWarps = kWarps - 9;  // all but the producer and the softmax
  static_assert(kWarpMma == 0 && kWarpProducer == 1 && kWarpSoft0 == 4 && kWarpConv0 == 12, "warps 0, 2, 3 and 12-15 scan");
  const int scan = warp == 0 ? 0 : (warp == 2 || warp == 3 ? warp - 1 : (warp >= kWarpConv0 ? warp - 9 : -1));
  if (scan >= 0) {
    int kt = kNoPage, kl = -kNoPage, vt = kNoPage, vl = -kNoPage;  // largest and least of keys and values
    for (int i = scan * 32 + lane; i < n_pages; i += 4 * 32 * kScanWarps) {
      int pg[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pg[e] = __ldg(table + min(i + e * 32 * kScanWarps, n_pages - 1));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool there = pg[e] >= 0 && int64_t(pg[e]) < p.c.num_pages;
        const int64_t at = int64_t(there ? pg[e] : 0) * H + h;
        const int ke = page_exp(__ldg(p.c.k_scale + at)), ve = page_exp(__ldg(p.c.v_scale + at));
        if (there) {
          kt = max(kt, ke);
          kl = min(kl, ke);
          vt = max(vt, ve);
          vl = min(vl, ve);
        } else if (p.status != nullptr) {
          atomicOr(p.status, FQ_KV_BAD_BATCH);
        }
      }
    }
    kt = __reduce_max_sync(0xffffffffu, kt);
    kl = __reduce_min_sync(0xffffffffu, kl);
    vt = __reduce_max_sync(0xffffffffu, vt);
    vl = __reduce_min_sync(0xffffffffu, vl);
    if (lane == 0) bars->range[scan] = make_int4(kt, -kl, vt, -vl);
  }
  // Barrier 1: the range and mbarriers are there (the converters and the producer, which has
  // asked for the first 128 keys' codes by then, wait for no more); barrier 2: Q and TMEM too.
  constexpr int kMeetScan = 1, kMeetAll = 2;
  uint32_t tmem = 0;
  tc_fence_before();
  __syncwarp();
  if (warp >= kWarpConv0) {
    named_bar(kMeetScan, 32 * (kScanWarps + 1));
    named_bar_arrive(kMeetAll, kThreads);
  } else {
    if (scan >= 0) named_bar_arrive(kMeetScan, 32 * (kScanWarps + 1));
    if (warp == kWarpMma || warp >= kWarpSoft0) named_bar(kMeetAll, kThreads);
    else named_bar_arrive(kMeetAll, kThreads);
  }
  tc_fence_after();
  if (warp == kWarpMma || warp >= kWarpSoft0) {
    tmem = bars->tmem_base;
  }
  int* abort = &bars->abort;

  if (warp == kWarpProducer) {
    // ---------------- codes and page factors ----------------
    // Lane i < 8 looks after keys 16 i .. 16 i + 15 of every step: their page (two steps ahead)
    // and its scale bytes (one step ahead), so no load is waited for where it is used. The lane
    // whose keys begin a TMA box issues the box.
    setmaxnreg_dec<kRegsLow>();
    const int box = ps < kKeys ? ps : kKeys;
    auto page_of = [&](int w) {  // page of this lane's keys among 128, -1: none
      const int key = w * kKeys + lane * 16;
      if (lane >= kKeys / 16 || w >= n_windows || key >= keys) return -1;
      const int pg = __ldg(table + (key >> ps_log));
      return pg >= 0 && int64_t(pg) < p.c.num_pages ? pg : -1;
    };
    auto bytes_of_page = [&](int pg) {
      if (pg < 0) return 0u;
      return uint32_t(__ldg(p.c.k_scale + int64_t(pg) * H + h)) | (uint32_t(__ldg(p.c.v_scale + int64_t(pg) * H + h)) << 8);
    };
    int pg0 = page_of(0), pg1 = page_of(1);
    auto row_of = [&](int pg, int w) {  // of the tensor maps
      return int(((int64_t(max(pg, 0)) * H + h) * ps + ((w * kKeys + lane * 16) & (ps - 1))) * D / 128);
    };
    auto ask = [&](int kv, int row, int slot) {
      tma_load_2d(sbase + uint32_t(G_::kOffRaw + slot * G_::kRaw + lane * 16 * D), kv == 0 ? &map_k : &map_v, 0, row,
                  &bars->raw_full[slot]);
    };
    const bool box_begins = lane < kKeys / 16 && (lane * 16) % box == 0;
    // the first two steps are asked for at once (where such a step takes only some of the pages, the
    // others' codes are zeroed)
    const int n_early = min(n_windows, 2);
    for (int w = 0; w < n_early; ++w) {
      const bool begins = box_begins && (w == 0 ? pg0 : pg1) >= 0;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, begins));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (lane == 0) mbar_expect_tx(&bars->raw_full[2 * w + kv], boxes * uint32_t(box * D));
        __syncwarp();
        if (begins) ask(kv, row_of(w == 0 ? pg0 : pg1, w), 2 * w + kv);
      }
    }
    uint32_t by0 = bytes_of_page(pg0);
    named_bar(kMeetScan, 32 * (kScanWarps + 1));
    const int4 r = bars->range[min(lane, kScanWarps - 1)];
    const int kt = __reduce_max_sync(0xffffffffu, r.x), kl = -__reduce_max_sync(0xffffffffu, r.y);
    const int vt = __reduce_max_sync(0xffffffffu, r.z), vl = -__reduce_max_sync(0xffffffffu, r.w);
    const bool apart = kt - kl > kSpan || vt - vl > kSpan;
    bool ok = true;
    int issued = 2 * n_early;  // units
    int j = 0;                 // step
    int k_unit = max(kt, kPageExpMin), v_unit = max(vt, kPageExpMin);  // exponents of the keys' and values' units
    // Step j: the pages `take` of keys w * 128 .. , this lane's with tensor map row `row` and exponents ke, ve.
    auto step = [&](uint32_t take, int w, int row, int ke, int ve, bool change, bool last) {
      const bool in = ((take >> lane) & 1u) != 0u;
#pragma unroll
      for (int kv = 0; ok && kv < 2; ++kv) {
        const int u = 2 * j + kv, slot = u % G_::kRaws;
        ok = u < G_::kRaws || warp_wait(&bars->raw_empty[slot], (u / G_::kRaws - 1) & 1, abort, p.status, kStRawEmpty);
        if (!ok) break;
        if (lane < kKeys / 16) bars->expo[slot][lane] = int8_t(!in ? 0 : (kv == 0 ? ke - k_unit + 6 : ve - v_unit));
        if (kv == 0 && lane == 0) {
          bars->valid[j & 15] = take | (change ? kChange : 0u) | (last ? kLast : 0u);
          if (change) bars->step[j & 15] = Step{w * kKeys, exp2i(k_unit - 6), v_unit};
        }
        __syncwarp();
        if (j < n_early) {  // asked for above
          if (lane == 0) mbar_arrive(&bars->raw_full[slot]);
          continue;
        }
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, in && box_begins));
        if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[slot], boxes * uint32_t(box * D));
        __syncwarp();
        if (in && box_begins) ask(kv, row, slot);
        issued = u + 1;
      }
      ++j;
    };
    if (!apart) {
      for (int w = 0; ok && w < n_windows; ++w) {
        const int pg2 = page_of(w + 2);
        const uint32_t by1 = bytes_of_page(pg1);
        step(__ballot_sync(0xffffffffu, pg0 >= 0), w, row_of(pg0, w), page_exp(by0 & 0xFFu), page_exp(by0 >> 8), w == 0,
             w + 1 == n_windows);
        pg0 = pg1;
        pg1 = pg2;
        by0 = by1;
      }
    } else {
      // first a step for each 128 keys, then those of the pages that were left out
      bool have_unit = false;
      int behind = 0;  // times 128 keys with such pages
#pragma unroll 1
      for (int pass = 0; pass < 2 && (pass == 0 || behind > 0); ++pass) {
#pragma unroll 1
        for (int w = 0; ok && w < n_windows; ++w) {
          pg0 = page_of(w);
          by0 = bytes_of_page(pg0);
          const int ke = page_exp(by0 & 0xFFu), ve = page_exp(by0 >> 8);
          Pages g;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool mine = (lane >> 2) == i;
            g.k[i] = __reduce_or_sync(0xffffffffu, mine ? uint32_t(ke + 127) << (8 * (lane & 3)) : 0u);
            g.v[i] = __reduce_or_sync(0xffffffffu, mine ? uint32_t(ve + 127) << (8 * (lane & 3)) : 0u);
          }
          uint32_t left = __ballot_sync(0xffffffffu, pg0 >= 0);
          uint32_t take = left != 0u ? next_pages(g, left) : 0u;
          if (left != take) behind += pass == 0 ? 1 : -1;
          if (pass == 1) left &= ~take;
          while (ok && (pass == 0 || left != 0u)) {
            if (pass == 1) take = next_pages(g, left);
            if (take != 0u) {
              k_unit = int(top_byte(g.k, take)) - 127;
              const int hi = int(top_byte(g.v, take)) - 127, lo = int(least_byte(g.v, take)) - 127;
              // a new unit leaves room above and below, so that neighbouring pages seldom need another
              if (!have_unit || hi > v_unit || lo < v_unit - kSpan) v_unit = hi + min(kSpan / 3, kSpan - (hi - lo));
              have_unit = true;
            }
            left &= ~take;
            step(take, w, row_of(pg0, w), ke, ve, true, behind == 0 && (pass == 0 ? w + 1 == n_windows : left == 0u));
            if (pass == 0) break;
          }
        }
      }
    }
    // the last copies have landed before the CTA may exit (the converters wait for each of them;
    // after an abort they may have left)
    if (!ok && lane == 0) {
      for (int u = max(issued - G_::kRaws, 0); u < issued; ++u) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&bars->raw_full[u % G_::kRaws]), (u / G_::kRaws) & 1) &&
               globaltimer() - t0 < kTimeoutNs / 4) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---------------- MMA issuer ----------------
    // Row tile 0 before row tile 1 in every step: that keeps the two half a step apart. (One issuer
    // for each let them fall into step, both in their softmax and then both waiting for the tensor
    // cores: 5400 clocks a step.)
    setmaxnreg_dec<kRegsLow>();
    constexpr uint32_t kIdS = (1u << 4) | (uint32_t(kKeys >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) /*V is MN-major*/ | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    auto wait_tile = [&](int u, uint32_t code) {
      return warp_wait(&bars->t_full[u % G_::kTiles], (u / G_::kTiles) & 1, abort, p.status, code);
    };
    auto scores = [&](int w, int j) {
      const int slot = 2 * j % G_::kTiles;
      mma_scores<D>(tmem + G_::kColS + uint32_t(w * 128), sw128_desc(sbase + uint32_t(w * G_::kQBytes)),
                    sw128_desc(sbase + uint32_t(G_::kOffTile + slot * G_::kTile)), kIdS);
      commit_e(&bars->s_full[w]);
      if (w == n_tiles - 1) commit_e(&bars->t_empty[slot]);
    };
    bool ok = wait_tile(0, kStKFull);
    if (ok) {
      tc_fence_after();
      for (int w = 0; w < n_tiles; ++w) scores(w, 0);
    }
    // P V of step j, then the row tile's next scores, which overwrite P
    bool last = !ok || (bars->valid[0] & kLast) != 0u;
    for (int j = 0, end = 0; ok && !end; ++j) {
      const int slot = (2 * j + 1) % G_::kTiles;
      const uint64_t v = desc_lbo(sbase + uint32_t(G_::kOffTile + slot * G_::kTile), kKeys * 128);
      // K of the next step, whose conversion follows V's of this one (or V alone in the last step)
      ok = wait_tile(last ? 2 * j + 1 : 2 * j + 2, last ? kStVFull : kStKFull);
      end = last;
      const uint32_t next = last ? 0u : bars->valid[(j + 1) & 15];
      for (int w = 0; ok && w < n_tiles; ++w) {
        const uint32_t t_o = tmem + G_::kColO + uint32_t(w * D), t_p = tmem + G_::kColS + uint32_t(w * 128);
        ok = warp_wait(&bars->p_full[w], j & 1, abort, p.status, kStPFull);
        if (!ok) break;
        tc_fence_after();
        mma_values<8>(t_o, t_p, v, kIdO, j > 0 ? 1u : 0u);
        if (w == n_tiles - 1) commit_e(&bars->t_empty[slot]);
        if (!last) {
          scores(w, j + 1);
        } else {
          commit_e(&bars->o_full[w]);
        }
      }
      last = (next & kLast) != 0u;
    }
    // every MMA issued here has completed before TMEM is released
    commit_e(&bars->mma_done);
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
    constexpr int kBatch = kIter < 4 ? kIter : 4;
    const int key0 = cw * 8 + (lane & 7), ch0 = lane >> 3;
    // the first 128 keys with some that the first row does not see
    const int64_t all_see = p.causal ? s.len - s.n + i0 + 1 - c0 : int64_t(keys);
    const int uneven = all_see < keys ? int(max(all_see, int64_t(0))) / kKeys * kKeys : 0x7FFFFFFF;
    bool ok = true;
    int first = 0;  // first key of the step
    int u = 0;
    for (bool end = false; ok && !end; ++u) {
      const int slot = u % G_::kRaws, tile_slot = u % G_::kTiles;
      ok = warp_wait(&bars->raw_full[slot], (u / G_::kRaws) & 1, abort, p.status, kStRawFull);
      if (ok && u >= G_::kTiles)
        ok = warp_wait(&bars->t_empty[tile_slot], (u / G_::kTiles - 1) & 1, abort, p.status, kStTEmpty);
      if (!ok) break;
      const uint32_t raw = sbase + uint32_t(G_::kOffRaw + slot * G_::kRaw);
      const uint32_t dst = sbase + uint32_t(G_::kOffTile + tile_slot * G_::kTile);
      // iteration it of a warp: eight keys (it % 4) * 32 + key0, chunks (it / 4) * 4 + ch0. A key's
      // factor: 2^expo, expo in [-15, 6]
      uint32_t f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = bars->expo[slot][(i * 32 + key0) >> 4];
        f[i] = 0x00010001u * (e >= -14 ? uint32_t(e + 15) << 10 : 1u << 9);
      }
      // address of the codes of iteration it: key (it % 4) * 32 + key0, chunk (it / 4) * 4 + ch0
      auto codes_at = [&](int it) {
        const uint32_t o = uint32_t(((it & 3) * 32 + key0) * D + ((it >> 2) * 4 + ch0) * 16);
        return raw + (o ^ (((o >> 7) & 7u) << 4));
      };
      uint32_t valid = bars->valid[(u >> 1) & 15];
      if ((u & 1) == 0) first += kKeys;
      else end = (valid & kLast) != 0u;
      if ((valid & kChange) != 0u) first = bars->step[(u >> 1) & 15].first;
      valid &= kAllThere;
      if (valid != kAllThere || first + kKeys > keys) {
        // Keys that are not there (behind the last one, on missing pages or those of another step): their stale
        // bytes may be E4M3's NaN pattern, so they are zeroed. A thread zeroes what it converts itself below.
#pragma unroll 1
        for (int it = 0; it < kIter; ++it) {
          const int key = (it & 3) * 32 + key0;
          if (first + key >= keys || ((valid >> (key >> 4)) & 1u) == 0u) sts128(codes_at(it), 0u, 0u, 0u, 0u);
        }
      }
      if ((u & 1) != 0 && first >= uneven) {
        bool any = false;
#pragma unroll
        for (int it = 0; it < kIter; ++it) any = has_nan(lds128(codes_at(it))) || any;
        if (any) {
          bars->nans = 1;
#pragma unroll 1
          for (int it = 0; it < kIter; ++it) {
            uint4 v = lds128(codes_at(it));
            hide_nans(v, first + (it & 3) * 32 + key0, ((it >> 2) * 4 + ch0) * 16, bars->nan_from);
            sts128(codes_at(it), v.x, v.y, v.z, v.w);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kIter; b += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = lds128(codes_at(b + i));
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int key = ((b + i) & 3) * 32 + key0, ch = ((b + i) >> 2) * 4 + ch0;
          const uint32_t at = dst + uint32_t((ch >> 2) * (kKeys * 128) + key * 128);
          const uint32_t c2 = uint32_t((ch & 3) * 2), k7 = uint32_t(key & 7);
          uint32_t y[8];
          cvt4(v[i].x, y);
          cvt4(v[i].y, y + 2);
          cvt4(v[i].z, y + 4);
          cvt4(v[i].w, y + 6);
          sts128(at + ((c2 ^ k7) << 4), hmul2(y[0], f[(b + i) & 3]), hmul2(y[1], f[(b + i) & 3]), hmul2(y[2], f[(b + i) & 3]), hmul2(y[3], f[(b + i) & 3]));
          sts128(at + (((c2 + 1) ^ k7) << 4), hmul2(y[4], f[(b + i) & 3]), hmul2(y[5], f[(b + i) & 3]), hmul2(y[6], f[(b + i) & 3]), hmul2(y[7], f[(b + i) & 3]));
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->raw_empty[slot]);
        mbar_arrive(&bars->t_full[tile_slot]);
      }
    }
  } else if (warp >= kWarpSoft0 && warp < kWarpSoft0 + 8) {
    // ---------------- softmax and output of row tile w ----------------
    setmaxnreg_inc<kRegsSoftmax>();
    const int w = (warp - kWarpSoft0) >> 2, tr = tid - kWarpSoft0 * 32;  // row of the CTA
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + G_::kColS + uint32_t(w * 128), t_o = t_lane + G_::kColO + uint32_t(w * D);
    float c_row = 1.0f;  // factor of the row's scores, but for the keys' unit
    float c = 1.0f;      // with it: z log2 e = S * c
    int vis = 0;      // keys of the chunk that this thread's row sees
    if (w < n_tiles) {
      const unsigned ti = (rem0 + unsigned(tr)) / Gu;
      if (p.scale != 0.0f) c_row = fabsf(p.scale) * kLog2e * exp2i(bars->q_exp[tr]);
      int64_t v = s.len;
      if (p.causal) v = min(v, s.len - s.n + i0 + int64_t(ti) + 1);
      vis = tr < rows ? int(max(min(v - c0, int64_t(keys)), int64_t(0))) : 0;
    }
    float m = -INFINITY;  // what the row's exponents are taken against (of z log2 e = S * c)
    int far = 0;          // m and the row's scores are in units of 2^far: see units_of
    int unit = 0;         // of O
    int ahead = 0;        // vis, less what the step's first key is beyond j * kKeys
    float2 l2 = make_float2(0.0f, 0.0f);
    bool ok = true;
    if (w < n_tiles) {
      bool end = false;
      for (int j = 0; !end; ++j) {
        ok = warp_wait(&bars->s_full[w], j & 1, abort, p.status, kStSFull);
        if (!ok) break;
        tc_fence_after();
        uint32_t valid = bars->valid[j & 15];
        int to = unit;
        end = (valid & kLast) != 0u;
        if ((valid & kChange) != 0u) {
          const Step st = bars->step[j & 15];
          ahead = vis - (st.first - j * kKeys);
          c = fmaxf(c_row * st.k_factor * exp2i(-far), 1e-37f);  // positive: -inf * c is -inf
          to = st.v_unit;
        }
        valid &= kAllThere;
        const int left = min(ahead - j * kKeys, kKeys);  // keys of the step that the row sees
        const bool masked = __any_sync(0xffffffffu, left < kKeys) || valid != kAllThere;
        float x[kKeys];
        auto load = [&]() {
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) tmem_ld32(t_s + uint32_t(i * 32), reinterpret_cast<uint32_t*>(x) + i * 32);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (i >= left || ((valid >> (i / 16)) & 1u) == 0u) x[i] = -INFINITY;
          }
        };
        load();
        float a0 = x[0], a1 = x[1], a2 = x[2], a3 = x[3];
#pragma unroll
        for (int i = 4; i < kKeys - 4; i += 8) {
          a0 = max3(a0, x[i], x[i + 1]);
          a1 = max3(a1, x[i + 2], x[i + 3]);
          a2 = max3(a2, x[i + 4], x[i + 5]);
          a3 = max3(a3, x[i + 6], x[i + 7]);
        }
        a0 = max3(a0, x[kKeys - 4], x[kKeys - 3]);
        a1 = max3(a1, x[kKeys - 2], x[kKeys - 1]);
        // (rounded up, as the differences to it are: x c - m below takes x c as it is, which then passes neither)
        float top = __fmul_ru(max3(fmaxf(a0, a1), a2, a3), c);
        // raise the reference where the row is beyond it by 2^kMost (or had none)
        const bool raise = top > m && !(__fsub_ru(top, m) <= kMost);
        if (__any_sync(0xffffffffu, raise) || to != unit) {
          float alpha = 1.0f;
          if (raise) {
            alpha = m == -INFINITY ? 0.0f : fast_exp2(m - (top - kBase));
            const int k = units_of(top * exp2i(far));
            c *= exp2i(far - k);
            m = __fsub_ru(top * exp2i(far - k), kBase);
            far = k;
          }
          l2.x *= alpha;
          l2.y *= alpha;
          alpha *= exp2i(unit - to);
          unit = to;
          if (j > 0) {
            // S of this step was issued after P V of the last and is complete, so O is at rest. The
            // scores are read again after it: their registers serve here.
#pragma unroll
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + uint32_t(i), o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(t_o + uint32_t(i), o);
              tmem_st16(t_o + uint32_t(i + 16), o + 16);
            }
            load();
          }
        }
        const float mu = m == -INFINITY ? 0.0f : m;
        const float2 c2 = make_float2(c, c), n2 = make_float2(-mu, -mu);
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
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[w]);
        l2 = __fadd2_rn(l2, __fadd2_rn(sum0, sum1));
      }
      if (ok) ok = warp_wait(&bars->o_full[w], 0, abort, p.status, kStOFull);
      if (ok) {
        tc_fence_after();
        const int r = tr;
        const bool live = r < rows;
        const int64_t row = my_row;
        const float L = l2.x + l2.y;
        const float inv = whole ? (L != 0.0f ? exp2i(unit) / L : 0.0f) : exp2i(unit);
        const bool nans = bars->nans != 0;
        auto show_nans = [&](uint32_t* o, int col) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (bars->nan_from[col + e] < vis) o[e] = 0x7FFFFFFFu;
        };
        if (whole) {
          // through shared memory (this warp's rows of Q, which every MMA is done with), so that a
          // row's 16-byte pieces leave side by side
          const uint32_t mine = sbase + uint32_t(w * G_::kQBytes + (warp & 3) * 32 * D * 2);
          constexpr int kPieces = kLpr;
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + uint32_t(i), o);
            tmem_wait_ld();
            if (nans) show_nans(o, i);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t y[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                y[q] = pack16(__uint_as_float(o[e + 2 * q]) * inv, __uint_as_float(o[e + 2 * q + 1]) * inv, kF16);
              const int piece = (i + e) / 8;
              sts128(mine + uint32_t(lane * D * 2) + uint32_t((piece ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
            }
          }
          __syncwarp();
          const int piece = lane % kPieces;
#pragma unroll
          for (int i0 = 0; i0 < 32 / kRpi; i0 += 8) {
            uint4 y[8];
            int64_t to[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = (i0 + i) * kRpi + lane / kPieces;
              y[i] = lds128(mine + uint32_t(rr * D * 2) + uint32_t((piece ^ (rr & 7)) << 4));
              to[i] = __shfl_sync(0xffffffffu, my_row, rr);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((warp - kWarpSoft0) * 32 + (i0 + i) * kRpi + lane / kPieces < rows)
                *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to[i] * D) + piece) = y[i];
          }
        } else {
          // the same for a partial result, 32 columns at a time (a thread's own row straight to the
          // workspace: 512 new tokens of 8192 124 us, so 118)
          const uint32_t mine = sbase + uint32_t(w * G_::kQBytes + (warp & 3) * 32 * D * 2);
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + uint32_t(i), o);
            tmem_wait_ld();
            if (nans) show_nans(o, i);
            __syncwarp();  // the last columns have been read
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              uint32_t y[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) y[q] = __float_as_uint(__uint_as_float(o[e + q]) * inv);
              sts128(mine + uint32_t(lane * 128) + uint32_t(((e / 4) ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int rr = k * 4 + lane / 8;
              const uint4 y = lds128(mine + uint32_t(rr * 128) + uint32_t(((lane ^ rr) & 7) << 4));
              const int64_t to = __shfl_sync(0xffffffffu, my_row, rr);
              if ((warp - kWarpSoft0) * 32 + rr < rows)
                *(reinterpret_cast<uint4*>(p.ws + (to * p.ws_splits + split) * (D + 4) + i) + lane % 8) = y;
            }
          }
        }
        if (live && whole) {
          if (p.lse != nullptr) p.lse[row] = L != 0.0f ? (m + log2f(L)) * exp2i(far) * kLn2 : -INFINITY;
        } else if (live) {
          float* dst = p.ws + (row * p.ws_splits + split) * (D + 4) + D;
          dst[0] = m * exp2i(far);
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

template <int D, bool kF16>
cudaError_t launch_tc(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  const uint64_t rows128 = uint64_t(p.c.num_pages) * p.c.kv_heads * p.c.page_size * D / 128;
  const int box = (p.c.page_size < kKeys ? p.c.page_size : kKeys) * D / 128;
  CUtensorMap map_k, map_v;
  if (!encode_bytes_2d(&map_k, p.c.k, rows128, 128, 128, uint32_t(box)) ||
      !encode_bytes_2d(&map_v, p.c.v, rows128, 128, 128, uint32_t(box)))
    return cudaErrorInvalidValue;
  auto kern = kv_attn_tc_kernel<D, kF16>;
  // setmaxnreg.inc draws on what the block was launched with
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs != kRegsLaunch) return cudaErrorInvalidKernelImage;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kern), Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(plan.tc_row_tiles) * p.c.kv_heads * plan.tc_splits * p.b.num_seqs;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  kern<<<unsigned(grid), kThreads, Geo<D>::kSmem, stream>>>(map_k, map_v, p, plan.tc_row_tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attn_tc(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream) {
  if (p.c.head_dim == 128)
    return p.fp16 ? launch_tc<128, true>(p, plan, stream) : launch_tc<128, false>(p, plan, stream);
  return p.fp16 ? launch_tc<64, true>(p, plan, stream) : launch_tc<64, false>(p, plan, stream);
}

}  // namespace fq
