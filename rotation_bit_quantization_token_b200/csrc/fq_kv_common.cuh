// What the two attention kernels over the 8-bit paged cache share: the rows of a sequence, the
// conversion of codes, a row's final result.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fq_kv.h"
#include "fq_ptx.cuh"

namespace fq {
namespace kv {

constexpr float kLog2e = 1.4426950408889634f;
// A kernel launched with programmatic serialization may start before the one ahead of it ends: the
// first tells that its dependents may be launched, the second waits until it has completed.
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int fp16) {
  if (fp16) return h2(a, b);
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two 16-bit elements as float32.
__device__ __forceinline__ float2 unpack16(uint32_t w, int fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Exponent qe such that amax * 2^-qe lies in [2^14, 2^15), or below where 2^-qe would not be a number: at
// most 113, for the largest bfloat16.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = int(__float_as_uint(amax) >> 23) - 127 - 14;
  return max(e, -126);
}

// Scale byte of a page as an exponent; a byte that fq_kv_append cannot have written still gives
// a number.
__device__ __forceinline__ int page_exp(uint32_t byte) {
  return min(max(int(byte) - 127, kPageExpMin), kPageExpMax);
}

// The rows (new token, head of the group) row0 .. row0 + count - 1 of sequence b and the keys
// that they can see.
struct Rows {
  int64_t t_first;  // first token row of the sequence
  int64_t n, len;   // new tokens, length
  int64_t q;        // new tokens whose queries are computed: the first max_q_len
  int64_t end;      // keys seen by at least one of the rows
  bool ok;
};
// a / b for a >= 0 (a 64-bit division takes several times as long as a 32-bit one).
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return (a >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ __forceinline__ Rows sequence_rows(const KvAttnParams& p, int b, int64_t row0, int count, int G) {
  Rows r;
  r.t_first = __ldg(p.b.cu_new + b);
  r.n = int64_t(__ldg(p.b.cu_new + b + 1)) - r.t_first;
  r.len = __ldg(p.b.seq_lens + b);
  r.ok = r.n >= 0 && r.t_first >= 0 && r.t_first + r.n <= p.T;
  r.ok = r.ok && r.len >= 0 && r.len <= p.max_seq_len && r.n <= r.len;
  if (!r.ok) r.n = 0;
  r.q = min(r.n, int64_t(p.max_q_len));
  const int64_t last = min(quotient(row0 + count - 1, G), r.q - 1);
  r.end = p.causal ? min(r.len, r.len - r.n + last + 1) : r.len;
  if (r.end < 0) r.end = 0;
  return r;
}

// A product with a probability of zero keeps a NaN of V, so in a tile of keys that some of the rows do
// not see, V's NaN codes are replaced by zeros, and the first key (of the chunk) that has one in column d
// is kept in nan_from[d]. What a row sees are the keys up to some one, so its output is NaN in the
// columns whose nan_from lies among them.
constexpr int kNoNan = 0x7FFFFFFF;
// Whether one of 16 codes is NaN: 1 added to its low seven bits carries into the eighth.
__device__ __forceinline__ bool has_nan(const uint4& v) {
  auto carry = [](uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; };
  return ((carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) & 0x80808080u) != 0u;
}
// Replaces the NaNs among 16 codes of one key, columns d0 .. d0 + 15.
__device__ __forceinline__ void hide_nans(uint4& v, int key, int d0, int* nan_from) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t nan = __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    w[i] &= ~nan;
    for (int e = 0; e < 4; ++e)
      if ((nan >> (8 * e)) & 1u) atomicMin(nan_from + d0 + 4 * i + e, key);
  }
}

// Whether the tensor-core kernel takes a sequence with q tokens' queries (else the other one does):
// more than p.tc_rows rows. Both kernels and the join decide by it.
__device__ __forceinline__ bool takes_tc(const KvAttnParams& p, int64_t q, int G) { return q * G > p.tc_rows; }

}  // namespace kv
}  // namespace fq
