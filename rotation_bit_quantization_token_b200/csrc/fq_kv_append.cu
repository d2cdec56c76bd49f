// Appends keys and values to the 8-bit paged cache, with the position rotation on the way.
//
// For a new token at position pos and pair j of its head: angle a = pos * inv_freq[j],
//     (x, y) -> (x cos a - y sin a, y cos a + x sin a)
// and for one page and head, with m the largest magnitude of the page's tokens,
//     e = smallest exponent with m <= 448 * 2^e (clamped),  code = e4m3(value * 2^-e).
// A page that held tokens before keeps max(e_old, e_new); when that grows by d, an older code c
// becomes e4m3(c * 2^-d), which changes only codes that turn subnormal.
//
// One CTA takes one page of one sequence (a work item) and a range of key / value heads. An item
// is found without the host: a sequence with n new tokens touches at most n / page_size + 2
// pages, so with start(b) = cu_new[b] / page_size + 2b the items of sequence b are start(b),
// start(b) + 1, ... and T / page_size + 2 num_seqs CTAs cover every batch; CTAs past a
// sequence's last page leave at once. sin and cos of the page's tokens are computed once per
// CTA (angle and reduction in float64: pos * inv_freq needs up to 48 bits) and serve all its
// heads. A warp carries up to kRows rows of one head in registers between the maximum and the
// encoding, so the inputs are read once; a page with more rows is shared by several warps,
// which meet in shared memory for the maximum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "fq_kv.h"
#include "fq_ptx.cuh"

namespace fq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 16;  // rows of a task in one warp's registers

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// E elements (2 or 4) at p, as float32
template <typename T, int E>
__device__ __forceinline__ void load_elems(const T* p, float* x) {
  if constexpr (E == 4) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const float2 a = unpack2<T>(__ldg(reinterpret_cast<const uint32_t*>(p)));
    x[0] = a.x; x[1] = a.y;
  }
}

// Two floats as E4M3 bytes (nearest even, saturating), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), clamped. For amax = f * 2^k, f in
// [1, 2): k - 8 when f <= 1.75, else k - 7.
__device__ __forceinline__ int page_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits == 0u) return kPageExpMin;
  int e = int(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kPageExpMin ? kPageExpMin : e;
  return e > kPageExpMax ? kPageExpMax : e;
}

// The E elements d0 .. d0 + E - 1 of one head's row, rotated. cs: (cos, sin) of the row's pairs.
template <typename T, int D, int E>
__device__ __forceinline__ void load_rotated(const T* row, int d0, const float2* cs, int rot, int interleaved,
                                             float* x) {
  load_elems<T, E>(row + d0, x);
  if (d0 >= rot) return;  // rot is a multiple of E
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 z = cs[(d0 + e) >> 1];
      const float a = x[e], b = x[e + 1];
      x[e] = a * z.x - b * z.y;
      x[e + 1] = b * z.x + a * z.y;
    }
  } else {
    const int half = rot >> 1;
    const bool low = d0 < half;
    float y[E];
    load_elems<T, E>(row + (low ? d0 + half : d0 - half), y);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 z = cs[(low ? d0 : d0 - half) + e];
      x[e] = low ? x[e] * z.x - y[e] * z.y : x[e] * z.x + y[e] * z.y;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(const KvAppendParams p) {
  constexpr int E = D / 32;  // elements of a row per lane
  extern __shared__ float2 s_cs[];  // [rows][rot / 2]
  __shared__ float s_max[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps = p.c.page_size, H = p.c.kv_heads;

  // ---- the work item ----
  const int item = blockIdx.x;
  int lo = 0, hi = p.b.num_seqs - 1;  // the last sequence with start(b) <= item
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (int64_t(__ldg(p.b.cu_new + mid)) / ps + 2 * int64_t(mid) <= item) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  const int64_t t_first = __ldg(p.b.cu_new + b);
  const int64_t n = int64_t(__ldg(p.b.cu_new + b + 1)) - t_first;
  const int64_t len = __ldg(p.b.seq_lens + b);
  const int64_t first = len - n;  // position of the first new token
  const int64_t local = int64_t(item) - (t_first / ps + 2 * int64_t(b));
  if (n <= 0 || local < 0) return;
  if (first < 0 || t_first < 0 || t_first + n > p.T) {
    if (local == 0 && tid == 0 && p.status != nullptr) atomicOr(p.status, FQ_KV_BAD_BATCH);
    return;
  }
  const int64_t page_idx = first / ps + local;
  const int64_t at0 = page_idx * ps;
  if (at0 >= len) return;
  const int r0 = first > at0 ? int(first - at0) : 0;  // rows r0 .. r1 - 1 of the page are new
  const int r1 = len - at0 < ps ? int(len - at0) : ps;
  const int rows = r1 - r0;
  const int64_t t0 = t_first + (at0 + r0 - first);  // token of row r0
  int page = -1;
  if (page_idx < p.b.table_width) page = __ldg(p.b.page_table + int64_t(b) * p.b.table_width + page_idx);
  const bool stored = page >= 0 && int64_t(page) < p.c.num_pages;
  if (!stored && tid == 0 && p.status != nullptr) atomicOr(p.status, FQ_KV_BAD_BATCH);

  // ---- sin and cos of the new rows ----
  const int half = p.rot_dim >> 1;
  for (int i = tid; i < rows * half; i += kThreads) {
    const int r = i / half, j = i - r * half;
    // turns = pos * f / (2 pi); the fraction of a turn is exact to 2^-52 of the turns
    const double turns = double(at0 + r0 + r) * double(__ldg(p.inv_freq + j)) * 0.15915494309189533577;
    float s, c;
    sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
    s_cs[i] = make_float2(c, s);
  }
  __syncthreads();

  const int h_begin = blockIdx.y * p.heads_per_cta;
  const int h_end = min(h_begin + p.heads_per_cta, H);
  const int d0 = lane * E;

  // ---- keys and values: a task is one head of K or of V; wpt warps share it ----
  int wpt = 1;
  while (wpt * kRows < rows) wpt *= 2;
  const int tasks = stored ? 2 * (h_end - h_begin) : 0;
  const int per_round = kWarps / wpt;
  for (int base = 0; base < tasks; base += per_round) {
    const int task = base + warp / wpt, part = warp % wpt;
    const bool active = task < tasks;
    const int h = h_begin + (task >> 1);
    const bool is_k = (task & 1) == 0;
    float x[kRows][E];
    float m = 0.0f;
    int old = 0;  // exponent of the page's older rows
    uint8_t* scale = (is_k ? p.c.k_scale : p.c.v_scale) + int64_t(page) * H + h;
    if (active) {
      if (r0 > 0) old = int(*scale) - 127;
      const int64_t stride = is_k ? p.k_stride : p.v_stride;
      const T* src = static_cast<const T*>(is_k ? p.k : p.v) + t0 * stride + int64_t(h) * D;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = part + i * wpt;
        if (r < rows) {
          if (is_k) load_rotated<T, D, E>(src + r * stride, d0, s_cs + r * half, p.rot_dim, p.interleaved, x[i]);
          else load_elems<T, E>(src + r * stride + d0, x[i]);
#pragma unroll
          for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(x[i][e]));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    // the maximum over the task's warps; it also orders every warp's read of the old exponent
    // before one of them writes the new one
    if (wpt > 1) {  // the same for the whole CTA
      if (lane == 0) s_max[warp] = m;
      __syncthreads();
      for (int w = 0; w < wpt; ++w) m = fmaxf(m, s_max[(warp / wpt) * wpt + w]);
      __syncthreads();
    }
    if (!active) continue;
    uint8_t* codes = static_cast<uint8_t*>(is_k ? p.c.k : p.c.v) + (int64_t(page) * H + h) * ps * D;
    int e = page_exponent(m);
    if (r0 > 0) {
      if (old < e) {
        // the older rows move to the new exponent
        const float f = ptx::exp2i(max(old - e, -126));
        for (int i = (part * 32 + lane) * 4; i < r0 * D; i += wpt * 128) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + i);
          const float2 a = e4m3x2_value(w), c = e4m3x2_value(w >> 16);
          *reinterpret_cast<uint32_t*>(codes + i) = e4m3x2(a.x * f, a.y * f) | (e4m3x2(c.x * f, c.y * f) << 16);
        }
      } else {
        e = min(old, kPageExpMax);
      }
    }
    const float f = ptx::exp2i(-e);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = part + i * wpt;
      if (r < rows) {
        uint8_t* dst = codes + (r0 + r) * D + d0;
        const uint32_t w = e4m3x2(x[i][0] * f, x[i][1] * f);
        if constexpr (E == 4)
          *reinterpret_cast<uint32_t*>(dst) = w | (e4m3x2(x[i][2] * f, x[i][3] * f) << 16);
        else
          *reinterpret_cast<uint16_t*>(dst) = uint16_t(w);
      }
    }
    if (part == 0 && lane == 0) *scale = uint8_t(e + 127);
  }

  // ---- queries ----
  if (p.q != nullptr) {
    const int G = p.q_heads / H;
    const int nh = (h_end - h_begin) * G;
    for (int i = warp; i < rows * nh; i += kWarps) {
      const int r = i / nh, h = h_begin * G + i % nh;
      float x[E];
      load_rotated<T, D, E>(static_cast<const T*>(p.q) + (t0 + r) * p.q_stride + int64_t(h) * D, d0, s_cs + r * half,
                            p.rot_dim, p.interleaved, x);
      T* dst = static_cast<T*>(p.q_out) + ((t0 + r) * p.q_heads + h) * D + d0;
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack2<T>(x[0], x[1]);
    }
  }
}

template <typename T, int D>
cudaError_t launch_append(const KvAppendParams& p0, int num_sms, cudaStream_t stream) {
  KvAppendParams p = p0;
  const int64_t items = p.T / p.c.page_size + 2 * int64_t(p.b.num_seqs);
  // heads are divided among CTAs until every SM has about four of them
  int groups = 1;
  while (groups < p.c.kv_heads && items * groups < 4 * int64_t(num_sms)) groups *= 2;
  p.heads_per_cta = (p.c.kv_heads + groups - 1) / groups;
  groups = (p.c.kv_heads + p.heads_per_cta - 1) / p.heads_per_cta;
  const int smem = p.c.page_size * (p.rot_dim / 2) * int(sizeof(float2));
  cudaError_t e = cudaFuncSetAttribute(kv_append_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kv_append_kernel<T, D><<<dim3(unsigned(items), unsigned(groups)), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  if (p.c.head_dim == 128)
    return fp16 ? launch_append<__half, 128>(p, num_sms, stream) : launch_append<__nv_bfloat16, 128>(p, num_sms, stream);
  return fp16 ? launch_append<__half, 64>(p, num_sms, stream) : launch_append<__nv_bfloat16, 64>(p, num_sms, stream);
}

}  // namespace fq
