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
// sequence's last page leave at once. (The search is 32 probes at a time: one by one it was most of
// a decode step's time.) sin and cos of the page's tokens are computed once per CTA (angle and
// reduction in float64: pos * inv_freq needs up to 48 bits) and serve all its heads.
//
// A lane holds four elements of a row, chosen so that it has both of each pair that is turned
// (elements d, d + 1 and their partners half the rotated part further on, or four neighbours), so
// every element is read once. A warp carries its rows of one head in registers between the maximum
// and the encoding; a page with more rows is shared by several warps, which meet in shared memory
// for the maximum. Queries need no page: the CTAs behind those of the items take them, a warp for
// one token and up to eight heads. 64 single tokens (8 + 32 heads of 128): 4.7 us, bound by the launch
// and four dependent reads; seven prompts of 300-2500 tokens: 36 us, 4.0 TB/s of the 2 + 1 bytes an
// element of k and v and 2 + 2 of q, bound by instructions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "fq_kv.h"
#include "fq_ptx.cuh"

namespace fq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

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

// A lane's four elements of a row: lo, lo + 1, hi, hi + 1.
struct Quad {
  int lo, hi;
  bool turned;    // the pairs are turned: (lo, hi) and (lo + 1, hi + 1), or neighbours if interleaved
};
__device__ __forceinline__ Quad quad_of(int q, int rot, int interleaved) {
  const int half = rot >> 1;
  Quad z;
  z.lo = 4 * q;
  z.hi = 4 * q + 2;
  z.turned = 4 * q < rot;
  if (!interleaved && z.turned) {
    z.lo = 2 * q;
    z.hi = half + 2 * q;
  }
  return z;  // lanes past rot / 4 hold the elements from rot on, four each
}

// kWritten: the kernel may write the row as well (queries in place), so it is not read as constant data.
template <bool kWritten, typename T>
__device__ __forceinline__ uint2 load_quad(const T* row, const Quad& z) {
  if constexpr (kWritten) {
    if (z.hi == z.lo + 2) return *reinterpret_cast<const uint2*>(row + z.lo);
    return make_uint2(*reinterpret_cast<const uint32_t*>(row + z.lo), *reinterpret_cast<const uint32_t*>(row + z.hi));
  }
  if (z.hi == z.lo + 2) return __ldg(reinterpret_cast<const uint2*>(row + z.lo));
  return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(row + z.lo)), __ldg(reinterpret_cast<const uint32_t*>(row + z.hi)));
}

// cs: (cos, sin) of the quad's two pairs
template <typename T>
__device__ __forceinline__ float4 turn(uint2 w, const Quad& z, int interleaved, float4 cs) {
  const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
  if (!z.turned) return make_float4(a.x, a.y, b.x, b.y);
  if (interleaved)
    return make_float4(a.x * cs.x - a.y * cs.y, a.y * cs.x + a.x * cs.y, b.x * cs.z - b.y * cs.w, b.y * cs.z + b.x * cs.w);
  return make_float4(a.x * cs.x - b.x * cs.y, a.y * cs.z - b.y * cs.w, b.x * cs.x + a.x * cs.y, b.y * cs.z + a.y * cs.w);
}

// (cos, sin) of angle pos * f: turns = pos * f / (2 pi); the fraction of a turn is exact to 2^-52 of
// the turns.
__device__ __forceinline__ float2 cos_sin_of(int64_t pos, float f) {
  const double turns = double(pos) * double(f) * 0.15915494309189533577;
  float s, c;
  sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
  return make_float2(c, s);
}

// The last b in [0, n) with key(b) <= x, keys rising, key(0) <= x assumed: 32 probes at a time, by a
// whole warp.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int x, const F& key) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int left = n; left > 1;) {  // it is one of b .. b + left - 1
    const int step = (left + 31) >> 5;
    const bool in = lane * step < left && key(b + lane * step) <= x;
    const int top = 31 - __clz(__ballot_sync(0xffffffffu, in) | 1u);
    b += top * step;
    left = min(step, left - top * step);
  }
  return b;
}

constexpr int kQHeads = 8;  // query heads of one token that a warp takes

// Queries: warp `task` takes heads kQHeads * (task % chunks) .. of token task / chunks.
template <typename T, int D>
__device__ __forceinline__ void rotate_queries(const KvAppendParams& p, int64_t task) {
  constexpr int kLpr = D / 4, kRps = 32 / kLpr;  // lanes per row, rows per step of a warp
  constexpr int kIter = kQHeads / kRps;
  const int lane = threadIdx.x & 31, lq = lane % kLpr, sub = lane / kLpr;
  const int chunks = (p.q_heads + kQHeads - 1) / kQHeads;
  const int64_t t = task / chunks;
  const int h0 = int(task - t * chunks) * kQHeads;
  if (t >= p.T) return;
  const Quad z = quad_of(lq, p.rot_dim, p.interleaved);
  uint2 w[kIter];
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const int h = h0 + k * kRps + sub;
    w[k] = make_uint2(0u, 0u);
    if (h < p.q_heads) w[k] = load_quad<true>(static_cast<const T*>(p.q) + t * p.q_stride + int64_t(h) * D, z);
  }
  const int b = warp_search(p.b.num_seqs, int(t), [&](int i) { return __ldg(p.b.cu_new + i); });
  const int64_t t_first = __ldg(p.b.cu_new + b), t_end = __ldg(p.b.cu_new + b + 1), len = __ldg(p.b.seq_lens + b);
  const int64_t pos = len - (t_end - t);
  if (t < t_first || t >= t_end || t_first < 0 || t_end > p.T || len < t_end - t_first) return;  // no sequence's token
  float4 cs = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
  if (z.turned) {
    // (one at a time: inv_freq is aligned to its elements only)
    const float2 a = cos_sin_of(pos, __ldg(p.inv_freq + 2 * lq)), c = cos_sin_of(pos, __ldg(p.inv_freq + 2 * lq + 1));
    cs = make_float4(a.x, a.y, c.x, c.y);
  }
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const int h = h0 + k * kRps + sub;
    if (h >= p.q_heads) continue;
    const float4 x = turn<T>(w[k], z, p.interleaved, cs);
    T* dst = static_cast<T*>(p.q_out) + (t * p.q_heads + h) * D;
    if (z.hi == z.lo + 2) {
      *reinterpret_cast<uint2*>(dst + z.lo) = make_uint2(pack2<T>(x.x, x.y), pack2<T>(x.z, x.w));
    } else {
      *reinterpret_cast<uint32_t*>(dst + z.lo) = pack2<T>(x.x, x.y);
      *reinterpret_cast<uint32_t*>(dst + z.hi) = pack2<T>(x.z, x.w);
    }
  }
}

template <typename T, int D, int kSteps>
__global__ void __launch_bounds__(kThreads, kSteps == 8 ? 4 : 2)
kv_append_kernel(const KvAppendParams p, const unsigned kv_ctas, const unsigned groups) {
  constexpr int kLpr = D / 4, kRps = 32 / kLpr;  // lanes per row, rows per step of a warp
  constexpr int kWarpRows = kSteps * kRps;
  extern __shared__ __align__(16) float2 s_cs[];  // [rows][rot / 2], read two at a time
  __shared__ float s_max[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x >= kv_ctas) {
    rotate_queries<T, D>(p, int64_t(blockIdx.x - kv_ctas) * kWarps + warp);
    return;
  }
  const int H = p.c.kv_heads;
  const int ps_log = 31 - __clz(p.c.page_size), ps = 1 << ps_log;

  // The first CTAs look after a sequence each and report it if its batch entries are out of range (its own
  // items may not be found then). There are two CTAs a sequence at least.
  const bool checks = blockIdx.x < unsigned(p.b.num_seqs) && p.status != nullptr;
  int c_first = 0, c_end = 0, c_len = 0;
  if (checks) {
    c_first = __ldg(p.b.cu_new + blockIdx.x);
    c_end = __ldg(p.b.cu_new + blockIdx.x + 1);
    c_len = __ldg(p.b.seq_lens + blockIdx.x);
  }

  // ---- the work item: the last sequence with start(b) <= item ----
  const int item = int(blockIdx.x / groups), group = int(blockIdx.x - unsigned(item) * groups);
  const int b = warp_search(p.b.num_seqs, item, [&](int i) { return (__ldg(p.b.cu_new + i) >> ps_log) + 2 * i; });
  const int64_t t_first = __ldg(p.b.cu_new + b);
  const int64_t n = int64_t(__ldg(p.b.cu_new + b + 1)) - t_first;
  const int64_t len = __ldg(p.b.seq_lens + b);
  if (checks && tid == 0 && (c_first < 0 || c_end < c_first || c_end > p.T || int64_t(c_end) - c_first > c_len))
    atomicOr(p.status, FQ_KV_BAD_BATCH);
  const int64_t first = len - n;  // position of the first new token
  const int64_t local = int64_t(item) - ((t_first >> ps_log) + 2 * int64_t(b));
  if (n <= 0 || local < 0) return;
  if (first < 0 || t_first < 0 || t_first + n > p.T) return;
  const int64_t page_idx = (first >> ps_log) + local;
  const int64_t at0 = page_idx << ps_log;
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
    s_cs[i] = cos_sin_of(at0 + r0 + r, __ldg(p.inv_freq + j));
  }
  __syncthreads();

  const int h_begin = group * p.heads_per_cta;
  const int h_end = min(h_begin + p.heads_per_cta, H);
  const int lq = lane % kLpr, sub = lane / kLpr;
  const Quad kz = quad_of(lq, p.rot_dim, p.interleaved), vz = quad_of(lq, 0, 1);
  auto cos_sin = [&](int r) {
    return kz.turned ? *reinterpret_cast<const float4*>(s_cs + r * half + 2 * lq) : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
  };

  // ---- keys and values: a task is one head of K or of V; wpt warps share it ----
  int wpt = 1;
  while (wpt * kWarpRows < rows) wpt *= 2;
  const int tasks = stored ? 2 * (h_end - h_begin) : 0;
  const int per_round = kWarps / wpt;
  for (int base = 0; base < tasks; base += per_round) {
    const int task = base + warp / wpt, part = warp % wpt;
    const bool active = task < tasks;
    const int h = h_begin + (task >> 1);
    const bool is_k = (task & 1) == 0;
    const Quad z = is_k ? kz : vz;
    float4 x[kSteps];
    float m = 0.0f;
    int old = 0;  // exponent of the page's older rows
    uint8_t* scale = (is_k ? p.c.k_scale : p.c.v_scale) + int64_t(page) * H + h;
    if (active) {
      const int64_t stride = is_k ? p.k_stride : p.v_stride;
      const T* src = static_cast<const T*>(is_k ? p.k : p.v) + t0 * stride + int64_t(h) * D;
      uint2 w[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = (part + i * wpt) * kRps + sub;
        w[i] = make_uint2(0u, 0u);
        if (r < rows) w[i] = load_quad<false>(src + r * stride, z);
      }
      if (r0 > 0) old = int(*scale) - 127;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = (part + i * wpt) * kRps + sub;
        x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < rows) x[i] = turn<T>(w[i], z, p.interleaved, is_k ? cos_sin(r) : make_float4(1.0f, 0.0f, 1.0f, 0.0f));
        m = fmaxf(m, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
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
    for (int i = 0; i < kSteps; ++i) {
      const int r = (part + i * wpt) * kRps + sub;
      if (r < rows) {
        uint8_t* dst = codes + (r0 + r) * D;
        const uint32_t lo = e4m3x2(x[i].x * f, x[i].y * f), hi = e4m3x2(x[i].z * f, x[i].w * f);
        if (z.hi == z.lo + 2) {
          *reinterpret_cast<uint32_t*>(dst + z.lo) = lo | (hi << 16);
        } else {
          *reinterpret_cast<uint16_t*>(dst + z.lo) = uint16_t(lo);
          *reinterpret_cast<uint16_t*>(dst + z.hi) = uint16_t(hi);
        }
      }
    }
    if (part == 0 && lane == 0) *scale = uint8_t(e + 127);
  }

}

template <typename T, int D, int kSteps>
cudaError_t launch_steps(const KvAppendParams& p0, int num_sms, cudaStream_t stream) {
  KvAppendParams p = p0;
  const int64_t items = p.T / p.c.page_size + 2 * int64_t(p.b.num_seqs);
  // Heads are divided among CTAs until every SM has two: a CTA's beginning (search, lengths, sin and
  // cos) is shared by its heads. With eight on an SM 64 sequences' single tokens took 6.6 us, with two
  // 4.7; seven prompts of 300-2500 tokens 39.9 and 35.8 (with sixteen 50.5).
  int groups = 1;
  while (groups < p.c.kv_heads && items * groups < 2 * int64_t(num_sms)) groups *= 2;
  p.heads_per_cta = (p.c.kv_heads + groups - 1) / groups;
  groups = (p.c.kv_heads + p.heads_per_cta - 1) / p.heads_per_cta;
  const int smem = p.c.page_size * (p.rot_dim / 2) * int(sizeof(float2));
  auto kern = kv_append_kernel<T, D, kSteps>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ptx::allow_smem(done, reinterpret_cast<const void*>(kern), 128 * (D / 2) * int(sizeof(float2)));
  if (e != cudaSuccess) return e;
  const int64_t q_tasks = p.q != nullptr ? p.T * ((p.q_heads + kQHeads - 1) / kQHeads) : 0;
  const int64_t kv_ctas = items * groups, ctas = kv_ctas + (q_tasks + kWarps - 1) / kWarps;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  kern<<<unsigned(ctas), kThreads, smem, stream>>>(p, unsigned(kv_ctas), unsigned(groups));
  return cudaGetLastError();
}

// A CTA's warps hold 8 * 8 rows of 128 elements, or 8 * 16 of 64: a page of 128 rows of 128 needs
// twice the steps (and registers).
template <typename T>
cudaError_t launch_type(const KvAppendParams& p, int num_sms, cudaStream_t stream) {
  if (p.c.head_dim == 64) return launch_steps<T, 64, 8>(p, num_sms, stream);
  return p.c.page_size == 128 ? launch_steps<T, 128, 16>(p, num_sms, stream) : launch_steps<T, 128, 8>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  return fp16 ? launch_type<__half>(p, num_sms, stream) : launch_type<__nv_bfloat16>(p, num_sms, stream);
}

}  // namespace fq
