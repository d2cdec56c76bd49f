// Host layer of the 8-bit paged cache: argument checks and launches of fq_kv_append and
// fq_kv_attention (include/fq.h). Nothing here reads device memory, allocates or waits.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fq_internal.h"
#include "fq_kv.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fq_status fail(cudaError_t e) {
  fq::record_cuda_error(int(e));
  return FQ_ERR_CUDA;
}

fq_status check_cache(const fq_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
    return FQ_ERR_NULLPTR;
  if (c->kv_heads < 1 || c->kv_heads > 256 || (c->head_dim != 64 && c->head_dim != 128)) return FQ_ERR_INVALID;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FQ_ERR_INVALID;
  if (c->num_pages < 1 || c->num_pages > 0x7FFFFFFF) return FQ_ERR_INVALID;
  // rows of 128 bytes are addressed by a 32-bit tensor-map coordinate
  if (c->num_pages * (int64_t(c->kv_heads) * c->page_size * c->head_dim / 128) > 0x7FFFFFFF) return FQ_ERR_INVALID;
  return aligned(c->k, 16) && aligned(c->v, 16) ? FQ_OK : FQ_ERR_INVALID;
}

fq_status check_batch(const fq_kv_batch* b) {
  if (b == nullptr || b->cu_new == nullptr || b->seq_lens == nullptr || b->page_table == nullptr) return FQ_ERR_NULLPTR;
  if (b->num_seqs < 1 || b->num_seqs > 65536 || b->table_width < 1 || b->table_width > (1 << 24)) return FQ_ERR_INVALID;
  return aligned(b->cu_new, 4) && aligned(b->seq_lens, 4) && aligned(b->page_table, 4) ? FQ_OK : FQ_ERR_INVALID;
}

// token arrays: rows of heads * head_dim elements, stride elements apart, 16-byte vectors
bool tokens_ok(const void* p, int64_t stride, int64_t row) {
  return aligned(p, 16) && stride % 8 == 0 && stride >= row && stride <= (int64_t(1) << 32);
}

fq_status sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? FQ_OK : fail(e);
}

fq_status check_attention(const fq_kv_cache* cache, const fq_kv_batch* batch, int64_t T, int32_t q_heads,
                          int32_t max_q_len, int64_t max_seq_len) {
  fq_status st = check_cache(cache);
  if (st == FQ_OK) st = check_batch(batch);
  if (st != FQ_OK) return st;
  if (T < 1 || T > (1 << 24) || q_heads < 1 || q_heads > 1024 || q_heads % cache->kv_heads != 0) return FQ_ERR_INVALID;
  if (max_q_len < 1 || max_q_len > T) return FQ_ERR_INVALID;
  if (max_seq_len < 1 || max_seq_len > int64_t(batch->table_width) * cache->page_size || max_seq_len > 0x7FFFFFFF)
    return FQ_ERR_INVALID;
  return FQ_OK;
}

}  // namespace

extern "C" {

fq_status fq_kv_append(const fq_kv_cache* cache, const fq_kv_batch* batch, int64_t T, fq_dtype dtype, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, const float* inv_freq, int32_t rot_dim,
                       int interleaved, const void* q, int64_t q_stride, int32_t q_heads, void* q_out,
                       uint32_t* status, struct CUstream_st* stream) {
  fq_status st = check_cache(cache);
  if (st == FQ_OK) st = check_batch(batch);
  if (st != FQ_OK) return st;
  if (k == nullptr || v == nullptr) return FQ_ERR_NULLPTR;
  if (T < 1 || T > (1 << 24) || (dtype != FQ_BF16 && dtype != FQ_FP16)) return FQ_ERR_INVALID;
  const int D = cache->head_dim, H = cache->kv_heads;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1)) return FQ_ERR_INVALID;
  if (rot_dim > 0 && inv_freq == nullptr) return FQ_ERR_NULLPTR;
  if (!tokens_ok(k, k_stride, int64_t(H) * D) || !tokens_ok(v, v_stride, int64_t(H) * D)) return FQ_ERR_INVALID;
  if (!aligned(inv_freq, 4) || !aligned(status, 4)) return FQ_ERR_INVALID;
  if ((q == nullptr) != (q_out == nullptr)) return FQ_ERR_NULLPTR;
  if (q != nullptr) {
    if (q_heads < 1 || q_heads > 1024 || q_heads % H != 0) return FQ_ERR_INVALID;
    if (!tokens_ok(q, q_stride, int64_t(q_heads) * D) || !aligned(q_out, 16)) return FQ_ERR_INVALID;
  } else if (q_heads != 0) {
    return FQ_ERR_NULLPTR;
  }
  int sms = 0;
  st = sm_count(&sms);
  if (st != FQ_OK) return st;
  fq::KvAppendParams p{};
  p.c = *cache; p.b = *batch; p.k = k; p.v = v; p.q = q; p.q_out = q_out; p.inv_freq = inv_freq; p.status = status;
  p.T = T; p.k_stride = k_stride; p.v_stride = v_stride; p.q_stride = q_stride;
  p.rot_dim = rot_dim; p.interleaved = interleaved; p.q_heads = q_heads;
  const cudaError_t e = fq::launch_kv_append(p, dtype == FQ_FP16, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FQ_OK : fail(e);
}

fq_status fq_kv_attention_workspace(const fq_kv_cache* cache, const fq_kv_batch* batch, int64_t T, int32_t q_heads,
                                    int32_t max_q_len, int64_t max_seq_len, int64_t* bytes) {
  if (bytes == nullptr) return FQ_ERR_NULLPTR;
  *bytes = 0;
  fq_status st = check_attention(cache, batch, T, q_heads, max_q_len, max_seq_len);
  int sms = 0;
  if (st == FQ_OK) st = sm_count(&sms);
  if (st != FQ_OK) return st;
  *bytes = fq::plan_kv_attn(*cache, *batch, T, q_heads, max_q_len, max_seq_len, sms).ws_bytes;
  return FQ_OK;
}

fq_status fq_kv_attention(const fq_kv_cache* cache, const fq_kv_batch* batch, int64_t T, fq_dtype dtype, const void* q,
                          int64_t q_stride, int32_t q_heads, int32_t max_q_len, int64_t max_seq_len, double scale,
                          int causal, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                          uint32_t* status, struct CUstream_st* stream) {
  fq_status st = check_attention(cache, batch, T, q_heads, max_q_len, max_seq_len);
  if (st != FQ_OK) return st;
  if (q == nullptr || out == nullptr) return FQ_ERR_NULLPTR;
  if (dtype != FQ_BF16 && dtype != FQ_FP16) return FQ_ERR_INVALID;
  if (!std::isfinite(scale) || std::fabs(scale) > 1e30 || (causal != 0 && causal != 1)) return FQ_ERR_INVALID;
  if (!tokens_ok(q, q_stride, int64_t(q_heads) * cache->head_dim) || !aligned(out, 16)) return FQ_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(workspace, 16) || !aligned(status, 4)) return FQ_ERR_INVALID;
  int sms = 0;
  st = sm_count(&sms);
  if (st != FQ_OK) return st;
  const fq::KvAttnPlan plan = fq::plan_kv_attn(*cache, *batch, T, q_heads, max_q_len, max_seq_len, sms);
  if (plan.ws_bytes > 0) {
    if (workspace == nullptr) return FQ_ERR_NULLPTR;
    if (workspace_bytes < plan.ws_bytes) return FQ_ERR_INVALID;
  }
  fq::KvAttnParams p{};
  p.c = *cache; p.b = *batch; p.q = q; p.out = out; p.lse = lse; p.ws = static_cast<float*>(workspace);
  p.status = status; p.T = T; p.q_stride = q_stride; p.max_seq_len = max_seq_len; p.q_heads = q_heads;
  p.max_q_len = max_q_len; p.causal = causal; p.fp16 = dtype == FQ_FP16; p.scale = float(scale);
  p.chunk = plan.chunk; p.splits = plan.splits; p.tile_rows = plan.tile_rows; p.tc_rows = plan.tc_rows;
  p.tc_chunk = plan.tc_chunk; p.tc_splits = plan.tc_splits;
  p.cluster = plan.cluster; p.ws_splits = plan.ws_splits;
  const cudaError_t e = fq::launch_kv_attn(p, plan, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FQ_OK : fail(e);
}

}  // extern "C"
