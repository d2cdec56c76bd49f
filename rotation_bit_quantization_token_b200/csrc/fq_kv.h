// Internal declarations of the 8-bit paged cache: argument blocks shared by the host layer
// (fq_kv_api.cu) and the kernels (fq_kv_append.cu, fq_kv_attn.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fq.h"

namespace fq {

constexpr int kPageExpMin = -40, kPageExpMax = 40;  // range of a page's shared exponent

struct KvAppendParams {
  fq_kv_cache c;
  fq_kv_batch b;
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  const float* inv_freq;
  uint32_t* status;
  int64_t T, k_stride, v_stride, q_stride;
  int rot_dim, interleaved, q_heads;
  int heads_per_cta;  // key / value heads of one CTA
};
cudaError_t launch_kv_append(const KvAppendParams& p, bool fp16, int num_sms, cudaStream_t stream);

struct KvAttnParams {
  fq_kv_cache c;
  fq_kv_batch b;
  const void* q;
  void* out;
  float* lse;
  float* ws;         // partial results: [T * q_heads, ws_splits, head_dim + 4]
  uint32_t* status;
  int64_t T, q_stride, max_seq_len;
  int q_heads, max_q_len, causal, fp16;
  float scale;
  int chunk;         // keys of one split
  int splits;        // splits of the longest sequence
  int tile_rows;     // rows of a CTA (8 or 16)
  int64_t tc_rows;   // sequences with more rows (new tokens * group) take the tensor-core kernel
  int tc_chunk, tc_splits;
  int cluster;       // the chunks of up to tile_rows rows are a cluster, which joins them itself
  int ws_splits;     // slots per row of the workspace: most chunks that the join kernel joins
};

// How fq_kv_attention divides its work; the workspace follows from it.
struct KvAttnPlan {
  int chunk, splits, tile_rows, row_tiles;  // mma.sync kernel: tile_rows rows and one chunk per CTA; 0 tiles: not launched
  int tc_chunk, tc_splits, tc_row_tiles;    // tensor-core kernel: 256 rows and one chunk per CTA; 0: not launched
  int64_t tc_rows;
  int cluster, ws_splits;                   // see KvAttnParams
  int64_t ws_bytes;
};
KvAttnPlan plan_kv_attn(const fq_kv_cache& c, const fq_kv_batch& b, int64_t T, int q_heads, int max_q_len,
                        int64_t max_seq_len, int num_sms);
cudaError_t launch_kv_attn(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream);
cudaError_t launch_kv_attn_tc(const KvAttnParams& p, const KvAttnPlan& plan, cudaStream_t stream);

constexpr int kTcRows = 256;  // rows of a CTA of the tensor-core kernel

}  // namespace fq
