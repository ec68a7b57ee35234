// Host-side launch interface of the paged-cache operators, between their C
// ABI (kv_api.hip) and their kernels (kv_table_kernels.hip,
// kv_append_kernels.hip, kv_attention_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spmv_kv.h"

namespace spmv {

// floor(n / d) for 0 <= n < 2^31 without a division: with s = ceil(log2 d)
// and mul = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (mulhi(mul, n) + n) >> s, and the sum stays below 2^32.
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return FastDiv{(uint32_t)((((uint64_t(1) << s) - d) << 32) / d + 1), s, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (__umulhi(f.mul, n) + n) >> f.shift;
}

struct KvResizeArgs {
  const int32_t* lengths;
  const int32_t* arg;          // grow: n_new; shrink: keep
  const int32_t* cursor;
  int32_t* pool;               // free_pages (grow only reads it)
  int32_t* table;              // (shrink only reads it)
  int32_t* lengths_out;
  int32_t* cursor_out;
  int32_t* token_ptr;
  int32_t* slots;
  int32_t* positions;
  int32_t* status;
  int64_t table_stride;
  int32_t table_tokens;        // table_width * page_size
  int32_t n_requests, n_free, n_tokens;
  FastDiv page;
};
hipError_t launch_kv_resize(const KvResizeArgs& a, bool grow, hipStream_t s);

struct KvAppendArgs {
  const void* src[2];          // k, v
  void* dst[2];
  const float* scale[2];
  int64_t src_token[2], src_head[2];                 // strides in elements
  int64_t dst_page[2], dst_token[2], dst_head[2];
  const int32_t* slots;
  int64_t n_slots;             // n_pages * page_size
  int64_t n_tokens;
  int32_t n_heads, head_dim;
  int32_t src_dtype, dst_dtype;
  bool aligned;                // 16-byte loads of src are allowed
  FastDiv page;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);

struct KvAttentionArgs {
  const void* q;
  void* out;
  float* lse;
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lengths;
  void* workspace;
  int64_t q_request, q_head, out_request, out_head;  // strides in elements
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  int64_t table_stride;
  int32_t table_tokens;        // table_width * page_size
  int32_t n_pages;
  int32_t n_requests, n_kv_heads, group, head_dim;   // group: query heads per key head
  int32_t window, sinks;       // window 0: all tokens
  int32_t cache_dtype, dtype;
  int32_t step_shift;          // set by the launch: see kv_units
  bool join_apart;             // set by the launch: a second one joins the cut rows
  bool q_aligned, out_aligned; // 16-byte loads of q, four-element stores of out
  float scale;
  FastDiv page;
};
hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t s);
size_t kv_attention_workspace(int group, int head_dim, int cache_dtype);
hipError_t launch_kv_attention_f32(const KvAttentionArgs& a, hipStream_t s);
hipError_t launch_kv_attention_f16(const KvAttentionArgs& a, hipStream_t s);
hipError_t launch_kv_attention_bf16(const KvAttentionArgs& a, hipStream_t s);
hipError_t launch_kv_attention_f8_f16(const KvAttentionArgs& a, hipStream_t s);
hipError_t launch_kv_attention_f8_bf16(const KvAttentionArgs& a, hipStream_t s);

}  // namespace spmv
