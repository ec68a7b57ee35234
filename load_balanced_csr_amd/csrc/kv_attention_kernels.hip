// spmv_kv_attention: which instantiation of kv_attention.hpp a call runs.
#include "kv_attention.hpp"

namespace spmv {

size_t kv_attention_workspace(int group, int head_dim, int cache_dtype) {
  return kKvCounterBytes + 2 * kKvMaxBlocks * sizeof(float) *
                               kv_slot_floats(kv_row_blocks(group, cache_dtype),
                                              kv_dim_pad(head_dim));
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t s) {
  if (a.cache_dtype == SPMV_KV_F8E4M3)
    return a.dtype == SPMV_KV_F16 ? launch_kv_attention_f8_f16(a, s)
                                  : launch_kv_attention_f8_bf16(a, s);
  switch (a.dtype) {
    case SPMV_KV_F32: return launch_kv_attention_f32(a, s);
    case SPMV_KV_F16: return launch_kv_attention_f16(a, s);
    default: return launch_kv_attention_bf16(a, s);
  }
}

}  // namespace spmv
