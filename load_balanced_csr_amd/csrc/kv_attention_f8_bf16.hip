// spmv_kv_attention on 8-bit caches with bf16 queries.
#include "kv_attention.hpp"

namespace spmv {
hipError_t launch_kv_attention_f8_bf16(const KvAttentionArgs& a, hipStream_t s) {
  return kv_row_blocks(a.group, a.cache_dtype) == 2 ? launch_kv_attention_dim<f8, bf16, 2>(a, s)
                                                    : launch_kv_attention_dim<f8, bf16, 1>(a, s);
}
}  // namespace spmv
