// spmv_kv_attention on 8-bit caches with f16 queries.
#include "kv_attention.hpp"

namespace spmv {
hipError_t launch_kv_attention_f8_f16(const KvAttentionArgs& a, hipStream_t s) {
  return kv_row_blocks(a.group, a.cache_dtype) == 2 ? launch_kv_attention_dim<f8, f16, 2>(a, s)
                                                    : launch_kv_attention_dim<f8, f16, 1>(a, s);
}
}  // namespace spmv
