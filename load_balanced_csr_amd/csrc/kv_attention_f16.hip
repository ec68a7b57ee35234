// spmv_kv_attention on f16 caches.
#include "kv_attention.hpp"

namespace spmv {
hipError_t launch_kv_attention_f16(const KvAttentionArgs& a, hipStream_t s) {
  return kv_row_blocks(a.group, a.cache_dtype) == 2 ? launch_kv_attention_dim<f16, f16, 2>(a, s)
                                                    : launch_kv_attention_dim<f16, f16, 1>(a, s);
}
}  // namespace spmv
