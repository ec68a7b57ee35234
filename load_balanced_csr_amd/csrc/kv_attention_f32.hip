// spmv_kv_attention on 32-bit caches.
#include "kv_attention.hpp"

namespace spmv {
hipError_t launch_kv_attention_f32(const KvAttentionArgs& a, hipStream_t s) {
  return launch_kv_attention_dim<float, float, 1>(a, s);
}
}  // namespace spmv
