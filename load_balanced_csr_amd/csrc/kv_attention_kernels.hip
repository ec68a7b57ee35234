// Attention of one new token per request over a paged cache
// (spmv_kv_attention).
#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "kv_internal.hpp"
#include "kv_types.hpp"

namespace spmv {
namespace {

constexpr int kMaxDim = 256;

// One wavefront per request and query head, everything in 32 bits. Lanes are
// tokens for the scores (each lane walks its key row), elements for the sum
// over the values; the running maximum m and sum l are those of the tokens
// seen so far, the accumulators rescaled by exp(m_old - m_new).
template <typename Q, typename C>
__global__ __launch_bounds__(kWave) void kv_attention_kernel(KvAttentionArgs a) {
  __shared__ float qs[kMaxDim];
  const int r = blockIdx.x, h = blockIdx.y, lane = lane_id();
  const int kh = h / a.group, D = a.head_dim;
  const Q* q = static_cast<const Q*>(a.q) + r * a.q_request + h * a.q_head;
  const float ks = a.k_scale ? a.k_scale[kh] : 1.f, vs = a.v_scale ? a.v_scale[kh] : 1.f;
  for (int d = lane; d < D; d += kWave) qs[d] = to_f32(q[d]) * a.scale * ks;
  __syncthreads();
  const int32_t n = min(max(a.lengths[r], 0), a.table_tokens);
  const int32_t from = a.window && n > a.window ? n - a.window : 0;
  const int32_t first = min(a.sinks, from);
  const int32_t seen = first + n - from;

  float m = -INFINITY, l = 0.f, acc[kMaxDim / kWave] = {};
  for (int32_t i0 = 0; i0 < seen; i0 += kWave) {
    const int32_t i = i0 + lane, t = i < first ? i : from + i - first;
    int32_t page = -1, at = 0;
    if (i < seen) {
      const uint32_t j = div_by(t, a.page);
      page = a.table[r * a.table_stride + j];
      at = t - j * a.page.d;
      if (page >= a.n_pages) page = -1;
    }
    float s = -INFINITY;
    if (page >= 0) {
      const C* k = static_cast<const C*>(a.k) + page * a.k_page + at * a.k_token + kh * a.k_head;
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(qs[d], to_f32(k[d]), s);
    }
    float top = s;
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float m_new = fmaxf(m, top);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float p = page >= 0 ? expf(s - base) : 0.f, keep = expf(m - base);
    float sum = p;
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
    l = l * keep + sum;
    m = m_new;
    for (int e = 0; e < kMaxDim / kWave; ++e) acc[e] *= keep;
    const int many = min(kWave, seen - i0);
    for (int j = 0; j < many; ++j) {
      const int32_t pj = __shfl(page, j), aj = __shfl(at, j);
      const float w = __shfl(p, j);
      if (pj < 0) continue;
      const C* v = static_cast<const C*>(a.v) + pj * a.v_page + aj * a.v_token + kh * a.v_head;
      for (int e = 0; e < kMaxDim / kWave; ++e) {
        const int d = e * kWave + lane;
        if (d < D) acc[e] = fmaf(w, to_f32(v[d]), acc[e]);
      }
    }
  }
  Q* out = static_cast<Q*>(a.out) + r * a.out_request + h * a.out_head;
  const bool none = m == -INFINITY && l == 0.f;
  for (int e = 0; e < kMaxDim / kWave; ++e) {
    const int d = e * kWave + lane;
    if (d < D) out[d] = from_f32<Q>(none ? 0.f : acc[e] / l * vs);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)r * a.n_kv_heads * a.group + h] = none ? -INFINITY : m + logf(l);
}

template <typename Q, typename C>
hipError_t launch(const KvAttentionArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv_attention_kernel<Q, C>),
                     dim3(a.n_requests, a.n_kv_heads * a.group), dim3(kWave), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(int, int, int) { return 0; }

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t s) {
  if (a.cache_dtype == SPMV_KV_F8E4M3)
    return a.dtype == SPMV_KV_F16 ? launch<f16, f8>(a, s) : launch<bf16, f8>(a, s);
  switch (a.dtype) {
    case SPMV_KV_F32: return launch<float, float>(a, s);
    case SPMV_KV_F16: return launch<f16, f16>(a, s);
    default: return launch<bf16, bf16>(a, s);
  }
}

}  // namespace spmv
