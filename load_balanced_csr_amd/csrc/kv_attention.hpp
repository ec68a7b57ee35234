// Attention of one new token per request over a paged cache: the kernel,
// instantiated per element type by kv_attention_*.hip.
//
// Mathematics. With the scores in powers of two, s = scale log2(e) q.k, a part
// of a row's tokens is summed up by its maximum m, l = sum 2^(s - m) and
// o = sum 2^(s - m) v; parts join by m = max m_i, l = sum l_i 2^(m_i - m), the
// same for o, in any grouping, and out = o / l.
//
// What bounds it. Every cached key and value is read once, 4 G operations for
// each pair of elements (G query heads share a key head): at G = 8 in 16 bits
// 8 operations a byte, far below the matrix cores' 300, so HBM is the bound
// and the design is about keeping loads in flight, and, for short rows, about
// latency.
//
// One wavefront takes a step of 16 or 32 consecutive tokens of one key head
// with up to 16 NB query heads. Both products run on the matrix cores with
// the query heads as the columns, and nothing passes through LDS:
//   S = K Q^T: a lane's A operand is 8 consecutive elements of one key, what
//     one 16-byte load brings (lane = token c, quarter g of each 64 bytes).
//   O^T = V^T P^T: the accumulator of S holds tokens 4g .. 4g+3 of query
//     column c in lane (c, g), which is how the B operand wants its 8 tokens
//     if the 32 tokens of two S tiles are numbered 8g + j <-> token 4g + j of
//     the first (j < 4) or second tile. So a lane loads from exactly those 8
//     values rows, 16 bytes each, 16 lanes side by side covering a row; an
//     8 x 8 transpose of 16-bit elements inside the lane (one v_perm per
//     word) gives the A operands, product e yielding elements 8c' + e.
// Rows of 32-bit elements need no transpose (one token per operand).
//
// Load balance. A row (request, key head, block of query heads) costs its
// tiles (4 steps, one for each wavefront of a workgroup) plus one, and each
// workgroup takes an equal run of the rows' costs laid end to end: the
// merge-path split with rows and tiles as its units. Every workgroup finds its
// run by a scan over the requests' lengths, so there is no planning launch.
// Rows that a run cuts leave partial (m, l, o) in the workspace; the
// workgroup that adds the last part (a counter per row) joins them in the
// order of the row, so the bits do not depend on who is last.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "kv_internal.hpp"
#include "kv_types.hpp"

namespace spmv {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));

// Rows that a partial slot holds, and workgroups the workspace is laid out for.
constexpr int kKvMaxBlocks = 1024;

constexpr int kv_dim_pad(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// 16-row blocks of query heads one workgroup takes: two when a key head has
// more than 16 (each block beyond the first reads the cache's rows again
// otherwise); 32-bit rows would not leave registers for it.
constexpr int kv_row_blocks(int group, int cache_dtype) {
  return group > 16 && cache_dtype != SPMV_KV_F32 ? 2 : 1;
}
constexpr size_t kv_slot_floats(int nb, int dpad) { return (size_t)16 * nb * (dpad + 2); }
constexpr size_t kKvCounterBytes = kKvMaxBlocks * sizeof(int32_t);

#if defined(__HIP_DEVICE_COMPILE__)

// Maximum and sum over the four lanes that share a query column (c, c + 16,
// c + 32, c + 48).
__device__ __forceinline__ float column_max(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma32(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Two 8-bit values, the low or high half of a word, as a word of 16-bit ones.
template <bool HIGH>
__device__ __forceinline__ uint32_t widen2(uint32_t w, bf16) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}
template <bool HIGH>
__device__ __forceinline__ uint32_t widen2(uint32_t w, f16) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

// The weights p >= 0 of two tokens as 16-bit words. A single rounding of them
// would add as much error to a 16-bit result as its own rounding does, so
// they are carried in two parts: hi cut towards zero, lo the rest. The rest
// is never 0 but at least the smallest value of its type: an infinite value
// times a rest of 0 would turn a sum that is infinite into NaN.
__device__ __forceinline__ void split2(float p0, float p1, bf16, uint32_t& hi, uint32_t& lo) {
  const uint32_t a = __float_as_uint(p0), b = __float_as_uint(p1);
  hi = __builtin_amdgcn_perm(b, a, 0x07060302);
  const float tiny = 0x1p-120f;
  const bf16x2 r = {(bf16)fmaxf(p0 - __uint_as_float(a & 0xffff0000u), tiny),
                    (bf16)fmaxf(p1 - __uint_as_float(b & 0xffff0000u), tiny)};
  lo = __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ void split2(float p0, float p1, f16, uint32_t& hi, uint32_t& lo) {
  const f16x2 h = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(p0, p1));
  hi = __builtin_bit_cast(uint32_t, h);
  const float tiny = 0x1p-24f;
  const f16x2 r = {(f16)fmaxf(p0 - (float)h.x, tiny), (f16)fmaxf(p1 - (float)h.y, tiny)};
  lo = __builtin_bit_cast(uint32_t, r);
}

#endif  // __HIP_DEVICE_COMPILE__

// What one instantiation works with. C: cache, Q: queries and output.
template <typename C, typename Q, int DPAD, int NB>
struct KvShape {
  static constexpr bool F32 = sizeof(C) == 4, F8 = sizeof(C) == 1;
  static constexpr int TS = F32 ? 1 : 2;              // 16-token tiles per step
  static constexpr int ST = 16 * TS;                  // tokens per step
  static constexpr int KL = DPAD * sizeof(C) / 64;    // 16-byte loads of a key per lane
  // elements of a value one lane loads at a time, and how often
  static constexpr int EV = F8 ? DPAD / 16 : F32 ? 4 : (DPAD >= 128 ? 8 : 4);
  static constexpr int NC = DPAD / (16 * EV);
  static constexpr int VW = EV * sizeof(C) / 4;       // words of them
  static constexpr int NT = 4 * TS;                   // tokens whose values a lane loads
  static constexpr int QW = (F32 ? DPAD / 4 : DPAD / 8);   // words of queries per lane and block
  // the second product's 16-bit type; 8-bit values are exact in f16, whose 11
  // bits serve the weights of an output of 8 without a second part
  typedef typename std::conditional<F8, f16, C>::type P;
  static constexpr bool SPLIT = !F32 && !(F8 && std::is_same<Q, bf16>::value);
  // f16 weights span 2^-24 .. 2^15: the maximum is put at 2^14, so that what
  // is lost below lies 2^-38 under it
  static constexpr float TOP = std::is_same<P, f16>::value && !F32 ? 14.f : 0.f;
};

// Steps of a row: those of the first tokens that stay visible, then those of
// the window, in absolute numbers, so that a step's 16-token tiles begin at
// multiples of 16 and lie in one page when pages are multiples of 16 tokens.
struct KvSpan {
  int32_t n, from, first;    // tokens; visible: t >= from or t < first
  int32_t s0, s1, steps;     // step i of the row is i < s0 ? i : s1 + i - s0
};
template <int ST>
__device__ __forceinline__ KvSpan kv_span(const KvAttentionArgs& a, int r) {
  KvSpan x;
  x.n = min(max(a.lengths[r], 0), a.table_tokens);
  x.from = a.window && x.n > a.window ? x.n - a.window : 0;
  x.first = min(a.sinks, x.from);
  x.s0 = (int32_t)(((uint32_t)x.first + ST - 1) / ST);
  x.s1 = max(x.from / ST, x.s0);
  x.steps = x.s0 + (int32_t)(((uint32_t)x.n + ST - 1) / ST) - x.s1;
  return x;
}
__device__ __forceinline__ int32_t kv_tiles(const KvSpan& x) {
  return (x.steps + kWavesPerBlock - 1) / kWavesPerBlock;
}

// One workgroup's part of a row ready to be written or joined: m, l per row
// in LDS, o of each wavefront in LDS, scaled to the common maximum.
template <typename C, typename Q, int DPAD, int NB, bool EXACT, bool PAGED16, int OCC>
__global__ __launch_bounds__(kBlock, OCC) void kv_attention_kernel(KvAttentionArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef KvShape<C, Q, DPAD, NB> S;
  constexpr int ST = S::ST, TS = S::TS, ROWS = 16 * NB, PITCH = DPAD + 4;
  __shared__ __align__(16) float red[kWavesPerBlock][ROWS][PITCH];
  __shared__ float wave_m[kWavesPerBlock][ROWS], wave_l[kWavesPerBlock][ROWS];
  __shared__ int64_t scan[kWavesPerBlock];
  __shared__ int64_t found_before;
  __shared__ int32_t found_row, last_one;

  const int tid = threadIdx.x, lane = lane_id(), c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int D = a.head_dim;
  const int chunks = (a.group + ROWS - 1) / ROWS;
  const int heads = a.n_kv_heads * chunks;       // rows per request

  // ---- this workgroup's run of the rows' costs -------------------------------
  const int per_thread = (a.n_requests + kBlock - 1) / kBlock;
  const int r0 = min(tid * per_thread, a.n_requests);
  const int r1 = min(r0 + per_thread, a.n_requests);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += (int64_t)(kv_tiles(kv_span<ST>(a, r)) + 1) * heads;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t x = __shfl_up(incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == kWave - 1) scan[wave] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWavesPerBlock; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  per = per < a.min_share ? a.min_share : per;
  const int64_t d0 = (int64_t)blockIdx.x * per;
  if (d0 >= total) return;                       // the whole workgroup
  const int64_t d1 = d0 + per < total ? d0 + per : total;
  if (before <= d0 && d0 < before + mine) {
    int r = r0;
    for (;; ++r) {
      const int64_t cost = (int64_t)(kv_tiles(kv_span<ST>(a, r)) + 1) * heads;
      if (d0 < before + cost) break;
      before += cost;
    }
    found_row = r;
    found_before = before;
  }
  __syncthreads();
  int r = __builtin_amdgcn_readfirstlane(found_row);
  int64_t request_at = found_before;             // unit at which request r begins

  const float sc = a.scale * 1.44269504088896f;
  const int64_t k_token_b = a.k_token * (int64_t)sizeof(C), v_token_b = a.v_token * (int64_t)sizeof(C);

  for (;; ++r) {
    const KvSpan x = kv_span<ST>(a, r);
    const int32_t tiles = kv_tiles(x), cost = tiles + 1;
    int hc = d0 > request_at ? (int)((d0 - request_at) / cost) : 0;
    for (; hc < heads; ++hc) {
      // ---- the part of row (r, hc) in this run: tiles [ta, tb) ---------------
      const int64_t row_at = request_at + (int64_t)hc * cost;
      if (row_at >= d1) return;
      const int32_t ta = d0 > row_at ? (int32_t)(d0 - row_at) - 1 : 0;
      const int32_t tb = row_at + cost <= d1 ? tiles : (int32_t)(d1 - row_at) - 1;
      const int32_t ta0 = ta < 0 ? 0 : ta;
      if (tiles > 0 && tb <= ta0) continue;      // only the row's own unit: nothing to sum
      const bool whole = ta0 == 0 && tb == tiles;
      const int kh = hc / chunks, first_head = (hc - kh * chunks) * ROWS;
      const int rows = min(ROWS, a.group - first_head);
      const int64_t q_head0 = (int64_t)kh * a.group + first_head;

      // ---- queries: B operands, zero past the group's last head ---------------
      uint32_t qf[NB][S::QW];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int row = nb * 16 + c;
        const Q* qp = static_cast<const Q*>(a.q) + r * a.q_request + (q_head0 + row) * a.q_head;
        constexpr int W = 4;                     // words per load: 16 bytes of queries
        constexpr int E = 16 / sizeof(Q);
#pragma unroll
        for (int i = 0; i < S::QW / W; ++i) {
          // the elements that go with the i-th operand of a key
          const int d = S::F8 ? (i / 2) * 64 + g * 16 + (i & 1) * 8 : i * 4 * E + g * E;
          alignas(16) Q e[E] = {};
          if (row < rows && d < D) {
            if (a.q_aligned) {
              *reinterpret_cast<u32x4*>(e) = *reinterpret_cast<const u32x4*>(qp + d);
            } else {
#pragma unroll
              for (int j = 0; j < E; ++j) e[j] = qp[d + j];
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w) qf[nb][i * W + w] = reinterpret_cast<const uint32_t*>(e)[w];
        }
      }
      const float srow = a.k_scale ? sc * a.k_scale[kh] : sc;

      const char* kb = static_cast<const char*>(a.k) + kh * a.k_head * (int64_t)sizeof(C);
      const char* vb = static_cast<const char*>(a.v) + kh * a.v_head * (int64_t)sizeof(C);
      const int32_t* table = a.table + r * a.table_stride;

      uint32_t kr[TS][S::KL][4], vr[S::NT][S::NC][S::VW];
      // Loads of one step; returns the mask of its visible tokens (all zero past the row).
      struct Where {
        uint32_t mask;
        int64_t off[2];          // PAGED16: unused; else this lane's token's offsets in bytes
        const char* k[TS];
        const char* v[TS];
      };
      auto locate = [&](int32_t step) {
        Where w;
        const int32_t i = step < x.steps ? step : 0;
        const int32_t t0 = (i < x.s0 ? i : x.s1 + i - x.s0) * ST;
        if (PAGED16) {
          bool ok[TS];
#pragma unroll
          for (int ts = 0; ts < TS; ++ts) {
            const int32_t tt = t0 + 16 * ts;
            int32_t page = -1;
            const uint32_t j = div_by((uint32_t)tt, a.page);
            if (tt < x.n)
              page = __builtin_amdgcn_readfirstlane(table[j]);
            ok[ts] = (uint32_t)page < (uint32_t)a.n_pages;
            const int64_t p = ok[ts] ? page : 0, at = tt - (int32_t)(j * a.page.d);
            w.k[ts] = kb + (p * a.k_page + at * a.k_token) * (int64_t)sizeof(C);
            w.v[ts] = vb + (p * a.v_page + at * a.v_token) * (int64_t)sizeof(C);
          }
          const int32_t t = t0 + lane;
          bool see = lane < ST && t < x.n && (t >= x.from || t < x.first);
          see = see && (TS == 1 || lane < 16 ? ok[0] : ok[TS - 1]);
          w.mask = (uint32_t)__ballot(see);
        } else {
          const int32_t t = t0 + (lane & (ST - 1));
          bool see = t < x.n && (t >= x.from || t < x.first);
          int64_t page = 0, at = 0;
          if (see) {
            const uint32_t j = div_by((uint32_t)t, a.page);
            const int32_t p = table[j];
            see = (uint32_t)p < (uint32_t)a.n_pages;
            page = see ? p : 0;
            at = see ? t - (int32_t)(j * a.page.d) : 0;
          }
          w.off[0] = (page * a.k_page + at * a.k_token) * (int64_t)sizeof(C);
          w.off[1] = (page * a.v_page + at * a.v_token) * (int64_t)sizeof(C);
          w.mask = (uint32_t)(__ballot(see) & ((uint64_t(1) << ST) - 1));
        }
        if (step >= x.steps) w.mask = 0;
        return w;
      };
      auto load_k = [&](const Where& w) {
#pragma unroll
        for (int ts = 0; ts < TS; ++ts) {
          const char* p;
          if (PAGED16)
            p = w.k[ts] + (uint32_t)(c * (int32_t)k_token_b + g * 16);
          else
            p = kb + __shfl(w.off[0], ts * 16 + c) + g * 16;
#pragma unroll
          for (int i = 0; i < S::KL; ++i) {
            if (EXACT || i * (64 / (int)sizeof(C)) + g * (16 / (int)sizeof(C)) < D) {
              const u32x4 v = *reinterpret_cast<const u32x4*>(p + i * 64);
#pragma unroll
              for (int e = 0; e < 4; ++e) kr[ts][i][e] = v[e];
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) kr[ts][i][e] = 0;
            }
          }
        }
      };
      auto load_v = [&](const Where& w) {
#pragma unroll
        for (int t = 0; t < S::NT; ++t) {
          const char* p;
          if (PAGED16)
            p = w.v[t / 4] + (uint32_t)((g * 4 + t % 4) * (int32_t)v_token_b + c * S::VW * 4);
          else
            p = vb + __shfl(w.off[1], t / 4 * 16 + g * 4 + t % 4) + c * S::VW * 4;
#pragma unroll
          for (int n = 0; n < S::NC; ++n) {
            if (EXACT || n * 16 * S::EV + c * S::EV < D) {
              if constexpr (S::VW == 4) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(p + n * 16 * S::VW * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) vr[t][n][e] = v[e];
              } else if constexpr (S::VW == 2) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(p + n * 16 * S::VW * 4);
                vr[t][n][0] = v[0];
                vr[t][n][1] = v[1];
              } else {
                vr[t][n][0] = *reinterpret_cast<const uint32_t*>(p + n * 16 * S::VW * 4);
              }
            } else {
#pragma unroll
              for (int e = 0; e < S::VW; ++e) vr[t][n][e] = 0;
            }
          }
        }
      };

      float m[NB], l[NB];
      f32x4 acc[NB][S::NC][S::EV];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb] = -INFINITY;
        l[nb] = 0.f;
#pragma unroll
        for (int n = 0; n < S::NC; ++n)
#pragma unroll
          for (int e = 0; e < S::EV; ++e) acc[nb][n][e] = f32x4{0.f, 0.f, 0.f, 0.f};
      }

      const int32_t step_end = min(tb * kWavesPerBlock, x.steps);
      int32_t step = ta0 * kWavesPerBlock + wave;
      if (step < step_end) {
        Where now = locate(step);
        load_k(now);
        load_v(now);
        for (;;) {
          const int32_t next = step + kWavesPerBlock;
          const bool more = next < step_end;
          const Where then = locate(more ? next : step);

          // S = K Q^T: score of token 16 ts + 4g + i with query column c
          f32x4 s[NB][TS];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int ts = 0; ts < TS; ++ts) s[nb][ts] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ts = 0; ts < TS; ++ts) {
#pragma unroll
            for (int i = 0; i < S::KL; ++i) {
              if constexpr (S::F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb)
                    s[nb][ts] = mfma4(__uint_as_float(kr[ts][i][e]),
                                      __uint_as_float(qf[nb][i * 4 + e]), s[nb][ts]);
              } else if constexpr (S::F8) {
                typedef Q X8 __attribute__((ext_vector_type(8)));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const u32x4 k8 = {widen2<false>(kr[ts][i][2 * h], Q()),
                                    widen2<true>(kr[ts][i][2 * h], Q()),
                                    widen2<false>(kr[ts][i][2 * h + 1], Q()),
                                    widen2<true>(kr[ts][i][2 * h + 1], Q())};
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    const uint32_t* q4 = &qf[nb][(2 * i + h) * 4];
                    const u32x4 q8 = {q4[0], q4[1], q4[2], q4[3]};
                    s[nb][ts] = mfma32(__builtin_bit_cast(X8, k8), __builtin_bit_cast(X8, q8),
                                       s[nb][ts]);
                  }
                }
              } else {
                typedef C X8 __attribute__((ext_vector_type(8)));
                const u32x4 k8 = {kr[ts][i][0], kr[ts][i][1], kr[ts][i][2], kr[ts][i][3]};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  const uint32_t* q4 = &qf[nb][i * 4];
                  const u32x4 q8 = {q4[0], q4[1], q4[2], q4[3]};
                  s[nb][ts] = mfma32(__builtin_bit_cast(X8, k8), __builtin_bit_cast(X8, q8),
                                     s[nb][ts]);
                }
              }
            }
          }
          if (more) load_k(then);

          const bool full = now.mask == (ST == 32 ? 0xffffffffu : 0xffffu);
          // bit 16 ts + i: this lane's token of tile ts is visible
          const uint32_t vis = full ? 0xffffffffu : now.mask >> (4 * g);
          float p[NB][TS][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float top = -INFINITY;
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float y = s[nb][ts][i] * srow;
                p[nb][ts][i] = vis >> (16 * ts + i) & 1 ? y : -INFINITY;
                top = fmaxf(top, p[nb][ts][i]);
              }
            top = column_max(top);
            // the reference point: TOP under the largest score so far (0 while
            // there is none, so that no difference of infinities arises)
            const float m_new = fmaxf(m[nb], top - S::TOP);
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float keep = __builtin_amdgcn_exp2f(m[nb] - base);
            m[nb] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int ts = 0; ts < TS; ++ts)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                p[nb][ts][i] = __builtin_amdgcn_exp2f(p[nb][ts][i] - base);
                sum += p[nb][ts][i];
              }
            l[nb] = l[nb] * keep + sum;
            if (!__all(keep == 1.f)) {
#pragma unroll
              for (int n = 0; n < S::NC; ++n)
#pragma unroll
                for (int e = 0; e < S::EV; ++e) acc[nb][n][e] *= keep;
            }
          }

          // values of tokens that are not visible are taken out, whatever they hold
          if (!full) {
#pragma unroll
            for (int t = 0; t < S::NT; ++t)
#pragma unroll
              for (int n = 0; n < S::NC; ++n)
#pragma unroll
                for (int e = 0; e < S::VW; ++e)
                  vr[t][n][e] = vis >> (16 * (t / 4) + t % 4) & 1 ? vr[t][n][e] : 0;
          }

          // O^T += V^T P^T
          if constexpr (S::F32) {
#pragma unroll
            for (int t = 0; t < S::NT; ++t)
#pragma unroll
              for (int n = 0; n < S::NC; ++n)
#pragma unroll
                for (int e = 0; e < S::EV; ++e)
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb)
                    acc[nb][n][e] = mfma4(__uint_as_float(vr[t][n][e]), p[nb][t / 4][t % 4],
                                          acc[nb][n][e]);
          } else {
            typedef typename S::P P;
            typedef P X8 __attribute__((ext_vector_type(8)));
            X8 hi[NB], lo[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              u32x4 h, o;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float x0 = p[nb][w / 2][2 * (w % 2)], x1 = p[nb][w / 2][2 * (w % 2) + 1];
                if constexpr (S::SPLIT) {
                  uint32_t hw, lw;
                  split2(x0, x1, P(), hw, lw);
                  h[w] = hw;
                  o[w] = lw;
                } else {
                  const f16x2 r2 = {(f16)x0, (f16)x1};
                  h[w] = __builtin_bit_cast(uint32_t, r2);
                }
              }
              hi[nb] = __builtin_bit_cast(X8, h);
              if constexpr (S::SPLIT) lo[nb] = __builtin_bit_cast(X8, o);
            }
            auto product = [&](int n, int e, u32x4 v8) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                acc[nb][n][e] = mfma32(__builtin_bit_cast(X8, v8), hi[nb], acc[nb][n][e]);
                if constexpr (S::SPLIT)
                  acc[nb][n][e] = mfma32(__builtin_bit_cast(X8, v8), lo[nb], acc[nb][n][e]);
              }
            };
#pragma unroll
            for (int n = 0; n < S::NC; ++n)
#pragma unroll
              for (int wd = 0; wd < S::VW; ++wd) {
                if constexpr (S::F8) {
                  // word wd: elements 4 wd .. 4 wd + 3 of each token
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    uint32_t pair[4];            // bytes: t, t+1 of element 2h, then of 2h + 1
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                      pair[t] = __builtin_amdgcn_perm(vr[2 * t + 1][n][wd], vr[2 * t][n][wd],
                                                      h ? 0x07030602 : 0x05010400);
                    product(n, 4 * wd + 2 * h,
                            u32x4{widen2<false>(pair[0], f16()), widen2<false>(pair[1], f16()),
                                  widen2<false>(pair[2], f16()), widen2<false>(pair[3], f16())});
                    product(n, 4 * wd + 2 * h + 1,
                            u32x4{widen2<true>(pair[0], f16()), widen2<true>(pair[1], f16()),
                                  widen2<true>(pair[2], f16()), widen2<true>(pair[3], f16())});
                  }
                } else {
                  // word wd: elements 2 wd, 2 wd + 1
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    u32x4 v8;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                      v8[t] = __builtin_amdgcn_perm(vr[2 * t + 1][n][wd], vr[2 * t][n][wd],
                                                    h ? 0x07060302 : 0x05040100);
                    product(n, 2 * wd + h, v8);
                  }
                }
              }
          }
          if (!more) break;
          load_v(then);
          now = then;
          step = next;
        }
      }

      // ---- the four wavefronts' parts to a common maximum ---------------------
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float sum = column_sum(l[nb]);
        if (g == 0) {
          wave_m[wave][nb * 16 + c] = m[nb];
          wave_l[wave][nb * 16 + c] = sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int row = nb * 16 + c;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWavesPerBlock; ++w) top = fmaxf(top, wave_m[w][row]);
        const float keep = __builtin_amdgcn_exp2f(m[nb] - (top == -INFINITY ? 0.f : top));
        if (row < rows) {
#pragma unroll
          for (int n = 0; n < S::NC; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < S::EV; e += 4) {
                const f32x4 o = {acc[nb][n][e][i] * keep, acc[nb][n][e + 1][i] * keep,
                                 acc[nb][n][e + 2][i] * keep, acc[nb][n][e + 3][i] * keep};
                *reinterpret_cast<f32x4*>(
                    &red[wave][row][n * 16 * S::EV + (g * 4 + i) * S::EV + e]) = o;
              }
        }
      }
      __syncthreads();

      // m, l of a row over the workgroup; o of its elements d .. d + 3
      auto row_m = [&](int row) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWavesPerBlock; ++w) top = fmaxf(top, wave_m[w][row]);
        return top;
      };
      auto row_l = [&](int row, float top) {
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWavesPerBlock; ++w)
          sum += wave_l[w][row] * __builtin_amdgcn_exp2f(wave_m[w][row] - base);
        return sum;
      };
      auto row_o = [&](int row, int d) {
        f32x4 o = *reinterpret_cast<const f32x4*>(&red[0][row][d]);
#pragma unroll
        for (int w = 1; w < kWavesPerBlock; ++w)
          o += *reinterpret_cast<const f32x4*>(&red[w][row][d]);
        return o;
      };
      const float vscale = a.v_scale ? a.v_scale[kh] : 1.f;
      auto write = [&](int row, int d, f32x4 o, float top, float sum) {
        Q* out = static_cast<Q*>(a.out) + r * a.out_request + (q_head0 + row) * a.out_head + d;
        const float inv = sum == 0.f ? 0.f : vscale / sum;
        alignas(16) Q y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = from_f32<Q>(sum == 0.f ? 0.f : o[e] * inv);
        if (a.out_aligned) {
          if constexpr (sizeof(Q) == 4)
            *reinterpret_cast<u32x4*>(out) = *reinterpret_cast<const u32x4*>(y);
          else
            *reinterpret_cast<u32x2*>(out) = *reinterpret_cast<const u32x2*>(y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = y[e];
        }
        if (a.lse && d == 0)
          a.lse[(int64_t)r * a.n_kv_heads * a.group + q_head0 + row] =
              sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
      };
      const int quads = D / 4;
      if (whole) {
        for (int i = tid; i < rows * quads; i += kBlock) {
          const int row = i / quads, d = (i - row * quads) * 4;
          const float top = row_m(row);
          write(row, d, row_o(row, d), top, row_l(row, top));
        }
      } else {
        // slot 2b: workgroup b's part of a row that began before it; 2b + 1: of one that
        // goes on after it
        int32_t* counters = static_cast<int32_t*>(a.workspace);
        float* slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kKvCounterBytes);
        constexpr int64_t SLOT = (int64_t)kv_slot_floats(NB, DPAD);
        const int64_t b0 = (row_at + 1) / per, b1 = (row_at + cost - 1) / per;   // first, last part
        auto slot_of = [&](int64_t b) { return slots + (2 * b + (b == b0 ? 1 : 0)) * SLOT; };
        float* slot = slot_of(blockIdx.x);
        for (int i = tid; i < rows * quads; i += kBlock) {
          const int row = i / quads, d = (i - row * quads) * 4;
          *reinterpret_cast<f32x4*>(slot + 2 * ROWS + row * DPAD + d) = row_o(row, d);
          if (d == 0) {
            const float top = row_m(row);
            slot[row] = top;
            slot[ROWS + row] = row_l(row, top);
          }
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int32_t seen = __hip_atomic_fetch_add(counters + b0, 1, __ATOMIC_ACQ_REL,
                                                      __HIP_MEMORY_SCOPE_AGENT);
          last_one = seen == (int32_t)(b1 - b0);
          // the next call finds it as this one did
          if (last_one) __hip_atomic_store(counters + b0, 0, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (last_one) {
          __threadfence();
          for (int i = tid; i < rows * quads; i += kBlock) {
            const int row = i / quads, d = (i - row * quads) * 4;
            float top = -INFINITY;
            for (int64_t b = b0; b <= b1; ++b) top = fmaxf(top, slot_of(b)[row]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int64_t b = b0; b <= b1; ++b) {
              const float* s = slot_of(b);
              const float w = __builtin_amdgcn_exp2f(s[row] - base);
              sum += s[ROWS + row] * w;
              o += *reinterpret_cast<const f32x4*>(s + 2 * ROWS + row * DPAD + d) * w;
            }
            write(row, d, o, top, sum);
          }
        }
      }
      __syncthreads();                           // red, wave_m and last_one are free again
    }
    request_at += (int64_t)cost * heads;
    if (request_at >= d1 || r + 1 >= a.n_requests) return;
  }
#endif
}

// How many workgroups of one instantiation a CU holds: what its registers and
// LDS leave.
template <typename C, int DPAD, int NB>
constexpr int kv_occupancy() {
  return NB == 2 ? (DPAD == 256 ? 1 : 2) : DPAD == 256 || (sizeof(C) == 4 && DPAD > 64) ? 1 : 2;
}

template <typename C, typename Q, int DPAD, int NB>
hipError_t launch_kv_attention_shape(const KvAttentionArgs& a, hipStream_t s) {
  constexpr int OCC = kv_occupancy<C, DPAD, NB>();
  const int chunks = (a.group + 16 * NB - 1) / (16 * NB);
  // no more workgroups than units: tiles at the table's full width, and one a row
  const int64_t steps = a.table_tokens / KvShape<C, Q, DPAD, NB>::ST + 3;
  const int64_t units = (int64_t)a.n_requests * a.n_kv_heads * chunks * (steps / 4 + 2);
  const int64_t most = (int64_t)a.n_cus * OCC < kKvMaxBlocks ? a.n_cus * OCC : kKvMaxBlocks;
  const int64_t want = (units + a.min_share - 1) / a.min_share;
  const unsigned blocks = (unsigned)(want < most ? want : most);
  // one page for each 16 tokens, and lane offsets within them in 32 bits
  const bool paged16 = a.page.d % 16 == 0 && a.k_token < (int64_t(1) << 24) &&
                       a.v_token < (int64_t(1) << 24);
  if (!paged16)
    hipLaunchKernelGGL((kv_attention_kernel<C, Q, DPAD, NB, false, false, OCC>), dim3(blocks),
                       dim3(kBlock), 0, s, a);
  else if (a.head_dim == DPAD)
    hipLaunchKernelGGL((kv_attention_kernel<C, Q, DPAD, NB, true, true, OCC>), dim3(blocks),
                       dim3(kBlock), 0, s, a);
  else
    hipLaunchKernelGGL((kv_attention_kernel<C, Q, DPAD, NB, false, true, OCC>), dim3(blocks),
                       dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <typename C, typename Q, int NB>
hipError_t launch_kv_attention_dim(const KvAttentionArgs& a, hipStream_t s) {
  switch (kv_dim_pad(a.head_dim)) {
    case 64: return launch_kv_attention_shape<C, Q, 64, NB>(a, s);
    case 128: return launch_kv_attention_shape<C, Q, 128, NB>(a, s);
    default: return launch_kv_attention_shape<C, Q, 256, NB>(a, s);
  }
}

}  // namespace spmv
