// What the kernels of the 4-bit key/value cache share: the places of a step's tokens, E2M1
// codes, and a head's rotation over the lanes that hold it.
#pragma once
#include "cbq_internal.hpp"
#include "rotate_device.hpp"

namespace cbq {

// Sequence of token t (offsets ascending), or -1: the last b with offsets[b] <= t, where t
// comes before offsets[b+1].  Any offsets give a b in [0, B) or -1.
__device__ __forceinline__ int kv_seq_of(const KvArgs& a, int64_t t) {
  if (!a.offsets) return (int)((uint32_t)t / (uint32_t)a.per_seq);
  int lo = 0, hi = a.B;                    // offsets[lo] <= t < offsets[hi], if at all
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= t) lo = mid; else hi = mid;
  }
  return a.offsets[lo] <= t && t < a.offsets[lo + 1] ? lo : -1;
}

// Position of token t of sequence b.
__device__ __forceinline__ int64_t kv_position(const KvArgs& a, int b, int64_t t) {
  const int64_t end = a.offsets ? (int64_t)a.offsets[b + 1] : (int64_t)(b + 1) * a.per_seq;
  return (int64_t)a.lens[b] - end + t;
}

// Page of position pos >= 0 of sequence b, or -1.
__device__ __forceinline__ int kv_page(const KvArgs& a, int b, int64_t pos) {
  const int64_t j = pos >> a.logp;
  if (j >= a.max_pages) return -1;
  const int p = a.table ? a.table[(int64_t)b * a.ld_table + j] : (int)(b * (int64_t)a.max_pages + j);
  return (uint32_t)p < (uint32_t)a.n_pages ? p : -1;
}

// Index of (page, head, place) among the cache's rows of D channels.
__device__ __forceinline__ int64_t kv_row(const KvArgs& a, int page, int head, int64_t pos) {
  return (((int64_t)page * a.n_kv + head) << a.logp) + (pos & ((1 << a.logp) - 1));
}

// Two E2M1 codes (byte SEL of x, low nibble first) as fp16, exact.
template <int SEL>
__device__ __forceinline__ f16x2 e2m1_pair(uint32_t x) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, SEL));
}

template <int M, typename T>
__device__ __forceinline__ T kv_xor_lane(T v) {
  if constexpr (sizeof(T) == 8) return xor_lane_f64<M>(v);
  else return xor_lane_f32<M>(v);
}

// One butterfly stage of N values a lane with the lane M away: v + p in the lower lane, p - v in the
// upper, as one fma by +-1 (an exact product; hidden from the compiler, which would select between two adds).
template <int M, int N, typename T>
__device__ __forceinline__ void kv_lane_stage(T* v, int lane) {
  T sgn = (lane & M) ? (T)-1 : (T)1;
  asm("" : "+v"(sgn));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const T p = kv_xor_lane<M>(v[i]);
    if constexpr (sizeof(T) == 8) v[i] = __builtin_fma(v[i], sgn, p);
    else v[i] = __builtin_fmaf(v[i], sgn, p);
  }
}

// Butterfly stages over the low bits of the index of N values in a lane, N = 2^k: strides from, 2 from, ... below to.
template <int N, typename T>
__device__ __forceinline__ void kv_reg_stages(T* v, int from, int to) {
#pragma unroll
  for (int h = 1; h < N; h *= 2) {
    if (h < from || h >= to) continue;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & h)) {
        const T x = v[i], y = v[i + h];
        v[i] = x + y;
        v[i + h] = x - y;
      }
  }
}

// The stages between L neighbouring lanes.
template <int L, int N, typename T>
__device__ __forceinline__ void kv_lane_stages(T* v, int lane) {
  kv_lane_stage<1, N>(v, lane);
  kv_lane_stage<2, N>(v, lane);
  if constexpr (L > 4) kv_lane_stage<4, N>(v, lane);
  if constexpr (L > 8) kv_lane_stage<8, N>(v, lane);
}

// Transform of D channels that lie 8 to a lane in D/8 lanes.
template <int D, typename T>
__device__ __forceinline__ void kv_transform(T* v, int lane) {
  kv_reg_stages<8>(v, 1, 8);
  kv_lane_stages<D / 8, 8>(v, lane);
}

}  // namespace cbq
