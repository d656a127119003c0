// Lane exchanges and butterfly stages of the block Walsh-Hadamard transform (gfx950, wave64),
// shared by the kernels that rotate and quantise activations.
#pragma once
#include "cbq_device.hpp"

namespace cbq {

// value of lane (lane ^ M), M a power of two below 64
template <int M>
__device__ __forceinline__ int xor_lane(int v) {
  if constexpr (M == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);    // quad_perm 1,0,3,2
  else if constexpr (M == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);  // quad_perm 2,3,0,1
  else if constexpr (M == 4) return __builtin_amdgcn_ds_swizzle(v, 0x101F);              // xor 4 in 32 lanes
  else if constexpr (M == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, false); // row_ror 8
  else if constexpr (M == 16) return __builtin_amdgcn_ds_swizzle(v, 0x401F);             // xor 16 in 32 lanes
  else return __shfl_xor(v, 32);
}

template <int M>
__device__ __forceinline__ double xor_lane_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)xor_lane<M>((int)(uint32_t)b);
  const uint32_t hi = (uint32_t)xor_lane<M>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int M>
__device__ __forceinline__ float xor_lane_f32(float v) {
  return __builtin_bit_cast(float, xor_lane<M>(__builtin_bit_cast(int, v)));
}

// one butterfly stage between lanes j and j ^ M (M lanes = N * M channels apart): the
// lower lane keeps v + p, the upper one v - p, which is the negative of the butterfly's
// p - v.  Each value is one fma(p, +-1, v) accumulating into v (the product by +-1 is
// exact, so it rounds the same sum an add would).  Partners always carry the same sign
// (they differ only in the stage's own lane bit), so after the lane stages a lane's
// values are the transform times (-1)^(number of upper stages), i.e. the parity of its
// lane bits inside the block; the quantiser takes that sign into its multiplier.
template <int M, int N = 32>
__device__ __forceinline__ void lane_stage(double* v, bool upper) {
  const double sgn = upper ? -1.0 : 1.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double p = xor_lane_f64<M>(v[i]);
    v[i] = __builtin_fma(p, sgn, v[i]);
  }
}

// Exchange between 16-lane rows: a pair (A, B) of one lane and the pair of the lane 16
// (SWAP32: 32) lanes away.  The lane in the even row (lower half) gets its partner's A in
// place of its own B; the partner gets this lane's B in place of its own A.  Each lane then
// holds (A of the even-row lane, A or B of the odd-row lane at the same place) and both
// compute the butterfly (A + B, A - B) in the same registers.
template <bool SWAP32>
__device__ __forceinline__ void swap_butterfly(double& a, double& b) {
  const uint64_t ua = __builtin_bit_cast(uint64_t, a), ub = __builtin_bit_cast(uint64_t, b);
  uint32_t alo = (uint32_t)ua, ahi = (uint32_t)(ua >> 32);
  uint32_t blo = (uint32_t)ub, bhi = (uint32_t)(ub >> 32);
  if constexpr (SWAP32) {
    const auto lo = __builtin_amdgcn_permlane32_swap(alo, blo, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(ahi, bhi, false, false);
    alo = lo[0]; blo = lo[1]; ahi = hi[0]; bhi = hi[1];
  } else {
    const auto lo = __builtin_amdgcn_permlane16_swap(alo, blo, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(ahi, bhi, false, false);
    alo = lo[0]; blo = lo[1]; ahi = hi[0]; bhi = hi[1];
  }
  const double A = __builtin_bit_cast(double, ((uint64_t)ahi << 32) | alo);
  const double B = __builtin_bit_cast(double, ((uint64_t)bhi << 32) | blo);
  a = A + B;
  b = A - B;
}

}  // namespace cbq
