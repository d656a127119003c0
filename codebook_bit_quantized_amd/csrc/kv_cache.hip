// The 4-bit key/value cache: a step's keys and values quantised into it, and read back.
//
// L lanes hold a head: channel 8Lj + 8l + i is value 8j + i of lane l, so that for each j the lanes' 16 bytes of bf16 are
// contiguous, and the transform is the stages of i and j in registers and log2(L) stages between lanes, DPP moves and
// swizzles: no LDS memory.  Four lanes for many heads, as a stage between lanes costs three instructions a value and one
// in registers one; D/8 lanes for few, as a lane's chain is then shorter.  Reading D = 128 takes eight lanes for many heads:
// each store then fills lines of 128 bytes (65536 tokens of 4 heads 31 us a call, with four lanes 44; writing the cache with
// eight 28 against 26 us, 16384 tokens of 8 heads).  The transform to be quantised is in fp64, as in cbq_rotate_quantize:
// exact, so a code does not depend on the order of its sums; reading back needs fp32 only, as sums of at most 128
// multiples of 1/2 up to 6 are exact there.
// A workgroup takes the heads of some consecutive tokens; their places (sequence, length, page: four dependent
// loads) are looked up once, by a lane each, and handed over in LDS.
//
// What bounds it.  Writing: 16384 tokens of 8 heads take 26 us, 17 not rotated, and 25 as torch's copy of the same rows;
// 65536 take 92, 84 and 101.  Rotated on the matrix cores (two products of exact fp32 sums, the values that lie 8 binades below
// their head's largest apart) they took 27 and 96: what it saved in fp64 instructions went into the exchange of lanes and
// fewer waves.  Reading: HBM (65536 tokens of 4 heads, 170 MB in 31 us, 5.5 TB/s of which four fifths are written).  A call
// for one token takes 3 us, the chain of its loads.
#include "kv_device.hpp"

namespace cbq {
namespace {

constexpr int kMaxTokens = 64;                          // tokens a workgroup takes at most

// Row index of head 0 at each token's place: kNowhere where it has none, kNobody where it has no sequence.
constexpr int64_t kNowhere = -1, kNobody = -2;

__device__ __forceinline__ void find_places(const KvArgs& a, int64_t t0, int tokens, int64_t* place) {
  if ((int)threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    const int b = kv_seq_of(a, t);
    int64_t at = kNobody;
    if (b >= 0) {
      const int64_t pos = kv_position(a, b, t);
      const int page = pos < 0 ? -1 : kv_page(a, b, pos);
      at = page < 0 ? kNowhere : kv_row(a, page, 0, pos);
    }
    place[threadIdx.x] = at;
  }
}

// v / s from y = RN(1 / s): the quotient's remainder is exact, and one step of it corrects the rounding (Markstein).  So it
// is v / s rounded to nearest for every mantissa of s and every v whose quotient lies next to a border of the codes, which is what
// they depend on.  y: one such step from the hardware's reciprocal, which is within one step of 1 / s.  That gives RN(1 / s) from
// any such start, but for a mantissa of ones: there from RN(1 / s) alone, which is what the hardware returns for it.  (All of it
// checked for every mantissa.)  For s and v / s away from the ends of the exponent range.
__device__ __forceinline__ float div_by(float v, float s, float y) {
  const float q = v * y;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, v), y, q), v);   // -0 stays -0
}

template <int D, int L>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a, const uint16_t* k, int64_t ldk, const uint16_t* v,
                                                       int64_t ldv, int64_t t0, int per, float c_b) {
  constexpr int C = D / L, J = C / 8, R = 256 / L;      // values a lane, runs of 8 of them, heads at a time
  __shared__ int64_t place[kMaxTokens];
  const int which = blockIdx.y, lane = threadIdx.x % L;
  t0 += (int64_t)blockIdx.x * per;
  const int tokens = (int)min((int64_t)per, a.T - t0), rows = tokens * a.n_kv;
  const uint16_t* src = which ? v : k;
  const int64_t ld = which ? ldv : ldk;
  const bool rot = (a.rotate >> which) & 1;
  u32x4 next[J];
  auto fetch = [&](int r) {
    if (r >= rows) return;                              // whole groups of lanes
    const int t = (int)((uint32_t)r / (uint32_t)a.n_kv);
    const uint16_t* p = src + (t0 + t) * ld + (r - t * a.n_kv) * D + 8 * lane;
#pragma unroll
    for (int j = 0; j < J; ++j) next[j] = *reinterpret_cast<const u32x4*>(p + 8 * L * j);
  };
  fetch(threadIdx.x / L);                              // on their way while the places are looked up
  find_places(a, t0, tokens, place);
  __syncthreads();
  for (int r = threadIdx.x / L; r < rows; r += R) {
    const int t = (int)((uint32_t)r / (uint32_t)a.n_kv), head = r - t * a.n_kv;
    u32x4 in[J];
#pragma unroll
    for (int j = 0; j < J; ++j) in[j] = next[j];
    fetch(r + R);
    const int64_t at = place[t];
    if (at < 0) continue;
    float f[C];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[8 * j + 2 * i] = __builtin_bit_cast(float, in[j][i] << 16);
        f[8 * j + 2 * i + 1] = __builtin_bit_cast(float, in[j][i] & 0xFFFF0000u);
      }
    if (rot) {
      double u[C];
#pragma unroll
      for (int i = 0; i < C; ++i) u[i] = f[i];
      kv_reg_stages<C>(u, 1, C);
      kv_lane_stages<L, C>(u, lane);
#pragma unroll
      for (int i = 0; i < C; ++i) f[i] = (float)u[i];
    }
    // the maximum over bit patterns: a float maximum would drop a NaN
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) m = max(m, __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)xor_lane<1>((int)m));
    m = max(m, (uint32_t)xor_lane<2>((int)m));
    if constexpr (L > 4) m = max(m, (uint32_t)xor_lane<4>((int)m));
    if constexpr (L > 8) m = max(m, (uint32_t)xor_lane<8>((int)m));
    const float s = __builtin_bit_cast(float, m) / 6.0f;
    float r8[C];
    if (s >= 0x1p-60f && s <= 0x1p60f) {
      const float y0 = __builtin_amdgcn_rcpf(s), y = __builtin_fmaf(__builtin_fmaf(-s, y0, 1.0f), y0, y0);
#pragma unroll
      for (int i = 0; i < C; ++i) r8[i] = div_by(f[i], s, y);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) r8[i] = f[i] / s;
    }
    const int64_t row = at + ((int64_t)head << a.logp);
    uint8_t* dst = a.codes[which] + row * (D / 2) + 4 * lane;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r8[8 * j], r8[8 * j + 1], 1.0f, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r8[8 * j + 2], r8[8 * j + 3], 1.0f, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r8[8 * j + 4], r8[8 * j + 5], 1.0f, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r8[8 * j + 6], r8[8 * j + 7], 1.0f, 3);
      *reinterpret_cast<uint32_t*>(dst + 4 * L * j) = s == 0.0f ? 0u : c;
    }
    if (lane == 0) a.scales[which][row] = rot ? s * c_b : s;
  }
}

template <int D, int L>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                                                      int first, int64_t t0, int per, float c_b) {
  constexpr int C = D / L, J = C / 8, R = 256 / L;
  __shared__ int64_t place[kMaxTokens];
  const int which = first + blockIdx.y, lane = threadIdx.x % L;
  t0 += (int64_t)blockIdx.x * per;
  const int tokens = (int)min((int64_t)per, a.T - t0), rows = tokens * a.n_kv;
  uint16_t* out = which ? v : k;
  const int64_t ld = which ? ldv : ldk;
  const bool rot = (a.rotate >> which) & 1;
  find_places(a, t0, tokens, place);
  __syncthreads();
  for (int r = threadIdx.x / L; r < rows; r += R) {
    const int t = (int)((uint32_t)r / (uint32_t)a.n_kv), head = r - t * a.n_kv;
    const int64_t at = place[t];
    if (at == kNobody) continue;                        // whole groups of lanes
    float f[C];
    float s = 0;
    if (at >= 0) {
      const int64_t row = at + ((int64_t)head << a.logp);
      const uint8_t* src = a.codes[which] + row * (D / 2) + 4 * lane;
      s = a.scales[which][row];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(src + 4 * L * j);
        const f16x2 p0 = e2m1_pair<0>(c), p1 = e2m1_pair<1>(c), p2 = e2m1_pair<2>(c), p3 = e2m1_pair<3>(c);
        f[8 * j] = (float)p0[0]; f[8 * j + 1] = (float)p0[1]; f[8 * j + 2] = (float)p1[0]; f[8 * j + 3] = (float)p1[1];
        f[8 * j + 4] = (float)p2[0]; f[8 * j + 5] = (float)p2[1]; f[8 * j + 6] = (float)p3[0]; f[8 * j + 7] = (float)p3[1];
      }
      if (rot) {
        kv_reg_stages<C>(f, 1, C);
        kv_lane_stages<L, C>(f, lane);
        s *= c_b;
      }
    }
    uint16_t* dst = out + (t0 + t) * ld + head * D + 8 * lane;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      u32x4 x = {0, 0, 0, 0};
      if (at >= 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = (uint32_t)f32_to_bf16_rne(f[8 * j + 2 * i] * s) | ((uint32_t)f32_to_bf16_rne(f[8 * j + 2 * i + 1] * s) << 16);
      __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(dst + 8 * L * j));   // past the caches: 54 us a call with ordinary stores, 65536 tokens, 42 so
    }
  }
}

// Launches over all tokens, `per` to a workgroup: as many as give it 256 heads, fewer where that leaves the chip idle.
template <typename F>
hipError_t over_tokens(const KvArgs& a, F launch) {
  int per = 256 / a.n_kv;
  per = per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per;
  while (per > 1 && a.T / per < 256) per /= 2;
  const int64_t most = int64_t(1) << 23;                // workgroups of a launch
  for (int64_t t0 = 0; t0 < a.T; t0 += most * per) {
    const int64_t left = (a.T - t0 + per - 1) / per;
    launch(t0, per, (uint32_t)(left < most ? left : most));
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

// Few heads: a lane holds 8 channels of one, else 4 or 8 lanes hold it (see the top).  Few and many lanes, D = 128, tokens of 8
// heads: write 1 token 3.4 and 4.3 us, 1024 5.5 and 5.5, 2048 8.1 and 6.0, 4096 13.6 and 9.7; read 1 3.0 and 3.1, 512 4.0 and
// 4.2, 1024 4.9 and 4.6, 2048 7.0 and 5.6, 16384 25.8 and 18.8.
bool few_heads(const KvArgs& a) { return a.T * a.n_kv <= 8192; }

}  // namespace

hipError_t launch_kv_write(const KvArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                           hipStream_t stream) {
  const float c_b = (float)(1.0 / std::sqrt((double)a.D));
  auto f = a.D == 64 ? few_heads(a) ? kv_write_kernel<64, 8> : kv_write_kernel<64, 4>
                     : few_heads(a) ? kv_write_kernel<128, 16> : kv_write_kernel<128, 4>;
  return over_tokens(a, [&](int64_t t0, int per, uint32_t blocks) {
    f<<<dim3(blocks, 2), 256, 0, stream>>>(a, k, ldk, v, ldv, t0, per, c_b);
  });
}

hipError_t launch_kv_read(const KvArgs& a, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv, hipStream_t stream) {
  const float c_b = (float)(1.0 / std::sqrt((double)a.D));
  auto f = a.D == 64 ? few_heads(a) ? kv_read_kernel<64, 8> : kv_read_kernel<64, 4>
                     : few_heads(a) ? kv_read_kernel<128, 16> : kv_read_kernel<128, 8>;
  return over_tokens(a, [&](int64_t t0, int per, uint32_t blocks) {
    f<<<dim3(blocks, k && v ? 2 : 1), 256, 0, stream>>>(a, k, ldk, v, ldv, k ? 0 : 1, t0, per, c_b);
  });
}

}  // namespace cbq
