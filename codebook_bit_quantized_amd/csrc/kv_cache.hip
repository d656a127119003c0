// The 4-bit key/value cache: a step's keys and values quantised into it, and read back.
//
// A head of D channels lies 8 channels (16 bytes of bf16, one dword of codes) to a lane in D/8
// lanes, so a wave holds 4 or 8 heads, loads and stores are contiguous over a token's heads, and
// the transform is three stages in registers and three or four between lanes, all of them DPP
// moves or swizzles: no LDS memory, no barrier.  The transform to be quantised is in fp64, as in
// cbq_rotate_quantize: exact, so a code does not depend on the order of its sums; reading back
// needs fp32 only, as sums of at most 128 multiples of 1/2 up to 6 are exact there.
#include "kv_device.hpp"

namespace cbq {
namespace {

template <int D>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a, const uint16_t* k, int64_t ldk, const uint16_t* v,
                                                       int64_t ldv, int64_t t0, uint32_t rows, float c_b) {
  constexpr int L = D / 8;                              // lanes of a head
  const int which = blockIdx.y;
  const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  if (row >= rows) return;
  const uint32_t tl = row / (uint32_t)a.n_kv, head = row - tl * (uint32_t)a.n_kv;
  const int64_t t = t0 + tl;
  const uint16_t* src = which ? v + t * ldv : k + t * ldk;
  const u32x4 in = *reinterpret_cast<const u32x4*>(src + head * D + lane * 8);
  const int b = kv_seq_of(a, t);
  if (b < 0) return;
  const int64_t pos = kv_position(a, b, t);
  if (pos < 0) return;
  const int page = kv_page(a, b, pos);
  if (page < 0) return;

  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __builtin_bit_cast(float, in[i] << 16);
    f[2 * i + 1] = __builtin_bit_cast(float, in[i] & 0xFFFF0000u);
  }
  const bool rot = (a.rotate >> which) & 1;
  if (rot) {
    double u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = f[i];
    kv_transform<D>(u, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)u[i];
  }
  // the maximum over bit patterns: a float maximum would drop a NaN
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)xor_lane<1>((int)m));
  m = max(m, (uint32_t)xor_lane<2>((int)m));
  m = max(m, (uint32_t)xor_lane<4>((int)m));
  if constexpr (D >= 128) m = max(m, (uint32_t)xor_lane<8>((int)m));
  const float s = __builtin_bit_cast(float, m) / 6.0f;
  uint32_t codes = 0;
  if (s != 0.0f) {
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0] / s, f[1] / s, 1.0f, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2] / s, f[3] / s, 1.0f, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4] / s, f[5] / s, 1.0f, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6] / s, f[7] / s, 1.0f, 3);
  }
  const int64_t at = kv_row(a, page, (int)head, pos);
  *reinterpret_cast<uint32_t*>(a.codes[which] + at * (D / 2) + lane * 4) = codes;
  if (lane == 0) a.scales[which][at] = rot ? s * c_b : s;
}

template <int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                                                      int first, int64_t t0, uint32_t rows, float c_b) {
  constexpr int L = D / 8;
  const int which = first + blockIdx.y;
  const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  if (row >= rows) return;
  const uint32_t tl = row / (uint32_t)a.n_kv, head = row - tl * (uint32_t)a.n_kv;
  const int64_t t = t0 + tl;
  const int b = kv_seq_of(a, t);
  if (b < 0) return;
  const int64_t pos = kv_position(a, b, t);
  const int page = pos < 0 ? -1 : kv_page(a, b, pos);
  uint16_t* dst = (which ? v + t * ldv : k + t * ldk) + head * D + lane * 8;
  u32x4 out = {0, 0, 0, 0};
  if (page >= 0) {
    const int64_t at = kv_row(a, page, (int)head, pos);
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(a.codes[which] + at * (D / 2) + lane * 4);
    float s = a.scales[which][at];
    const f16x2 p0 = e2m1_pair<0>(codes), p1 = e2m1_pair<1>(codes), p2 = e2m1_pair<2>(codes), p3 = e2m1_pair<3>(codes);
    float f[8] = {(float)p0[0], (float)p0[1], (float)p1[0], (float)p1[1],
                  (float)p2[0], (float)p2[1], (float)p3[0], (float)p3[1]};
    if ((a.rotate >> which) & 1) {
      kv_transform<D>(f, lane);
      s *= c_b;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out[i] = (uint32_t)f32_to_bf16_rne(f[2 * i] * s) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1] * s) << 16);
  }
  *reinterpret_cast<u32x4*>(dst) = out;
}

// Launches over at most 2^31 / L lanes of heads each (row indices and lanes stay in 32 bits).
template <typename F>
hipError_t over_tokens(const KvArgs& a, F launch) {
  const int64_t per = ((int64_t(1) << 31) / (a.D / 8) - 256) / a.n_kv;
  for (int64_t t0 = 0; t0 < a.T; t0 += per) {
    const uint32_t rows = (uint32_t)((a.T - t0 < per ? a.T - t0 : per) * a.n_kv);
    const uint32_t blocks = (rows * (uint32_t)(a.D / 8) + 255) / 256;
    launch(t0, rows, blocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_write(const KvArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                           hipStream_t stream) {
  const float c_b = (float)(1.0 / std::sqrt((double)a.D));
  return over_tokens(a, [&](int64_t t0, uint32_t rows, uint32_t blocks) {
    auto f = a.D == 64 ? kv_write_kernel<64> : kv_write_kernel<128>;
    f<<<dim3(blocks, 2), 256, 0, stream>>>(a, k, ldk, v, ldv, t0, rows, c_b);
  });
}

hipError_t launch_kv_read(const KvArgs& a, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv, hipStream_t stream) {
  const float c_b = (float)(1.0 / std::sqrt((double)a.D));
  return over_tokens(a, [&](int64_t t0, uint32_t rows, uint32_t blocks) {
    auto f = a.D == 64 ? kv_read_kernel<64> : kv_read_kernel<128>;
    f<<<dim3(blocks, k && v ? 2 : 1), 256, 0, stream>>>(a, k, ldk, v, ldv, k ? 0 : 1, t0, rows, c_b);
  });
}

}  // namespace cbq
