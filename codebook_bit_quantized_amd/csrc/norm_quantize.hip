// Norms around a block: the block's expert rows combined, normed, gated and added to the
// residual stream, and the next norm fused with the rotation and the quantiser.
//
// Per token, with every sum and product in fp64:
//   y      = sum_j w_j rows[slot_j] + sum_s shared rows            (when there are rows)
//   y      = y * rsqrt(mean y^2 + eps) * post_weight               (optional)
//   v      = bf16(fp32(residual + scale * gate * y)),  or the given bf16 row
//   n      = bf16(fp32(v * rsqrt(mean v^2 + eps) * weight))        (optional from here on)
//   codes  = the block Walsh-Hadamard transform of n, absmax-quantised per token
// The roundings to bf16 are those of the residual stream and of the activations the
// quantiser takes; they go through fp32 because that is how a bf16 value is formed from a
// wider one elsewhere.  fp64 sums make them (and so the codes) independent of the order
// of summation, except where a value lies within about 2^-50 of a rounding border.
//
// One workgroup per token, CPT channels a thread: 8 (16 beyond K = 8192), so one token's work
// is spread over K / 512 waves (a single token's latency is what decode sees), or 32 for the
// norm before a block of many tokens (norm_width).  A thread's channels are runs of 8, kRun
// apart, so that a wave's loads and stores are contiguous whatever CPT is.  With expert rows it is
// bound by reading them (4096 x 2048, 8 fp32 rows each, gates, norms and codes: 344 MB in 76 us,
// 4.5 TB/s of the 5.1 a large copy reaches; 8 bf16 rows 210 MB in 61 us); the norm alone by its
// vector instructions, mostly the transform's exchanges in fp64 (4096 x 2048: 42 MB in 20 us;
// without codes 34 MB in 10 us).  The transform's first stages run in the thread, the next ones
// between lanes, then between a thread's runs, and the ones across waves in one LDS pass whatever
// their number (each thread reads its partners in the block's other waves and adds them with
// their signs).
#include "cbq_internal.hpp"
#include "few_device.hpp"
#include "rotate_device.hpp"

namespace cbq {

namespace {

// 1 / sqrt(a) for normal a > 0: the hardware estimate, then two steps of Newton's iteration
// y' = y + y (1 - a y^2) / 2, each of which doubles the number of right bits (the estimate
// has more than 20), leaving an error of a few units of 2^-53.
__device__ __forceinline__ double rsqrt_f64(double a) {
  double y = __builtin_amdgcn_rsq(a);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double e = __builtin_fma(-a * y, y, 1.0);
    y = __builtin_fma(0.5 * y, e, y);
  }
  return y;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  v += xor_lane_f64<1>(v);
  v += xor_lane_f64<2>(v);
  v += xor_lane_f64<4>(v);
  v += xor_lane_f64<8>(v);
  v += xor_lane_f64<16>(v);
  v += xor_lane_f64<32>(v);
  return v;
}

// Absolute maxima are taken over the bit patterns of |v|, which order as the values do and put
// NaN above infinity, so a row that is not finite gets a scale that is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
  v = max(v, (uint32_t)xor_lane<1>((int)v));
  v = max(v, (uint32_t)xor_lane<2>((int)v));
  v = max(v, (uint32_t)xor_lane<4>((int)v));
  v = max(v, (uint32_t)xor_lane<8>((int)v));
  v = max(v, (uint32_t)xor_lane<16>((int)v));
  v = max(v, (uint32_t)xor_lane<32>((int)v));
  return v;
}

// A thread's N channels are runs of 8, kRun apart, so a wave's loads and stores are contiguous;
// n: channels from the first run's start to the row's end (whole runs).
constexpr int kRun = 512;

template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, int n, float* f) {
#pragma unroll
  for (int h = 0; h < N / 8; ++h) {
    if (kRun * h >= n) continue;
    const u32x4 q = *reinterpret_cast<const u32x4*>(p + kRun * h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[8 * h + 2 * i] = __builtin_bit_cast(float, q[i] << 16);
      f[8 * h + 2 * i + 1] = __builtin_bit_cast(float, q[i] & 0xFFFF0000u);
    }
  }
}

template <int N>
__device__ __forceinline__ void load_f32(const float* p, int n, float* f) {
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    if (kRun * (h / 2) >= n) continue;
    const f32x4 q = *reinterpret_cast<const f32x4*>(p + kRun * (h / 2) + 4 * (h % 2));
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * h + i] = q[i];
  }
}

// fp64 -> fp32 -> bf16, two roundings to nearest even.  The empty asm keeps the compiler from
// merging them into one rounding of the fp64 value, which differs where fp32 lands on a
// midpoint of two bf16 values (about one value in 2^17).
__device__ __forceinline__ uint32_t f64_to_bf16(double d) {
  float f = (float)d;
  asm("" : "+v"(f));
  return f32_to_bf16_rne(f);
}

// rounds fp64 to fp32 and that to bf16, stores the bf16 and returns their values
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, int n, bool store, const double* d, float* f) {
#pragma unroll
  for (int h = 0; h < N / 8; ++h) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = f64_to_bf16(d[8 * h + 2 * i]);
      const uint32_t hi = f64_to_bf16(d[8 * h + 2 * i + 1]);
      q[i] = lo | (hi << 16);
      f[8 * h + 2 * i] = __builtin_bit_cast(float, lo << 16);
      f[8 * h + 2 * i + 1] = __builtin_bit_cast(float, hi << 16);
    }
    if (store && kRun * h < n) *reinterpret_cast<u32x4*>(p + kRun * h) = q;
  }
}

}  // namespace

// SRC: where the normed row comes from.  kNormX: the bf16 row x; kNormF32 / kNormBF16: the
// block's rows of that type, combined and added to the residual; kRotateF32: no norm, fp32
// rows (whose transform then rounds like any fp64 sum).
template <int CPT, int NT, int SRC>
__global__ void __launch_bounds__(NT)
norm_quantize_kernel(NormArgs a) {
  extern __shared__ double xchg[];           // cross-wave transform stages: [8][blockDim]
  __shared__ double s_sum[2][16];            // per-wave sums of squares: post norm, norm
  __shared__ uint32_t s_max[16];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nw = (int)blockDim.x >> 6;
  const int64_t t = a.t0 + blockIdx.x;
  const int c0 = wave * 64 * CPT + lane * 8;
  const int left = a.K - c0;                 // K is a multiple of 32, so whole runs
  const bool act = left > 0;
  float f[CPT];                              // the row that is normed and quantised

  if constexpr (SRC == kRotateF32) {
    if (act) load_f32<CPT>(static_cast<const float*>(a.rows) + t * a.ldr + c0, left, f);
  } else if constexpr (SRC == kNormX) {
    if (act) load_bf16<CPT>(a.x + t * a.ldx + c0, left, f);
  } else {
    using Row = std::conditional_t<SRC == kNormF32, float, uint16_t>;
    const Row* rows = reinterpret_cast<const Row*>(a.rows) + c0;
    const int n = a.topk + a.n_shared;
    float res[CPT], gate[CPT], pw[CPT];
    double y[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) y[i] = 0.0;
    if (act) {
      // everything is requested up front, RB of the rows before the first is used: a token's
      // rows lie apart, and each load that waits for another costs its whole latency
      constexpr int RB = CPT == 8 && NT <= 512 ? 8 : CPT == 8 ? 4 : 2;   // what the registers hold
      float r[RB][CPT];
      auto row_of = [&](int j) {
        return j < a.topk ? (int64_t)a.slot_of[t * a.topk + j] : a.T * a.topk + (j - a.topk) * a.T + t;
      };
      auto load_row = [&](int j, float* d) {
        if constexpr (SRC == kNormF32) load_f32<CPT>(rows + row_of(j) * a.ldr, left, d);
        else load_bf16<CPT>(rows + row_of(j) * a.ldr, left, d);
      };
#pragma unroll
      for (int j = 0; j < RB; ++j)
        if (j < n) load_row(j, r[j]);
      load_bf16<CPT>(a.x + t * a.ldx + c0, left, res);
      if (CPT == 8 && a.gate != nullptr) load_bf16<CPT>(a.gate + t * a.ldg + c0, left, gate);
      if (CPT == 8 && a.post_weight != nullptr) load_f32<CPT>(a.post_weight + c0, left, pw);
#pragma unroll 1
      for (int j0 = 0; j0 < n; j0 += RB) {
        if (j0 > 0) {
#pragma unroll
          for (int j = 0; j < RB; ++j)
            if (j0 + j < n) load_row(j0 + j, r[j]);
        }
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          if (j0 + j < n) {
            const double w = j0 + j < a.topk ? (double)a.topk_w[t * a.topk + j0 + j] : 1.0;
#pragma unroll
            for (int i = 0; i < CPT; ++i)
              if (kRun * (i / 8) < left) y[i] = __builtin_fma(w, (double)r[j][i], y[i]);
          }
        }
      }
    }
    if (a.post_weight != nullptr) {
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < CPT; ++i) ss = __builtin_fma(y[i], y[i], ss);
      ss = wave_sum_f64(ss);
      if (CPT > 8 && act) load_f32<CPT>(a.post_weight + c0, left, pw);   // 16 channels leave no registers for it above
      if (lane == 0) s_sum[0][wave] = ss;
      lds_barrier();
      double tot = 0.0;
      for (int w = 0; w < nw; ++w) tot += s_sum[0][w];
      const double rn = rsqrt_f64(tot * a.inv_K + (double)a.post_eps);
#pragma unroll
      for (int i = 0; i < CPT; ++i) y[i] = kRun * (i / 8) < left ? y[i] * rn * (double)pw[i] : 0.0;
    }
    if (act) {
      if (a.gate != nullptr) {
        if (CPT > 8) load_bf16<CPT>(a.gate + t * a.ldg + c0, left, gate);
#pragma unroll
        for (int i = 0; i < CPT; ++i) y[i] *= (double)gate[i];
      }
#pragma unroll
      for (int i = 0; i < CPT; ++i) y[i] = __builtin_fma((double)a.scale, y[i], (double)res[i]);
      store_bf16<CPT>(a.out + t * a.ldo + c0, left, true, y, f);
    }
    if (a.weight == nullptr) return;         // uniform over the launch
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i)
    if (kRun * (i / 8) >= left) f[i] = 0.0f;

  // ---- RMS norm ----
  double v[CPT];
  if constexpr (SRC != kRotateF32) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < CPT; ++i) ss = __builtin_fma((double)f[i], (double)f[i], ss);
    ss = wave_sum_f64(ss);
    if (lane == 0) s_sum[1][wave] = ss;
    lds_barrier();
    double tot = 0.0;
    for (int w = 0; w < nw; ++w) tot += s_sum[1][w];
    const double rn = rsqrt_f64(tot * a.inv_K + (double)a.eps);
    float wt[CPT];
    load_f32<CPT>(a.weight + c0, left, wt);
#pragma unroll
    for (int i = 0; i < CPT; ++i) v[i] = kRun * (i / 8) < left ? (double)f[i] * rn * (double)wt[i] : 0.0;
    store_bf16<CPT>(a.normed + t * a.ldn + c0, left, a.normed != nullptr, v, f);
  }
  if (a.codes == nullptr) return;            // uniform over the launch
#pragma unroll
  for (int i = 0; i < CPT; ++i) v[i] = (double)f[i];

  // ---- block Walsh-Hadamard transform (fp64, exact for bf16 rows within the bound that
  // rotate_quantize states) ----
  const int b = 1 << a.logb;
  auto in_thread = [&](auto distance) {
    constexpr int h = decltype(distance)::value;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      if (!(i & h)) {
        const double p = v[i], q = v[i + h];
        v[i] = p + q;
        v[i + h] = p - q;
      }
    }
  };
  if (b > 1) in_thread(std::integral_constant<int, 1>{});
  if (b > 2) in_thread(std::integral_constant<int, 2>{});
  if (b > 4) in_thread(std::integral_constant<int, 4>{});
  if (b > 8) lane_stage<1, CPT>(v, (lane & 1) != 0);
  if (b > 16) lane_stage<2, CPT>(v, (lane & 2) != 0);
  if (b > 32) lane_stage<4, CPT>(v, (lane & 4) != 0);
  if (b > 64) lane_stage<8, CPT>(v, (lane & 8) != 0);
  if (b > 128) lane_stage<16, CPT>(v, (lane & 16) != 0);
  if (b > 256) lane_stage<32, CPT>(v, (lane & 32) != 0);
  if constexpr (CPT >= 16)
    if (b > kRun) in_thread(std::integral_constant<int, 8>{});
  if constexpr (CPT >= 32)
    if (b > 2 * kRun) in_thread(std::integral_constant<int, 16>{});
  const int wpb = b / (64 * CPT);            // waves per block
  if (wpb > 1) {
    // v of wave w is the sum over the block's waves w' of (-1)^popcount(w & w') v of w'
    const int wb = wave & (wpb - 1), first = (wave - wb) * 64 + lane;
    const int pitch = (int)blockDim.x;
#pragma unroll
    for (int c = 0; c < CPT; c += 8) {
      if (c > 0) lds_barrier();
#pragma unroll
      for (int i = 0; i < 8; ++i) xchg[i * pitch + tid] = v[c + i];
      lds_barrier();
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c + i] = (__builtin_popcount(wb) & 1) ? -v[c + i] : v[c + i];
      for (int w = 0; w < wpb; ++w) {
        if (w == wb) continue;
        const double sg = (__builtin_popcount(w & wb) & 1) ? -1.0 : 1.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c + i] = __builtin_fma(xchg[i * pitch + first + 64 * w], sg, v[c + i]);
      }
    }
  }

  // ---- per-token absmax ----
  float u[CPT];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    u[i] = (float)v[i];
    top = max(top, abs_bits(u[i]));
  }
  top = wave_max_bits(top);
  if (lane == 0) s_max[wave] = top;
  lds_barrier();
  top = s_max[0];
  for (int w = 1; w < nw; ++w) top = max(top, s_max[w]);
  const float amax = __builtin_bit_cast(float, top);

  // ---- quantise: the fp32 sequence of rotate_quantize (s = M / Q, q = clamp(rint(v / s)),
  // the quotient as fp64(v) * fp64(1 / s) rounded to fp32, rint by the magic-number add);
  // the lane stages' sign, the parity of the lane's bits inside the block, is folded in ----
  const float Q = a.act_bits == 4 ? 7.0f : 127.0f;
  const float lo = a.act_bits == 4 ? -8.0f : -127.0f;
  constexpr float kMagic = 12582912.0f;
  const float s = amax / Q;
  const int lpb = b / 8 < 64 ? b / 8 : 64;   // lanes per block within a wave
  const bool neg = lpb > 1 && (__builtin_popcount((unsigned)lane & (unsigned)(lpb - 1)) & 1);
  const double rs = amax != 0.0f ? (neg ? -1.0 : 1.0) / (double)s : 0.0;
  if constexpr (SRC == kRotateF32) {
    // the codes as fp16, in the order the few-row GEMM dequantises weights to
    uint8_t* dst = a.codes + t * few_row16_bytes(a.K);
#pragma unroll
    for (int k = 0; k < CPT / 8; ++k) {
      if (c0 + kRun * k >= (a.K + 127) / 128 * 128) continue;   // the fp16 rows hold zeros up to there
      f16x2 d[4];                            // (k0, k2) (k4, k6) (k1, k3) (k5, k7)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = (float)((double)u[8 * k + i] * rs);
        d[(i & 1) * 2 + (i >> 2)][(i >> 1) & 1] =
            (_Float16)(__builtin_amdgcn_fmed3f(r + kMagic, kMagic + lo, kMagic + Q) - kMagic);
      }
      *reinterpret_cast<u32x4*>(dst + few_pos16(c0 + kRun * k)) =
          u32x4{__builtin_bit_cast(uint32_t, d[0]), __builtin_bit_cast(uint32_t, d[1]),
                __builtin_bit_cast(uint32_t, d[2]), __builtin_bit_cast(uint32_t, d[3])};
    }
    if (tid == 0) a.scales[t] = amax != 0.0f ? s * a.c_b : 0.0f;
    return;
  }
  uint32_t q[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const float r = (float)((double)u[i] * rs);
    q[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(r + kMagic, kMagic + lo, kMagic + Q));
  }
  auto low_bytes = [&](int i0, int i1, int i2, int i3) {
    const uint32_t l = perm(q[i1], q[i0], 0x0C0C0400u), h = perm(q[i3], q[i2], 0x0C0C0400u);
    return perm(h, l, 0x05040100u);
  };
  uint32_t w[CPT / 4];
  if (a.act_bits == 4) {
#pragma unroll
    for (int k = 0; k < CPT / 8; ++k) {
      const uint32_t ev = low_bytes(8 * k, 8 * k + 2, 8 * k + 4, 8 * k + 6);
      const uint32_t od = low_bytes(8 * k + 1, 8 * k + 3, 8 * k + 5, 8 * k + 7);
      w[k] = (ev & 0x0F0F0F0Fu) | ((od << 4) & 0xF0F0F0F0u);
    }
    uint8_t* dst = a.codes + t * (a.K / 2) + c0 / 2;
#pragma unroll
    for (int k = 0; k < CPT / 8; ++k)
      if (kRun * k < left) *reinterpret_cast<uint32_t*>(dst + kRun / 2 * k) = w[k];
  } else {
#pragma unroll
    for (int k = 0; k < CPT / 4; ++k) w[k] = low_bytes(4 * k, 4 * k + 1, 4 * k + 2, 4 * k + 3);
    uint8_t* dst = a.codes + t * a.K + c0;
#pragma unroll
    for (int k = 0; k < CPT / 8; ++k)
      if (kRun * k < left) *reinterpret_cast<u32x2*>(dst + kRun * k) = u32x2{w[2 * k], w[2 * k + 1]};
  }
  if (tid == 0) a.scales[t] = amax != 0.0f ? s * a.c_b : 0.0f;
}

template <int CPT, int NT>
static void launch_nt(const NormArgs& a, int src, unsigned tokens, unsigned threads, size_t lds, hipStream_t stream) {
  const dim3 grid(tokens), block(threads);
  if (src == kNormX) hipLaunchKernelGGL((norm_quantize_kernel<CPT, NT, kNormX>), grid, block, lds, stream, a);
  else if (src == kNormF32) hipLaunchKernelGGL((norm_quantize_kernel<CPT, NT, kNormF32>), grid, block, lds, stream, a);
  else if (src == kNormBF16) hipLaunchKernelGGL((norm_quantize_kernel<CPT, NT, kNormBF16>), grid, block, lds, stream, a);
  else hipLaunchKernelGGL((norm_quantize_kernel<CPT, NT, kRotateF32>), grid, block, lds, stream, a);
}

// Channels a thread of the norm before a block: 8 is the shortest chain, and the faster one up
// to about 4 million values; beyond, 32 where they fill the waves, as a wave's reductions and
// exchanges then serve four times the channels (us, 8 against 32: 512 x 4096 10.1 / 12.3, 1024 x
// 2048 9.4 / 10.6, 2048 x 2048 14.6 / 14.7, 4096 x 2048 21.2 / 20.1, 4096 x 4096 41.8 / 34.3,
// 2048 x 8192 58 / 38; waves filled to 62 %: 4096 x 2560 21.7 / 26.8).  Beyond 8192 channels a workgroup's
// 1024 threads need 16 (or 32).
static int norm_width(int64_t T, int K) {
  const int threads = K / 32, full = (threads + 63) / 64 * 64;
  if (T * K >= (1 << 22) && 10 * threads >= 9 * full) return 32;
  return K <= 8192 ? 8 : 16;
}

hipError_t launch_norm_quantize(NormArgs a, int src, int b, hipStream_t stream) {
  a.logb = 0;
  while ((1 << a.logb) < b) ++a.logb;
  a.c_b = (float)(1.0 / std::sqrt((double)b));
  a.inv_K = 1.0 / (double)a.K;
  const int cpt = src == kNormX ? norm_width(a.T, a.K) : a.K <= 8192 ? 8 : 16;
  const unsigned threads = (unsigned)((a.K / cpt + 63) / 64 * 64);
  // cross-wave transform stages only where a block spans waves
  const size_t lds = a.codes != nullptr && b > 64 * cpt ? (size_t)8 * threads * sizeof(double) : 0;
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kMaxGrid = 1 << 21;
  for (a.t0 = 0; a.t0 < a.T; a.t0 += kMaxGrid) {
    const unsigned n = (unsigned)(a.T - a.t0 < kMaxGrid ? a.T - a.t0 : kMaxGrid);
    if (cpt == 32) hipLaunchKernelGGL((norm_quantize_kernel<32, 512, kNormX>), dim3(n), dim3(threads), lds, stream, a);
    else if (cpt == 16) launch_nt<16, 1024>(a, src, n, threads, lds, stream);
    else if (threads <= 256) launch_nt<8, 256>(a, src, n, threads, lds, stream);
    else if (threads <= 512) launch_nt<8, 512>(a, src, n, threads, lds, stream);
    else launch_nt<8, 1024>(a, src, n, threads, lds, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace cbq
