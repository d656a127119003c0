// The whole MoE layer for a few tokens (a decode batch): routing, gate/up with SwiGLU, the
// rotation and quantisation of h, down and the weighted combine.
//
// CodeQuant2, Figures 3 and 4 (codebook weights looked up in on-chip tables); the AI Radio
// episode, introduction (a router in front of the experts).
//
// What the layer costs beyond the bytes of its weights is launches, dependent loads and, at
// 4 bits, the vector instructions of the table lookups.  Rows are numbered by choice (row
// t * topk + j is token t's j-th choice, row T * topk + s * T + t shared expert s), which
// needs no counting and no row lists in memory: a workgroup finds its expert's rows by
// scanning the chosen ids.  Two forms:
//
// A batch:
//   1. per token: the chosen ids and weights, and the input codes converted to fp16 once (per
//      wave and chunk the conversion is 44 of about 230 vector instructions of a gate/up pair,
//      and of 140 of a single matrix);
//   2. gate/up: h = silu(g) * u in fp32;
//   3. rotation and quantisation of h's rows, codes left in fp16 (norm_quantize.hip);
//   4. down: the expert rows;
//   5. the weighted sum of each token's rows.
// One token with a short h (one_token_form), where launches and dependent loads are most of it:
//   1. gate/up whose waves find their choice's expert from the logits themselves;
//   2. one kernel for the rest: every workgroup rotates and quantises all rows of h (a few
//      thousand values) as the batch form does, a wave a row, multiplies its 16 columns of down and combines them.
// These two run every instruction a few times only, so instruction fetches count: their loops
// stay rolled where the unrolled code would run once.
//
// Measured (us; weights of three layers in turn): 128 experts, top 8, 2048 x 768, 4 bits: one
// token 9.4 + 9.6 (the batch form takes 24 a call, this one 17.6); 32 tokens 4.7 + 49 + 4.8 + 31
// + 5.2.  64 + 2 experts, 2048 x 1408, 3 and 2 bits, 8 tokens 3.7 + 26 + 4.7 + 14 + 4.6.  8
// experts, top 2, 4096 x 14336, 4 bits, 16 tokens 4.9 + 110 + 9.7 + 62 + 4.8.
// h is kept in fp32 up to the quantiser: the codes are those of the unrounded h up to fp32
// sums (a bf16 h would move a code wherever its rounding crosses a border).
#include "cbq_internal.hpp"
#include "few_device.hpp"
#include "rotate_device.hpp"
#include "route_device.hpp"

namespace cbq {

namespace {

typedef double f64x2 __attribute__((ext_vector_type(2)));

// maximum of v over the wave (DPP row rotations, then four scalar reads)
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto ror = [](uint32_t x, auto n) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x120 + decltype(n)::value, 0xF, 0xF, false);
  };
  v = max(v, ror(v, std::integral_constant<int, 1>{}));
  v = max(v, ror(v, std::integral_constant<int, 2>{}));
  v = max(v, ror(v, std::integral_constant<int, 4>{}));
  v = max(v, ror(v, std::integral_constant<int, 8>{}));
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}

// a logit's key; 0 stands for an expert that is taken (or none), which one NaN would map to
__device__ __forceinline__ uint32_t expert_key(float l) { return max(order_bits(l), 1u); }

// the expert of rank j in a token's logits (ties to the lower id): j + 1 rounds of a wave
// maximum; whole waves only.  NI: 64-expert groups (E <= 64 * NI)
template <int NI>
__device__ __forceinline__ int expert_of_rank(const float* row, int E, int j, int lane) {
  uint32_t key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? expert_key(row[e]) : 0u;
  }
  int e = 0;
#pragma unroll 1
  for (int r = 0; r <= j; ++r) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) m = max(m, key[i]);
    m = wave_max_u32(m);
    e = 0;
#pragma unroll
    for (int i = NI - 1; i >= 0; --i) {
      const uint64_t at = __ballot(key[i] == m);
      if (at) e = 64 * i + __builtin_ctzll(at);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane + 64 * i == e) key[i] = 0u;
  }
  return e;
}

// the softmax weight of a choice: lane j < topk holds the j-th chosen logit; lg: the token's
// logits.  Whole waves only.
__device__ __forceinline__ float choice_weight(float l, const float* lg, int E, int topk, int renormalize, int lane) {
  const float top = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l), 0));
  const float ex = lane < topk ? expf(l - top) : 0.0f;
  float den = ex;
  if (!renormalize) {
    den = 0.0f;
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < E) den += expf(lg[lane + 64 * i] - top);
  }
  den += xor_lane_f32<1>(den);
  den += xor_lane_f32<2>(den);
  den += xor_lane_f32<4>(den);
  den += xor_lane_f32<8>(den);
  den += xor_lane_f32<16>(den);
  den += xor_lane_f32<32>(den);
  return ex / den;
}

}  // namespace

// One workgroup per token: wave 0 ranks the logits by topk rounds of a wave maximum (ties to
// the lower id) and forms the weights, the others convert the token's codes.  Latency-bound
// (about 4.5 us): a chain of loads and rounds.
template <int ABITS>
__global__ void __launch_bounds__(256)
few_prepare_kernel(const float* __restrict__ logits, int T, int E, int topk, int renormalize,
                   const uint8_t* __restrict__ codes, int K, int32_t* __restrict__ ids, float* __restrict__ wts,
                   uint8_t* __restrict__ codes16) {
  const int t = blockIdx.x, lane = threadIdx.x & 63;
  const int64_t pitch = few_row16_bytes(K);
  for (int p = threadIdx.x - 64; p >= 0 && p < (int)(pitch / 64); p += 192) {   // 32 channels each
    uint32_t raw[ABITS] = {}, d[16];
    if (32 * p < K) {
      const u32x4* src = reinterpret_cast<const u32x4*>(codes + (int64_t)t * (K * ABITS / 8) + p * 4 * ABITS);
#pragma unroll
      for (int h = 0; h < ABITS / 4; ++h) {
        const u32x4 v = src[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[4 * h + i] = v[i];
      }
    }
    codes32_to_f16<ABITS>(raw, d);           // zero codes past K
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<u32x4*>(codes16 + t * pitch + few_pos16(32 * p + 8 * j)) =
          u32x4{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]};
  }
  if (threadIdx.x >= 64) return;
  const float* lg = logits + (int64_t)t * E;
  uint32_t key[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? expert_key(lg[e]) : 0u;
  }
  int mine = 0;
  for (int r = 0; r < topk; ++r) {
    const uint32_t m = wave_max_u32(max(max(key[0], key[1]), max(key[2], key[3])));
    int e = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint64_t at = __ballot(key[i] == m);
      if (at) e = 64 * i + __builtin_ctzll(at);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i == e) key[i] = 0u;
    if (lane == r) mine = e;
  }
  const float w = choice_weight(lg[mine], lg, E, topk, renormalize, lane);
  if (lane < topk) {
    ids[t * topk + lane] = mine;
    wts[t * topk + lane] = w;
  }
}

// Rows of this workgroup's expert, in LDS: code row and output row of each.
struct FewRows {
  int n;
  int16_t code[kFewRows], out[kFewRows];
};

// h = silu(g) * u with the accurate exponential and division: its error moves codes of h
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// A batch's grouped GEMM on fp16 codes.  PAIR: gate/up (code rows are tokens, 16 columns of
// both matrices a wave); else down (code rows are choices, 32 columns a wave, so a wave always
// dequantises two sets of 16 weight rows for each piece of codes it loads).  Workgroups of
// CW * SK waves: CW column tiles, each with K split over SK waves.  blockIdx.y: an expert, or,
// when there are fewer choices than experts, a choice (the first one of its expert does the
// work).  An expert of more than 16 rows sweeps its weights twice.
// Bound by reading the weights and, at 4 bits, by looking them up (23 vector instructions for 8
// weights: about 26 us of the 49 for 362 million weights), which overlap in part: 128 experts
// at 32 tokens 181 MB in 49 us (3.7 TB/s) and 95 MB in 31 us; 8 wide experts 477 MB in 110 us
// (4.3 TB/s) and 236 MB in 62 us, where a large copy reaches 5.1.  Five waves a SIMD and two
// chunks in flight: four waves measured 3 % faster (128 experts) to 4 % slower (8 wide ones),
// four chunks the same to 15 % slower (their registers cost waves).
template <int BITS, bool PAIR, bool BLK, int DEPTH>
__global__ void __launch_bounds__(512, 5)
few_gemm_kernel(FewArgs a, int CW, int SK) {
  extern __shared__ f32x4 red[];
  __shared__ FewRows s_rows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave / SK, sk = wave - cw * SK;
  const int T = a.T, E = a.E, topk = a.topk;
  // shared experts, which every token visits, come last in y and are started first
  const int y = (int)(gridDim.y - 1 - blockIdx.y);
  const int routed = (int)gridDim.y - a.n_shared;
  const bool by_choice = routed < E, shared = y >= routed;
  const int e = shared ? E + y - routed : by_choice ? a.ids[y] : y;
  if (shared) {
    if (threadIdx.x < T) {
      const int row = T * topk + (y - routed) * T + threadIdx.x;
      s_rows.code[threadIdx.x] = (int16_t)(PAIR ? threadIdx.x : row);
      s_rows.out[threadIdx.x] = (int16_t)row;
    }
    if (threadIdx.x == 0) s_rows.n = T;
  } else if (wave == 0) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {            // T * topk <= 256
      const int p = 64 * i + lane;
      const bool is = p < T * topk && a.ids[p] == e;
      const uint64_t at = __ballot(is);
      const int pos = n + __popcll(at & ((1ull << lane) - 1));
      if (is && pos < kFewRows) {
        s_rows.code[pos] = (int16_t)(PAIR ? p / topk : p);
        s_rows.out[pos] = (int16_t)p;
      }
      n += __popcll(at);
    }
    if (lane == 0) s_rows.n = min(n, kFewRows);
  }
  const int n0 = (blockIdx.x * CW + cw) * (PAIR ? 16 : 32);
  const int nchunks = (a.K + 127) >> 7;
  const int cpw = (nchunks + SK - 1) / SK;
  const int c0 = sk * cpw, c1 = min(nchunks, c0 + cpw);
  FewWeights<BITS, 2> W;
  W.init(a.w, !PAIR, (uint32_t)e < (uint32_t)(E + a.n_shared) ? e : 0, n0, a.N, a.K, a.blocked, lane);
  uint32_t ring[DEPTH][2][BITS];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);
  lds_barrier();
  const int me = s_rows.n;
  if (me == 0 || (by_choice && !shared && s_rows.out[0] != y)) return;

  const int64_t pitch = few_row16_bytes(a.K);
  const __amdgpu_buffer_rsrc_t cres = make_rsrc(a.codes, 0x7FFFFFFFu);
  for (int m0 = 0; m0 < me; m0 += 16) {
    if (m0 > 0) {
      if (SK > 1) lds_barrier();             // red is free again
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);
    }
    f32x4 acc[2];
    acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int ma = m0 + (lane & 15);
    const uint32_t aoff = ma < me ? (uint32_t)(s_rows.code[ma] * pitch) + (uint32_t)((lane >> 4) * 16) : kOffNone;
    few_sweep16<BITS, 2, BLK, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
    few_reduce<2>(red, cw, sk, SK, lane, acc);
    if (sk != 0) continue;
    // lane holds D[m = 4 * (lane >> 4) + i][n = lane & 15]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 4 * (lane >> 4) + i;
      if (m >= me) continue;
      const float sc = a.scales[s_rows.code[m]];
      float* out = a.out + (int64_t)s_rows.out[m] * a.N + n0 + (lane & 15);
      if constexpr (PAIR) {
        if (n0 < a.N) out[0] = swiglu(acc[0][i] * sc, acc[1][i] * sc);
      } else {
        if (n0 < a.N) out[0] = acc[0][i] * sc;
        if (n0 + 16 < a.N) out[16] = acc[1][i] * sc;
      }
    }
  }
}

// Gate/up of one token, on its packed codes.  blockIdx.y: a choice, then the shared experts;
// row y of h.  The SK waves split K.  Bound by its chain of loads: the logits, then the
// codebooks and first indices of the expert they name, about 1 us each, behind the launch and
// the instruction fetches (8 experts of 2048 x 768, 13 MB: 9.4 us).
template <int BITS, int ABITS, bool BLK, int DEPTH>
__global__ void __launch_bounds__(512, 4)
few_gate_one_kernel(FewArgs a, int SK) {
  __shared__ float s_part[8][32];
  const int lane = threadIdx.x & 63;
  const int sk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int y = (int)blockIdx.y;
  int e = a.E + y - a.topk;
  if (y < a.topk) {
    e = a.E <= 64    ? expert_of_rank<1>(a.logits, a.E, y, lane)
        : a.E <= 128 ? expert_of_rank<2>(a.logits, a.E, y, lane)
                     : expert_of_rank<4>(a.logits, a.E, y, lane);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.ids[y] = e;
  }
  const int n0 = blockIdx.x * 16;
  const int nchunks = (a.K + 127) >> 7;
  const int cpw = (nchunks + SK - 1) / SK;
  const int c0 = sk * cpw, c1 = min(nchunks, c0 + cpw);
  FewWeights<BITS, 2> W;
  W.init(a.w, false, e, n0, a.N, a.K, a.blocked, lane);
  uint32_t ring[DEPTH][2][BITS];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);
  f32x4 acc[2][2];
  acc[0][0] = acc[1][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // row 0 of A is the token, the others are zero
  const uint32_t aoff[2] = {(lane & 15) == 0 ? (uint32_t)((lane >> 4) * 4 * ABITS) : kOffNone, kOffNone};
  const __amdgpu_buffer_rsrc_t cres = make_rsrc(a.codes, 0x7FFFFFFFu);
  few_sweep<BITS, ABITS, 2, BLK, 1, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
  const float sc = a.scales[0];
  if (lane < 16) {
    s_part[sk][lane] = acc[0][0][0];
    s_part[sk][16 + lane] = acc[1][0][0];
  }
  lds_barrier();
  if (threadIdx.x < 32) {
    float v = 0.0f;
#pragma unroll 4
    for (int k = 0; k < SK; ++k) v += s_part[k][lane];
    v *= sc;
    const float u = xor_lane_f32<16>(v);
    if (lane < 16) a.out[(int64_t)y * a.N + n0 + lane] = swiglu(v, u);
  }
}

// Bytes of LDS a value of h takes while few_down_one_kernel transforms it: fp64 where blocks of
// more than 256 channels pass through LDS between their stages, else the fp32 result.
__host__ __device__ constexpr int one_token_value_bytes(int F) { return (F & -F) > 256 ? 8 : 4; }

// The rest of the one-token form.  Workgroup: 16 columns of y; wave = row << ksh | split of K.
// Every workgroup repeats the rotation of all rows (6144 values at 8 rows of 768), which costs
// less than the launches it saves while the rows are few and short (one_token_form): 9.6 us for
// the 6.8 MB of down, of which the transform in fp64 instead of fp32 is 1.0 (with fp32 a code or
// the scale differed between a token alone and in a batch).
template <int BITS, bool BLK, int DEPTH>
__global__ void __launch_bounds__(1024)
few_down_one_kernel(FewDownArgs a, int ksh) {
  extern __shared__ uint8_t s_codes[];       // fp16 codes of every row, [R][pitch]
  __shared__ float s_part[16][16];           // by wave
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = (int)blockDim.x >> 6, F = a.F, topk = a.topk;
  const int row = wave >> ksh, split = wave & ((1 << ksh) - 1);
  const float* h = a.h + (int64_t)row * F;
  const int id = lane < topk ? a.ids[lane] : 0;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // the row's first 256 channels are requested with the ids
  f32x4 next = split == 0 && 4 * lane < F ? *reinterpret_cast<const f32x4*>(h + 4 * lane) : zero;
  const int e = row < topk ? __builtin_amdgcn_readlane(id, row) : a.E + row - topk;
  const int n0 = blockIdx.x * 16;
  const int nchunks = (F + 127) >> 7, cpw = (nchunks + (1 << ksh) - 1) >> ksh;
  const int c0 = split * cpw, c1 = min(nchunks, c0 + cpw);
  const int pitch = (int)few_row16_bytes(F);
  // the weights' first chunks are on their way while h is transformed
  FewWeights<BITS, 1> W;
  W.init(&a.w, false, e, n0, a.H, F, a.blocked, lane);
  uint32_t ring[DEPTH][1][BITS];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);
  const float lg = a.logits[id];

  // Rotation of row `row` by its first wave, 256 channels a pass (4 consecutive ones a lane), in
  // fp64 and rounded once to fp32 as rotate_quantize does: butterflies in the lane and between
  // lanes, then, for blocks beyond 256 channels, passes over the row's LDS.  u holds four
  // channels' fp32 results in 16 bytes, or, where such passes need the fp64 values, in the first
  // 16 of their 32.
  const int b = F & -F;                      // >= 32
  const int usz = one_token_value_bytes(F);
  uint8_t* u = s_codes + (size_t)(nw >> ksh) * pitch + (size_t)row * ((F + 255) & ~255) * usz;
  if (split == 0) {
    uint32_t top = 0;                        // of |v|'s bits, which put NaN above infinity
    auto take = [&](const double* d, uint8_t* to) {   // d rounded to fp32, stored and in the maximum
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = (float)d[k];
        top = max(top, __builtin_bit_cast(uint32_t, f[k]) & 0x7FFFFFFFu);
      }
      *reinterpret_cast<f32x4*>(to) = f32x4{f[0], f[1], f[2], f[3]};
    };
#pragma unroll 1
    for (int c = 4 * lane; c < ((F + 255) & ~255); c += 256) {
      const f32x4 x = next;
      next = c + 256 < F ? *reinterpret_cast<const f32x4*>(h + c + 256) : zero;
      const double p[4] = {(double)x[0] + (double)x[1], (double)x[0] - (double)x[1], (double)x[2] + (double)x[3],
                           (double)x[2] - (double)x[3]};
      double v[4] = {p[0] + p[2], p[1] + p[3], p[0] - p[2], p[1] - p[3]};
      auto stage = [&](auto m) {
        constexpr int M = decltype(m)::value;
        const double sg = (lane & M) ? -1.0 : 1.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __builtin_fma(v[k], sg, xor_lane_f64<M>(v[k]));
      };
      stage(std::integral_constant<int, 1>{});
      stage(std::integral_constant<int, 2>{});
      stage(std::integral_constant<int, 4>{});
      if (b > 32) stage(std::integral_constant<int, 8>{});
      if (b > 64) stage(std::integral_constant<int, 16>{});
      if (b > 128) stage(std::integral_constant<int, 32>{});
      if (b <= 256) {
        take(v, u + c * 4);                  // zeros past F
      } else {
#pragma unroll
        for (int k = 0; k < 4; k += 2) *reinterpret_cast<f64x2*>(u + c * 8 + 8 * k) = f64x2{v[k], v[k + 1]};
      }
    }
    // a lane only ever touches its own channels (mod 256), so these passes need no barrier
#pragma unroll 1
    for (int m = 256; m < b; m *= 2) {
#pragma unroll 1
      for (int c = 4 * lane; c < F; c += 256) {
        if (c & m) continue;
        double x[4], z[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const f64x2 p = *reinterpret_cast<const f64x2*>(u + c * 8 + 8 * k);
          const f64x2 q = *reinterpret_cast<const f64x2*>(u + (c + m) * 8 + 8 * k);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[k + i] = p[i] + q[i];
            z[k + i] = p[i] - q[i];
          }
        }
        if (2 * m == b) {
          take(x, u + c * 8);
          take(z, u + (c + m) * 8);
        } else {
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            *reinterpret_cast<f64x2*>(u + c * 8 + 8 * k) = f64x2{x[k], x[k + 1]};
            *reinterpret_cast<f64x2*>(u + (c + m) * 8 + 8 * k) = f64x2{z[k], z[k + 1]};
          }
        }
      }
    }
    const float amax = __builtin_bit_cast(float, wave_max_u32(top));
    // the quantiser of rotate_quantize
    const float Q = a.act_bits == 4 ? 7.0f : 127.0f, lo = a.act_bits == 4 ? -8.0f : -127.0f;
    constexpr float kMagic = 12582912.0f;
    const float s = amax / Q;
    const double rs = amax != 0.0f ? 1.0 / (double)s : 0.0;
#pragma unroll 1
    for (int c = 4 * lane; c < pitch / 2; c += 256) {   // zeros past F
      const f32x4 v = *reinterpret_cast<const f32x4*>(u + c * usz);
      f16x2 q[2];                            // (k0, k2), (k1, k3) of this half group
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float r = (float)((double)v[k] * rs);
        q[k & 1][k >> 1] = (_Float16)(__builtin_amdgcn_fmed3f(r + kMagic, kMagic + lo, kMagic + Q) - kMagic);
      }
      uint8_t* d = s_codes + row * pitch + few_pos16(c & ~7) + (c & 4);
      *reinterpret_cast<uint32_t*>(d) = __builtin_bit_cast(uint32_t, q[0]);
      *reinterpret_cast<uint32_t*>(d + 8) = __builtin_bit_cast(uint32_t, q[1]);
    }
    // the row's factor: its scale and its choice's weight (1 for a shared expert)
    float f = amax != 0.0f ? s * a.c_b : 0.0f;
    if (row < topk) {
      const float w = choice_weight(lg, a.logits, a.E, topk, a.renormalize, lane);
      f *= __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), row));
    }
    if (lane == 0) s_part[wave][0] = f;
  }
  lds_barrier();
  const float f = s_part[row << ksh][0];

  // D row 0 is the wave's row; the other rows of A are zero
  f32x4 acc = zero;
  const uint8_t* arow = s_codes + row * pitch + (lane >> 4) * 16;
#pragma unroll 1
  for (int c = c0; c < c1; c += DEPTH) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      if (c + i < c1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4 av = {0, 0, 0, 0};
          if ((lane & 15) == 0) av = *reinterpret_cast<const u32x4*>(arow + (c + i) * 256 + j * 64);
          uint32_t d[4];
          dequant8<BITS, BLK>(W.tab[0], ring[i][0], j, d);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, av), as_f16x8(d[0], d[1], d[2], d[3]), acc,
                                                       0, 0, 0);
        }
      }
      W.load(c + DEPTH + i, c1, ring[i]);
    }
  }
  lds_barrier();                             // every wave has read its row's factor
  if (lane < 16) s_part[wave][lane] = acc[0] * f;
  lds_barrier();
  if (threadIdx.x < 64) {                    // quarters of the waves, then their sums
    const int n = lane & 15, w0 = (lane >> 4) * 4;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (w0 + i < nw) y += s_part[w0 + i][n];
    y += xor_lane_f32<16>(y);
    y += xor_lane_f32<32>(y);
    if (lane < 16) {
      if (a.y_bf16) static_cast<uint16_t*>(a.y)[n0 + n] = f32_to_bf16_rne(y);
      else static_cast<float*>(a.y)[n0 + n] = y;
    }
  }
}

// y[t] = sum_j w_j out[t * topk + j] + the shared rows.  One workgroup per token and 1024
// columns.
__global__ void __launch_bounds__(256)
few_combine_kernel(const float* __restrict__ rows, const float* __restrict__ wts, int T, int topk, int n_shared, int H,
                   void* __restrict__ y, int64_t ldy, int bf16) {
  const int t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= H) return;
  f32x4 r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < topk) r[j] = *reinterpret_cast<const f32x4*>(rows + (int64_t)(t * topk + j) * H + c);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < topk) acc += wts[t * topk + j] * r[j];
#pragma unroll 1
  for (int s = 0; s < n_shared; ++s)
    acc += *reinterpret_cast<const f32x4*>(rows + (int64_t)(T * topk + s * T + t) * H + c);
  if (bf16) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)f32_to_bf16_rne(acc[2 * i]) | ((uint32_t)f32_to_bf16_rne(acc[2 * i + 1]) << 16);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(y) + t * ldy + c) = u32x2{w[0], w[1]};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + t * ldy + c) = acc;
  }
}

// K is split until about 4096 waves share the sweep, while each keeps at least four chunks:
// half as many waves leave the down sweeps the same to 15 % slower (64 + 2 experts at 8 tokens
// 14.4 -> 16.6 us), twice as many all of them 18 % faster (the same experts' down at 32 tokens
// 27.5 -> 22.6 us) to 7 % slower (at 8 tokens 15.4 us); two or eight chunks at least: within 4 %.
template <int BITS, bool PAIR, bool BLK>
static hipError_t launch_few_gemm(const FewArgs& a, hipStream_t stream) {
  const int ys = (a.T * a.topk < a.E ? a.T * a.topk : a.E) + a.n_shared;
  const int tiles = PAIR ? a.N / 16 : (a.N + 31) / 32;
  const int nchunks = (a.K + 127) / 128;
  int SK = 1;
  while (SK < 8 && (int64_t)tiles * ys * SK < 4096 && SK * 4 <= nchunks) SK *= 2;
  const int CW = SK < 4 ? 4 / SK : 1;
  const dim3 grid((unsigned)((tiles + CW - 1) / CW), (unsigned)ys), block((unsigned)(64 * CW * SK));
  const size_t lds = (size_t)(SK - 1) * CW * 2 * 64 * sizeof(f32x4);
  hipLaunchKernelGGL((few_gemm_kernel<BITS, PAIR, BLK, 2>), grid, block, lds, stream, a, CW, SK);
  return hipGetLastError();
}

template <bool PAIR>
static hipError_t launch_few_bits(const FewArgs& a, int bits, hipStream_t s) {
  if (bits == 4) return launch_few_gemm<4, PAIR, false>(a, s);
  if (bits == 2) return launch_few_gemm<2, PAIR, false>(a, s);
  return a.blocked ? launch_few_gemm<3, PAIR, true>(a, s) : launch_few_gemm<3, PAIR, false>(a, s);
}

template <int BITS, int ABITS, bool BLK>
static hipError_t launch_gate_one(const FewArgs& a, hipStream_t stream) {
  const int nchunks = (a.K + 127) / 128;
  int SK = 1;
  while (SK < 8 && SK * 4 <= nchunks) SK *= 2;
  const dim3 grid((unsigned)(a.N / 16), (unsigned)(a.topk + a.n_shared));
  hipLaunchKernelGGL((few_gate_one_kernel<BITS, ABITS, BLK, 2>), grid, dim3(64 * SK), 0, stream, a, SK);
  return hipGetLastError();
}

template <int ABITS>
static hipError_t launch_gate_one_bits(const FewArgs& a, int bits, hipStream_t s) {
  if (bits == 4) return launch_gate_one<4, ABITS, false>(a, s);
  if (bits == 2) return launch_gate_one<2, ABITS, false>(a, s);
  return a.blocked ? launch_gate_one<3, ABITS, true>(a, s) : launch_gate_one<3, ABITS, false>(a, s);
}

template <int BITS, bool BLK>
static hipError_t launch_down_one(const FewDownArgs& a, hipStream_t stream) {
  const int R = a.topk + a.n_shared, nchunks = (a.F + 127) / 128;
  int ksh = 0;
  while (R << (ksh + 1) <= 16 && (2 << ksh) <= nchunks) ++ksh;
  // fp16 codes and the transform's values of every row
  const size_t lds = (size_t)R * (few_row16_bytes(a.F) + (a.F + 255) / 256 * 256 * one_token_value_bytes(a.F));
  hipLaunchKernelGGL((few_down_one_kernel<BITS, BLK, 4>), dim3((unsigned)(a.H / 16)), dim3((unsigned)(64 * R << ksh)), lds,
                     stream, a, ksh);
  return hipGetLastError();
}

// The one-token form: its rows have a wave each, which transforms F values, and all of them
// together their codes and values in LDS (at most 120 KB at these limits).  Beyond the limits
// that repeated work costs more than the batch form's three launches (4 bits, us a call in a
// graph, this form / batch): 8 rows of 768 17.6 / 24.1, 8 of 1408 24.9 / 28.4, 8 of 1536 27.0 /
// 28.8, 6 of 2048 30.2 / 30.0, 2 of 2048 18.6 / 19.8, 2 of 4096 31.3 / 25.4.
static bool one_token_form(int64_t T, int topk, int n_shared, int F) {
  const int R = topk + n_shared;
  return T == 1 && R <= 16 && F <= 2048 && R * F <= 12288;
}

// Workspace: ids and weights, the input's fp16 codes, then h, its fp16 codes and scales, then
// the expert rows, each 256-byte aligned.
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
struct FewLayout {
  size_t wts, x16, h, h16, scales, rows, bytes;
  FewLayout(int64_t T, int topk, int n_shared, int H, int F) {
    const size_t R = (size_t)T * (topk + n_shared);
    wts = up256((size_t)T * topk * 4);
    x16 = wts + up256((size_t)T * topk * 4);
    h = x16 + up256((size_t)T * few_row16_bytes(H));
    h16 = h + up256(R * F * 4);
    scales = h16 + up256(R * few_row16_bytes(F));
    rows = scales + up256(R * 4);
    bytes = rows + up256(R * H * 4);
  }
};

size_t moe_few_workspace_bytes(int64_t T, int topk, int n_shared, int H, int F) {
  return FewLayout(T, topk, n_shared, H, F).bytes;
}

hipError_t launch_moe_few(const MoeFewArgs& m, hipStream_t stream) {
  const FewLayout L(m.T, m.topk, m.n_shared, m.H, m.F);
  uint8_t* ws = static_cast<uint8_t*>(m.ws);
  int32_t* ids = reinterpret_cast<int32_t*>(ws);
  float* wts = reinterpret_cast<float*>(ws + L.wts);
  const int R = m.T * (m.topk + m.n_shared);
  FewArgs a{};
  a.logits = m.logits; a.ids = ids; a.T = m.T; a.E = m.E; a.topk = m.topk; a.n_shared = m.n_shared;
  a.scales = m.scales; a.w[0] = m.gate; a.w[1] = m.up; a.N = m.F; a.K = m.H;
  a.blocked = m.blocked_gu; a.out = reinterpret_cast<float*>(ws + L.h);
  const float c_b = (float)(1.0 / std::sqrt((double)(m.F & -m.F)));
  hipError_t e;
  if (one_token_form(m.T, m.topk, m.n_shared, m.F)) {
    a.codes = m.codes;
    e = m.act_bits == 4 ? launch_gate_one_bits<4>(a, m.bits_gu, stream) : launch_gate_one_bits<8>(a, m.bits_gu, stream);
    if (e != hipSuccess) return e;
    FewDownArgs d{};
    d.h = a.out; d.ids = ids; d.logits = m.logits; d.E = m.E; d.topk = m.topk; d.n_shared = m.n_shared;
    d.renormalize = m.renormalize; d.act_bits = m.act_bits; d.H = m.H; d.F = m.F; d.w = m.down; d.blocked = m.blocked_d;
    d.c_b = c_b; d.y = m.y; d.y_bf16 = m.y_bf16;
    if (m.bits_d == 4) return launch_down_one<4, false>(d, stream);
    if (m.bits_d == 2) return launch_down_one<2, false>(d, stream);
    return m.blocked_d ? launch_down_one<3, true>(d, stream) : launch_down_one<3, false>(d, stream);
  }
  if (m.act_bits == 4)
    hipLaunchKernelGGL(few_prepare_kernel<4>, dim3((unsigned)m.T), dim3(256), 0, stream, m.logits, m.T, m.E, m.topk,
                       m.renormalize, m.codes, m.H, ids, wts, ws + L.x16);
  else
    hipLaunchKernelGGL(few_prepare_kernel<8>, dim3((unsigned)m.T), dim3(256), 0, stream, m.logits, m.T, m.E, m.topk,
                       m.renormalize, m.codes, m.H, ids, wts, ws + L.x16);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.codes = ws + L.x16;
  e = launch_few_bits<true>(a, m.bits_gu, stream);
  if (e != hipSuccess) return e;
  NormArgs n{};
  n.rows = ws + L.h; n.ldr = m.F; n.codes = ws + L.h16; n.scales = reinterpret_cast<float*>(ws + L.scales);
  n.act_bits = m.act_bits; n.T = R; n.K = m.F;
  e = launch_norm_quantize(n, kRotateF32, m.F & -m.F, stream);
  if (e != hipSuccess) return e;
  a.codes = ws + L.h16; a.scales = reinterpret_cast<float*>(ws + L.scales); a.w[0] = a.w[1] = m.down;
  a.N = m.H; a.K = m.F; a.blocked = m.blocked_d; a.out = reinterpret_cast<float*>(ws + L.rows);
  e = launch_few_bits<false>(a, m.bits_d, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_combine_kernel, dim3((unsigned)m.T, (unsigned)((m.H + 1023) / 1024)), dim3(256), 0, stream,
                     reinterpret_cast<const float*>(ws + L.rows), wts, m.T, m.topk, m.n_shared, m.H, m.y, m.ldy, m.y_bf16);
  return hipGetLastError();
}

}  // namespace cbq
