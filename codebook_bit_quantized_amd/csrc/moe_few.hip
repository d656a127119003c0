// The whole MoE layer for a few tokens (a decode batch): routing, gate/up with SwiGLU, the
// rotation and quantisation of h, down and the weighted combine.
//
// CodeQuant2, Figures 3 and 4 (codebook weights looked up in on-chip tables); the AI Radio
// episode, introduction (a router in front of the experts).
//
// At one to 32 tokens the layer is a few launches that each read weights once, and what it
// costs beyond those bytes is launches and dependent loads.  So there is no routing kernel and
// there are no row lists in memory: every workgroup of the gate/up kernel finds the rows of its
// expert from the logits (the rank of expert e in a token's logits is the number of experts
// ahead of it), and rows are numbered by choice (row t * topk + j is token t's j-th choice,
// row T * topk + s * T + t shared expert s), which needs no counting.  Kernels:
//   1. gate/up: h = silu(g) * u in fp32, and the chosen ids;
//   2. rotation and quantisation of h's rows (norm_quantize.hip, without the norm);
//   3. down: the rows of its expert found from the ids;
//   4. the weighted sum of each token's rows, with the softmax weights from the logits.
// h is kept in fp32 up to the quantiser: the codes are those of the unrounded h up to fp32
// sums (a bf16 h would move a code wherever its rounding crosses a border).
#include "cbq_internal.hpp"
#include "few_device.hpp"
#include "route_device.hpp"

namespace cbq {

namespace {

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

// the expert of rank j in a token's logits (ties to the lower id); whole waves only
__device__ __forceinline__ int expert_of_rank(const float* row, int E, int j, int lane) {
  uint32_t key[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? order_bits(row[e]) : 0u;
  }
  int e = 0;
  for (int r = 0; r <= j; ++r) {
    const uint32_t m = wave_max_u32(max(max(key[0], key[1]), max(key[2], key[3])));
    e = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint64_t at = __ballot(key[i] == m);
      if (at) e = 64 * i + __builtin_ctzll(at);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i == e) key[i] = 0u;
  }
  return e;
}

// the rank of expert e in a token's logits; whole waves only
__device__ __forceinline__ int rank_of_expert(const float* row, int E, int e, int lane) {
  const uint32_t ke = order_bits(row[e]);
  int n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = lane + 64 * i;
    bool ahead = false;
    if (o < E) {
      const uint32_t k = order_bits(row[o]);
      ahead = k > ke || (k == ke && o < e);
    }
    n += __popcll(__ballot(ahead));
  }
  return n;
}

}  // namespace

// Rows of this workgroup's expert, in LDS: code row and output row of each.
struct FewRows {
  int n, e;
  int16_t code[kFewRows], out[kFewRows];
  int16_t rank[kFewRows];
};

// PAIR: the gate/up kernel (rows from the logits; writes h and ids), else the down kernel
// (rows from the ids; writes the expert rows).  Workgroups of CW * SK waves: CW column tiles
// of 16 weight rows, each with K split over SK waves.
template <int BITS, int ABITS, bool PAIR, bool BLK, int DEPTH>
__global__ void __launch_bounds__(PAIR ? 512 : 1024)
few_gemm_kernel(FewArgs a, int CW, int SK) {
  constexpr int NW = PAIR ? 2 : 1;
  extern __shared__ f32x4 red[];
  __shared__ FewRows s_rows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nwaves = CW * SK;
  const int cw = wave / SK, sk = wave - cw * SK;
  const int T = a.T, E = a.E, topk = a.topk;
  // shared experts, which every token visits, come last in y and are started first
  const int y = (int)(gridDim.y - 1 - blockIdx.y);
  const int routed = (int)gridDim.y - a.n_shared;
  const bool by_choice = routed < E;         // one y per choice (t, j) instead of one per expert
  const bool shared = y >= routed;

  int e = shared ? E + y - routed : y;
  if (by_choice && !shared) {
    if constexpr (PAIR) {
      e = expert_of_rank(a.logits + (int64_t)(y / topk) * E, E, y % topk, lane);
    } else {
      e = a.ids[y];
      if ((uint32_t)e >= (uint32_t)E) return;       // only where logits were not numbers
    }
  }
  const int n0 = (blockIdx.x * CW + cw) * 16;
  const int nchunks = (a.K + 127) >> 7;
  const int cpw = (nchunks + SK - 1) / SK;
  const int c0 = sk * cpw, c1 = min(nchunks, c0 + cpw);
  FewWeights<BITS, NW> W;
  W.init(a.w, e, n0, a.N, a.K, a.blocked, lane);
  uint32_t ring[DEPTH][NW][BITS];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);

  // ---- the expert's rows ----
  if (shared) {
    if (threadIdx.x < T) {
      const int row = T * topk + (y - routed) * T + threadIdx.x;
      s_rows.code[threadIdx.x] = (int16_t)(PAIR ? threadIdx.x : row);
      s_rows.out[threadIdx.x] = (int16_t)row;
    }
    if (threadIdx.x == 0) s_rows.n = T;
  } else if constexpr (PAIR) {
    for (int t = wave; t < T; t += nwaves) {
      const int r = T == 1 && by_choice ? y : rank_of_expert(a.logits + (int64_t)t * E, E, e, lane);
      if (lane == 0) s_rows.rank[t] = (int16_t)(r < topk ? r : -1);
    }
    lds_barrier();
    if (wave == 0) {
      const int r = lane < T ? s_rows.rank[lane] : -1;
      const uint64_t mine = __ballot(r >= 0);
      if (r >= 0) {
        const int p = __popcll(mine & ((1ull << lane) - 1));
        s_rows.code[p] = (int16_t)lane;
        s_rows.out[p] = (int16_t)(lane * topk + r);
        if (blockIdx.x == 0) a.ids[lane * topk + r] = e;
      }
      // by choice, the first token that chose the expert works for all of them
      if (lane == 0) s_rows.n = by_choice && mine && __builtin_ctzll(mine) != y / topk ? 0 : __popcll(mine);
    }
  } else {
    if (wave == 0) {
      int n = 0;
      for (int base = 0; base < T * topk; base += 64) {
        const int p = base + lane;
        const bool is = p < T * topk && a.ids[p] == e;
        const uint64_t mine = __ballot(is);
        const int at = n + __popcll(mine & ((1ull << lane) - 1));
        if (is && at < kFewRows) {
          s_rows.code[at] = (int16_t)p;
          s_rows.out[at] = (int16_t)p;
        }
        n += __popcll(mine);
      }
      if (lane == 0) s_rows.n = min(n, kFewRows);
    }
    lds_barrier();
    if (by_choice && s_rows.n > 0 && s_rows.out[0] != y) return;   // an earlier choice works for it
  }
  lds_barrier();
  const int me = s_rows.n;
  if (me == 0) return;

  // ---- the products ----
  f32x4 acc[NW][2];
#pragma unroll
  for (int i = 0; i < NW; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t code_bytes = (int64_t)a.K * ABITS / 8;
  uint32_t aoff[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int m = s * 16 + (lane & 15);
    aoff[s] = m < me ? (uint32_t)(s_rows.code[m] * code_bytes) + (uint32_t)((lane >> 4) * 4 * ABITS) : kOffNone;
  }
  const __amdgpu_buffer_rsrc_t cres = make_rsrc(a.codes, 0x7FFFFFFFu);
  if (me > 16) few_sweep<BITS, ABITS, NW, BLK, 2, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
  else few_sweep<BITS, ABITS, NW, BLK, 1, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
  few_reduce<NW>(red, cw, sk, SK, me > 16 ? 2 : 1, lane, acc);

  // lane holds D[m = 4 * (lane >> 4) + i][n = lane & 15]
  if (sk != 0 || n0 >= a.N) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = s * 16 + 4 * (lane >> 4) + i;
      if (m >= me) continue;
      const float sc = a.scales[s_rows.code[m]];
      float v = acc[0][s][i] * sc;
      if constexpr (PAIR) {
        // silu(g) * u with the accurate exponential and division: its error moves codes of h
        const float u = acc[NW - 1][s][i] * sc;
        v = v / (1.0f + expf(-v)) * u;
      }
      a.out[(int64_t)s_rows.out[m] * a.N + n0 + (lane & 15)] = v;
    }
  }
}

// y[t] = sum_j w_j out[t * topk + j] + the shared rows, w the softmax over the chosen logits
// (or over all).  One workgroup per token and 1024 columns.
__global__ void __launch_bounds__(256)
few_combine_kernel(const float* __restrict__ rows, const float* __restrict__ logits, const int32_t* __restrict__ ids,
                   int T, int E, int topk, int n_shared, int renormalize, int H, void* __restrict__ y, int64_t ldy,
                   int bf16) {
  __shared__ float s_w[8];
  const int t = blockIdx.x, lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    const float* lg = logits + (int64_t)t * E;
    int id = lane < topk ? ids[t * topk + lane] : 0;
    id = (uint32_t)id < (uint32_t)E ? id : 0;       // only where logits were not numbers
    const float l = lane < topk ? lg[id] : -INFINITY;
    const float top = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l), 0));
    const float ex = lane < topk ? expf(l - top) : 0.0f;
    float den = ex;
    if (!renormalize) {
      den = 0.0f;
      for (int e = lane; e < E; e += 64) den += expf(lg[e] - top);
    }
    for (int m = 32; m >= 1; m >>= 1) den += __shfl_xor(den, m);
    if (lane < topk) s_w[lane] = ex / den;
  }
  __syncthreads();
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= H) return;
  f32x4 r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < topk) r[j] = *reinterpret_cast<const f32x4*>(rows + (int64_t)(t * topk + j) * H + c);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < topk) acc += s_w[j] * r[j];
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

template <int BITS, int ABITS, bool PAIR, bool BLK>
static hipError_t launch_few_gemm(const FewArgs& a, hipStream_t stream) {
  constexpr int NW = PAIR ? 2 : 1;
  const int ys = (a.T * a.topk < a.E ? a.T * a.topk : a.E) + a.n_shared;
  const int tiles = a.N / 16;
  const int nchunks = (a.K + 127) / 128;
  int SK = 1;
  while (SK < (PAIR ? 8 : 16) && (int64_t)tiles * ys * SK < 2048 && SK * 8 <= nchunks) SK *= 2;
  int CW = 4 / SK;
  if (CW < 1) CW = 1;
  const dim3 grid((unsigned)((tiles + CW - 1) / CW), (unsigned)ys), block((unsigned)(64 * CW * SK));
  const size_t lds = (size_t)(SK - 1) * CW * NW * 2 * 64 * sizeof(f32x4);
  hipLaunchKernelGGL((few_gemm_kernel<BITS, ABITS, PAIR, BLK, 4>), grid, block, lds, stream, a, CW, SK);
  return hipGetLastError();
}

template <bool PAIR>
static hipError_t launch_few_bits(const FewArgs& a, int bits, int act_bits, hipStream_t s) {
  const bool blk = a.blocked != 0;
  if (act_bits == 4) {
    if (bits == 4) return launch_few_gemm<4, 4, PAIR, false>(a, s);
    if (bits == 2) return launch_few_gemm<2, 4, PAIR, false>(a, s);
    return blk ? launch_few_gemm<3, 4, PAIR, true>(a, s) : launch_few_gemm<3, 4, PAIR, false>(a, s);
  }
  if (bits == 4) return launch_few_gemm<4, 8, PAIR, false>(a, s);
  if (bits == 2) return launch_few_gemm<2, 8, PAIR, false>(a, s);
  return blk ? launch_few_gemm<3, 8, PAIR, true>(a, s) : launch_few_gemm<3, 8, PAIR, false>(a, s);
}

// Workspace: ids, then h, its codes and scales, then the expert rows, each 256-byte aligned.
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
struct FewLayout {
  size_t h, codes, scales, rows, bytes;
  FewLayout(int64_t T, int topk, int n_shared, int H, int F, int act_bits) {
    const size_t R = (size_t)T * (topk + n_shared);
    h = up256((size_t)T * topk * 4);
    codes = h + up256(R * F * 4);
    scales = codes + up256(R * (size_t)F * act_bits / 8);
    rows = scales + up256(R * 4);
    bytes = rows + up256(R * H * 4);
  }
};

size_t moe_few_workspace_bytes(int64_t T, int topk, int n_shared, int H, int F, int act_bits) {
  return FewLayout(T, topk, n_shared, H, F, act_bits).bytes;
}

hipError_t launch_moe_few(const MoeFewArgs& m, hipStream_t stream) {
  const FewLayout L(m.T, m.topk, m.n_shared, m.H, m.F, m.act_bits);
  uint8_t* ws = static_cast<uint8_t*>(m.ws);
  int32_t* ids = reinterpret_cast<int32_t*>(ws);
  const int R = m.T * (m.topk + m.n_shared);
  FewArgs a{};
  a.logits = m.logits; a.ids = ids; a.T = m.T; a.E = m.E; a.topk = m.topk; a.n_shared = m.n_shared;
  a.codes = m.codes; a.scales = m.scales; a.w[0] = m.gate; a.w[1] = m.up; a.N = m.F; a.K = m.H;
  a.blocked = m.blocked_gu; a.out = reinterpret_cast<float*>(ws + L.h);
  hipError_t e = launch_few_bits<true>(a, m.bits_gu, m.act_bits, stream);
  if (e != hipSuccess) return e;
  NormArgs n{};
  n.rows = ws + L.h; n.ldr = m.F; n.codes = ws + L.codes; n.scales = reinterpret_cast<float*>(ws + L.scales);
  n.act_bits = m.act_bits; n.T = R; n.K = m.F;
  e = launch_norm_quantize(n, kRotateF32, m.F & -m.F, stream);
  if (e != hipSuccess) return e;
  a.codes = ws + L.codes; a.scales = reinterpret_cast<float*>(ws + L.scales); a.w[0] = a.w[1] = m.down;
  a.N = m.H; a.K = m.F; a.blocked = m.blocked_d; a.out = reinterpret_cast<float*>(ws + L.rows);
  e = launch_few_bits<false>(a, m.bits_d, m.act_bits, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_combine_kernel, dim3((unsigned)m.T, (unsigned)((m.H + 1023) / 1024)), dim3(256), 0, stream,
                     reinterpret_cast<const float*>(ws + L.rows), m.logits, ids, m.T, m.E, m.topk, m.n_shared,
                     m.renormalize, m.H, m.y, m.ldy, m.y_bf16);
  return hipGetLastError();
}

}  // namespace cbq
