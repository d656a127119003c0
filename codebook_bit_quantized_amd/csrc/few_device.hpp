// The codebook GEMM of a few rows, shared by the few-token MoE layer and the projection with
// adapters (gfx950, wave64).
//
// A wave owns 16 weight rows n (of each matrix of a gate/up pair) and a range of 128-channel
// chunks; lane l serves row n0 + (l & 15) and channels 32 (l >> 4) .. + 31 of each chunk, so a
// chunk of the blocked layout is one coalesced load of 64 * 4 * BITS bytes per matrix.  The
// lane's codebook row sits in registers as byte tables (v_perm lookups); the dequantised
// weights are the B operand of 16x16x32 fp16 MFMAs whose A operand holds up to 16 rows' codes
// (one or two such sub-tiles share each dequantised weight).  Products are exact; sums are
// fp32.
//
// What bounds it is the latency of a short sweep, then HBM: a wave has few chunks, so the
// first DEPTH chunks' weights (which depend on the expert alone) are requested before the
// rows are known, and the ring is refilled as it is used.
#pragma once
#include "cbq_internal.hpp"

namespace cbq {

constexpr int kFewRows = 32;                 // rows of one expert at most: two 16-row sub-tiles

// One wave's view of its weights.
template <int BITS, int NW>
struct FewWeights {
  RowTable<BITS> tab[NW];
  __amdgpu_buffer_rsrc_t res[NW];
  uint32_t lane_off;                         // byte offset of the lane's first indices, kOffNone: no row
  uint32_t step;                             // bytes between chunks
  int K, g;

  // e: expert; n0: the wave's first weight row (n0 < N, or the wave has no rows)
  __device__ __forceinline__ void init(const GemmW* w, int e, int n0, int N, int K_, int blocked, int lane) {
    K = K_;
    g = lane >> 4;
    const int nl = lane & 15;
    const int64_t row_bytes = index_row_bytes(K, BITS, blocked != 0);
    const bool ok = n0 < N;
    const int n = ok ? n0 + nl : 0;
    lane_off = !ok ? kOffNone
               : blocked ? (uint32_t)(n0 * row_bytes) + (uint32_t)(lane * 4 * BITS)
                         : (uint32_t)(n * row_bytes) + (uint32_t)(g * 4 * BITS);
    step = blocked ? 256u * BITS : 16u * BITS;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      tab[i].load(w[i].codebook + ((int64_t)e * N + n) * (1 << BITS));
      res[i] = make_rsrc(w[i].idx + (int64_t)e * N * row_bytes, (uint32_t)(N * row_bytes));
    }
  }
  // chunk c's raw indices; past c_end or K they read as zeros, which the zero codes cancel
  __device__ __forceinline__ void load(int c, int c_end, uint32_t (&w)[NW][BITS]) const {
    const bool ok = c < c_end && c * 128 + g * 32 < K;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      buf_load<4 * BITS>(res[i], ok ? lane_off : kOffNone, w[i], (uint32_t)c * step);
  }
};

// The sweep over chunks [c0, c1) for NSUB live sub-tiles.  ring holds the first DEPTH chunks'
// raw indices; aoff[s] is the byte offset of the lane's code row (and slice) of sub-tile s,
// kOffNone where there is none.
template <int BITS, int ABITS, int NW, bool BLK, int NSUB, int DEPTH>
__device__ __forceinline__ void few_sweep(const FewWeights<BITS, NW>& W, uint32_t (&ring)[DEPTH][NW][BITS],
                                          __amdgpu_buffer_rsrc_t cres, const uint32_t* aoff, int c0, int c1,
                                          f32x4 (&acc)[NW][2]) {
  uint32_t ca[DEPTH][NSUB][ABITS];
  auto load_codes = [&](int c, uint32_t (&d)[NSUB][ABITS]) {
    const bool ok = c < c1 && c * 128 + W.g * 32 < W.K;
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
      for (int h = 0; h < ABITS / 4; ++h)
        buf_load<16>(cres, ok ? aoff[s] + 16 * h : kOffNone, &d[s][4 * h], (uint32_t)(c * 128 * ABITS / 8));
  };
  auto chunk = [&](const uint32_t (&w)[NW][BITS], const uint32_t (&a)[NSUB][ABITS]) {
    uint32_t ad[NSUB][16], bd[NW][16];
#pragma unroll
    for (int s = 0; s < NSUB; ++s) codes32_to_f16<ABITS>(a[s], ad[s]);
#pragma unroll
    for (int i = 0; i < NW; ++i) dequant32<BITS, BLK>(W.tab[i], w[i], bd[i]);
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const f16x8 A = as_f16x8(ad[s][4 * j], ad[s][4 * j + 1], ad[s][4 * j + 2], ad[s][4 * j + 3]);
          const f16x8 B = as_f16x8(bd[i][4 * j], bd[i][4 * j + 1], bd[i][4 * j + 2], bd[i][4 * j + 3]);
          acc[i][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A, B, acc[i][s], 0, 0, 0);
        }
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) load_codes(c0 + i, ca[i]);
  int c = c0;
  for (; c + DEPTH - 1 < c1; c += DEPTH) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      chunk(ring[i], ca[i]);
      W.load(c + DEPTH + i, c1, ring[i]);
      load_codes(c + DEPTH + i, ca[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i)
    if (c + i < c1) chunk(ring[i], ca[i]);
}

// Adds the K splits' sums in split order into the first split's wave, through LDS; every wave
// of the workgroup calls it.  red: [(SK - 1) * CW][NW][2][64].
template <int NW>
__device__ __forceinline__ void few_reduce(f32x4* red, int cw, int sk, int SK, int nsub, int lane, f32x4 (&acc)[NW][2]) {
  if (SK == 1) return;
  if (sk > 0) {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s < nsub) red[(((cw * (SK - 1) + sk - 1) * NW + i) * 2 + s) * 64 + lane] = acc[i][s];
  }
  lds_barrier();
  if (sk == 0) {
    for (int v = 0; v < SK - 1; ++v)
#pragma unroll
      for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (s < nsub) acc[i][s] += red[(((cw * (SK - 1) + v) * NW + i) * 2 + s) * 64 + lane];
  }
}

}  // namespace cbq
