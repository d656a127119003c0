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

// Weights 8 j .. 8 j + 7 of a lane's 32 raw indices, in the order the code conversion gives.
template <int BITS, bool BLK>
__device__ __forceinline__ void dequant8(const RowTable<BITS>& t, const uint32_t (&w)[BITS], int j, uint32_t* d) {
  if constexpr (BITS == 4) {
    dequant4(t, w[j], d);
  } else if constexpr (BITS == 3 && BLK) {
    dequant3_blk(t, j < 3 ? w[j] : group3_blk(w), d);
  } else if constexpr (BITS == 3) {
    dequant3(t, j == 0 ? w[0] : j == 1 ? __builtin_amdgcn_alignbit(w[1], w[0], 24)
                     : j == 2 ? __builtin_amdgcn_alignbit(w[2], w[1], 16) : w[2] >> 8, d);
  } else {
    uint32_t both[8];
    dequant2(t, w[j >> 1], both);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = both[4 * (j & 1) + i];
  }
}

// One wave's view of its weights.
template <int BITS, int NW>
struct FewWeights {
  RowTable<BITS> tab[NW];
  __amdgpu_buffer_rsrc_t res[NW];
  uint32_t lane_off[NW];                     // byte offset of the lane's first indices, kOffNone: no row
  uint32_t step;                             // bytes between chunks
  int K, g;

  // e: expert; n0: the wave's first weight row (n0 < N, or the wave has no rows); pair: the
  // NW sets are NW consecutive groups of 16 rows of one matrix instead of NW matrices
  __device__ __forceinline__ void init(const GemmW* w, bool pair, int e, int n0, int N, int K_, int blocked, int lane) {
    K = K_;
    g = lane >> 4;
    const int nl = lane & 15;
    const int64_t row_bytes = index_row_bytes(K, BITS, blocked != 0);
    step = blocked ? 256u * BITS : 16u * BITS;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int nb = pair ? n0 + 16 * i : n0;
      const bool ok = nb < N;
      const int n = ok ? nb + nl : 0;
      lane_off[i] = !ok ? kOffNone
                    : blocked ? (uint32_t)(nb * row_bytes) + (uint32_t)(lane * 4 * BITS)
                              : (uint32_t)(n * row_bytes) + (uint32_t)(g * 4 * BITS);
      const GemmW& m = w[pair ? 0 : i];
      tab[i].load(m.codebook + ((int64_t)e * N + n) * (1 << BITS));
      res[i] = make_rsrc(m.idx + (int64_t)e * N * row_bytes, (uint32_t)(N * row_bytes));
    }
  }
  // chunk c's raw indices; past c_end or K they read as zeros, which the zero codes cancel
  __device__ __forceinline__ void load(int c, int c_end, uint32_t (&w)[NW][BITS]) const {
    const bool ok = c < c_end && c * 128 + g * 32 < K;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      buf_load<4 * BITS>(res[i], ok ? lane_off[i] : kOffNone, w[i], (uint32_t)c * step);
  }
};

// The sweep over chunks [c0, c1) for NSUB live sub-tiles.  ring holds the first DEPTH chunks'
// raw indices; aoff[s] is the byte offset of the lane's code row (and slice) of sub-tile s,
// kOffNone where there is none.
template <int BITS, int ABITS, int NW, bool BLK, int NSUB, int DEPTH>
__device__ __forceinline__ void few_sweep(const FewWeights<BITS, NW>& W, uint32_t (&ring)[DEPTH][NW][BITS],
                                          __amdgpu_buffer_rsrc_t cres, const uint32_t* aoff, int c0, int c1,
                                          f32x4 (&acc)[NW][2]) {
  // the codes are in L2 (a few rows that every workgroup reads), so a shorter ring serves them
  constexpr int CD = DEPTH < 2 ? 1 : 2;
  static_assert(DEPTH % CD == 0, "the codes' ring must divide the weights'");
  uint32_t ca[CD][NSUB][ABITS];
  auto load_codes = [&](int c, uint32_t (&d)[NSUB][ABITS]) {
    const bool ok = c < c1 && c * 128 + W.g * 32 < W.K;
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
      for (int h = 0; h < ABITS / 4; ++h)
        buf_load<16>(cres, ok ? aoff[s] + 16 * h : kOffNone, &d[s][4 * h], (uint32_t)(c * 128 * ABITS / 8));
  };
  auto chunk = [&](const uint32_t (&w)[NW][BITS], const uint32_t (&a)[NSUB][ABITS]) {
    // 8 channels a lane at a time, so few converted values are live at once
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f16x8 A[NSUB];
#pragma unroll
      for (int s = 0; s < NSUB; ++s) {
        uint32_t d[4];
        codes8_group<ABITS, false>(a[s], j, d);
        A[s] = as_f16x8(d[0], d[1], d[2], d[3]);
      }
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        uint32_t d[4];
        dequant8<BITS, BLK>(W.tab[i], w[i], j, d);
        const f16x8 B = as_f16x8(d[0], d[1], d[2], d[3]);
#pragma unroll
        for (int s = 0; s < NSUB; ++s) acc[i][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A[s], B, acc[i][s], 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < CD; ++i) load_codes(c0 + i, ca[i]);
  int c = c0;
  for (; c + DEPTH - 1 < c1; c += DEPTH) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      chunk(ring[i], ca[i % CD]);
      W.load(c + DEPTH + i, c1, ring[i]);
      load_codes(c + CD + i, ca[i % CD]);
      __builtin_amdgcn_sched_barrier(0);     // keeps later chunks' conversions out of this one
    }
  }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) {
    if (c + i < c1) {
      chunk(ring[i], ca[i % CD]);
      if (i + CD < DEPTH - 1) load_codes(c + CD + i, ca[i % CD]);
    }
  }
}

// Row codes already converted to fp16, in the order the weights are dequantised to: row r,
// 128-channel chunk c, group j of 8 channels of slice g (channels 128 c + 32 g + 8 j ..) is the
// 16 bytes at r * 2 Kp + 256 c + 64 j + 16 g (Kp: K rounded up to 128, zeros past K).
__host__ __device__ inline int64_t few_row16_bytes(int K) { return (int64_t)((K + 127) / 128) * 256; }

__device__ __forceinline__ uint32_t few_pos16(int c) {   // byte of channel c's group
  return (uint32_t)((c >> 7) * 256 + ((c & 31) >> 3) * 64 + ((c & 127) >> 5) * 16);
}

// The sweep of few_sweep over such rows, one sub-tile: no conversions, a third of the vector
// work of a single 4-bit matrix.  Each group's registers are refilled with the next chunk's as
// soon as they are used.  aoff: byte offset of the lane's row and slice, kOffNone: none.
template <int BITS, int NW, bool BLK, int DEPTH>
__device__ __forceinline__ void few_sweep16(const FewWeights<BITS, NW>& W, uint32_t (&ring)[DEPTH][NW][BITS],
                                            __amdgpu_buffer_rsrc_t cres, uint32_t aoff, int c0, int c1, f32x4 (&acc)[NW]) {
  uint32_t a[4][4];
  auto load_a = [&](int c, int j) { buf_load<16>(cres, c < c1 ? aoff + 64 * j : kOffNone, a[j], (uint32_t)(c * 256)); };
  auto chunk = [&](int c, const uint32_t (&w)[NW][BITS]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        uint32_t d[4];
        dequant8<BITS, BLK>(W.tab[i], w[i], j, d);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_f16x8(a[j][0], a[j][1], a[j][2], a[j][3]),
                                                        as_f16x8(d[0], d[1], d[2], d[3]), acc[i], 0, 0, 0);
      }
      load_a(c + 1, j);
    }
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) load_a(c0, j);
  int c = c0;
  for (; c + DEPTH - 1 < c1; c += DEPTH) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      chunk(c + i, ring[i]);
      W.load(c + DEPTH + i, c1, ring[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i)
    if (c + i < c1) chunk(c + i, ring[i]);
}

// Adds the K splits' sums in split order into the first split's wave, through LDS; every wave
// of the workgroup calls it.  red: [(SK - 1) * CW][NACC][64].
template <int NACC>
__device__ __forceinline__ void few_reduce(f32x4* red, int cw, int sk, int SK, int lane, f32x4 (&acc)[NACC]) {
  if (SK == 1) return;
  f32x4* mine = red + (size_t)cw * (SK - 1) * NACC * 64 + lane;
  if (sk > 0) {
#pragma unroll
    for (int i = 0; i < NACC; ++i) mine[((sk - 1) * NACC + i) * 64] = acc[i];
  }
  lds_barrier();
  if (sk == 0) {
#pragma unroll 4
    for (int v = 0; v < SK - 1; ++v)
#pragma unroll
      for (int i = 0; i < NACC; ++i) acc[i] += mine[(v * NACC + i) * 64];
  }
}

}  // namespace cbq
