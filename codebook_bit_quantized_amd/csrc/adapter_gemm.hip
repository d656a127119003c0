// A shared codebook projection with low-rank adapters of many requests beside it:
//   out[t] = scale_t * sum_k q[t][k] W[n][k]  +  s_a * B_a (A_a x[t]),   a = adapter_of[t].
//
// CodeQuant2, Figure 3 (the projection's codebook weights); the adapters are full-precision
// updates trained beside frozen quantised weights.
//
// Two launches.  The first forms u[t] = s_a A_a x[t] (fp32, [T][rank]) for every token that
// has an adapter; the second is the projection, whose epilogue adds B_a u[t] before the only
// store of out, so the adapters cost no pass over out.  A tile works through the distinct
// adapters among its own tokens (one or two where requests are contiguous, up to one a token in
// a decode batch), with results taken only for the tokens of that adapter, so another adapter's
// infinities never reach a token.  Beyond a decode batch, tiles of both launches take their
// group's tokens by adapter (order_by_adapter), which no result depends on: 4096 tokens in
// random order over 32 adapters of rank 64 168 + 549 us without, 66 + 418 with.
#include "cbq_internal.hpp"
#include "adapter_device.hpp"
#include "few_device.hpp"

namespace cbq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// u = s_a A_a x for 16 tokens (ORDER: of a group of 256 in their order by adapter) and RT * 16
// rank rows, part z of K.  Workgroup (tile, y, z): the distinct adapters y, y + ny, ... of the
// tile, rank rows from 16 RT (z / parts) on, channels of part z % parts; the waves split those
// and their sums meet in LDS in wave order.  The parts are summed by the projection.  Bound by
// load latency in a decode batch (so K is cut into enough parts to have all of an adapter's
// rows in flight at once: 16 tokens, K = 9728, rank 32, 16 adapters, 10 MB: 23.5 us in one part,
// 5.5 in 16), by its short sweeps in a prefill batch (4096 x 2560, rank 16: 21 MB of x in 13 us).
template <int RT, bool ORDER>
__global__ void __launch_bounds__(256)
adapter_shrink_kernel(AdapterArgs a, const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ lora_a,
                      const float* __restrict__ adapter_scale, int64_t T, int K, float* __restrict__ u) {
  __shared__ f32x4 red[3][RT][64];
  __shared__ __attribute__((aligned(16))) uint32_t s_key[ORDER ? 256 : 1];
  __shared__ int s_tok[16], s_of[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  // neighbouring tiles, which mostly share adapters, on one XCD
  const int nt = (int)gridDim.x, xcd = (int)blockIdx.x & 7;
  const int tile = xcd * (nt >> 3) + min(xcd, nt & 7) + ((int)blockIdx.x >> 3);
  int of;
  int64_t t0 = (int64_t)tile * 16;           // the first token, or the first of the group
  if constexpr (!ORDER) {
    of = t0 + m < T ? a.of[t0 + m] : -1;
    if (threadIdx.x < 16) s_tok[threadIdx.x] = threadIdx.x;
    lds_barrier();
  } else {
    t0 &= ~(int64_t)255;
    const int first = (tile & 15) * 16, n = (int)min(T - t0, (int64_t)256);
    if (threadIdx.x < 16) s_of[threadIdx.x] = -1;
    order_by_adapter<256>(a.of + t0, n, a.n_adapters, threadIdx.x, s_key, [&](int place, int t, int ad) {
      if ((place & ~15) == first) {
        s_tok[place & 15] = t;
        s_of[place & 15] = ad;
      }
    });
    lds_barrier();
    of = s_of[m];
  }
  const int part = (int)blockIdx.z % a.parts, r0 = (int)blockIdx.z / a.parts * 16 * RT;
  // 64-channel steps [k0, k1) of this wave
  const int nc = (K + 63) >> 6, cpp = (nc + a.parts - 1) / a.parts, p1 = min(nc, (part + 1) * cpp), cpw = (cpp + 3) >> 2;
  const int k0 = part * cpp + wave * cpw, k1 = min(p1, k0 + cpw);

  uint32_t todo = (uint32_t)__ballot((uint32_t)of < (uint32_t)a.n_adapters) & 0xFFFFu;
  for (int i = 0; todo != 0; ++i) {
    const int ad = __builtin_amdgcn_readlane(of, __builtin_ctz(todo));
    const uint32_t mine = (uint32_t)__ballot(of == ad) & 0xFFFFu;
    todo &= ~mine;
    if (i % (int)gridDim.y != (int)blockIdx.y) continue;
    // Every load has a valid address, so none needs a lane's branch: other adapters' rows of x
    // and ranks past the last only feed results that are not stored.  A step is 64 channels, a
    // whole 128-byte line of each row: lane group g takes 16 g .. 16 g + 15, in two loads on end
    // (with steps of half a line L1 had lost the line before its other half was read).
    const uint16_t* px = x + (t0 + s_tok[(mine >> m) & 1u ? m : __builtin_ctz(mine)]) * ldx;
    const char* pa = reinterpret_cast<const char*>(lora_a + ((int64_t)ad * a.rank + r0) * K);
    uint32_t ra[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) ra[q] = (uint32_t)(min(q * 16 + m, a.rank - 1 - r0) * K) * 2;
    f32x4 acc[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int UN = 3;                    // steps in flight (4: registers cost waves)
    for (int k = k0; k < k1; k += UN) {
      u32x4 xv[UN][2], av[UN][2][RT];
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        if (k + j >= k1) continue;
        // the last step's channels past K: any valid ones, cleared below
        const int c = min((k + j) * 64 + 16 * g, K - 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          xv[j][h] = *reinterpret_cast<const u32x4*>(px + c + 8 * h);
#pragma unroll
          for (int q = 0; q < RT; ++q) av[j][h][q] = *reinterpret_cast<const u32x4*>(pa + ra[q] + (uint32_t)(2 * c + 16 * h));
        }
      }
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        if (k + j >= k1) continue;
        if ((k + j) * 64 + 64 > K && g >= 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            xv[j][h] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < RT; ++q) av[j][h][q] = u32x4{0, 0, 0, 0};
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < RT; ++q)
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j][h]),
                                                             __builtin_bit_cast(bf16x8, av[j][h][q]), acc[q], 0, 0, 0);
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int q = 0; q < RT; ++q) red[wave - 1][q][lane] = acc[q];
    }
    lds_barrier();
    if (wave == 0) {
      const float s = adapter_scale != nullptr ? adapter_scale[ad] : 1.0f;
      float* up = u + part * a.part_stride;
#pragma unroll
      for (int q = 0; q < RT; ++q) {
#pragma unroll
        for (int w = 0; w < 3; ++w) acc[q] += red[w][q][lane];
        const int r = r0 + q * 16 + m;       // lane holds D[4 g + i][m]
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (((mine >> (4 * g + i)) & 1u) && r < a.rank) up[(t0 + s_tok[4 * g + i]) * a.rank + r] = s * acc[q][i];
      }
    }
    lds_barrier();                           // red is free for the next adapter
  }
}

// The projection of at most 32 tokens, a decode batch: the sweep of few_device.hpp over CW
// column tiles and SK splits of K, and in each wave its share of the adapters' rank (groups of
// 8, dealt to the splits), both reduced in split order.  Every lane forms its own outputs'
// adapter terms, so tokens with different adapters cost no more than tokens with one.
// Latency-bound: 2560 -> 9728 at one token 9.0 us for 12.8 MB (cbq_codebook_lut_gemm without
// adapters: 8.2), 9728 -> 2560 at 16 tokens with 16 adapters 12.8 us for 15 MB (10.7), where its
// 160 workgroups leave 96 CUs without one.
template <int BITS, int ABITS, bool BLK, int DEPTH>
__global__ void __launch_bounds__(1024)
few_adapter_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, GemmW w, int T, int N, int K,
                   int blocked, AdapterArgs a, float* __restrict__ out, int64_t ldo, int CW, int SK) {
  extern __shared__ f32x4 red[];
  float* s_u = reinterpret_cast<float*>(red + (size_t)(SK - 1) * CW * 4 * 64);   // [T][rank]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave / SK, sk = wave - cw * SK;
  const int m = lane & 15, g = lane >> 4;
  const int n0 = (blockIdx.x * CW + cw) * 16;
  const int nchunks = (K + 127) >> 7;
  const int cpw = (nchunks + SK - 1) / SK;
  const int c0 = sk * cpw, c1 = min(nchunks, c0 + cpw);
  FewWeights<BITS, 1> W;
  W.init(&w, false, 0, n0, N, K, blocked, lane);
  uint32_t ring[DEPTH][1][BITS];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) W.load(c0 + i, c1, ring[i]);
  // the tokens' middle vectors, their parts summed in order (rows without an adapter: whatever
  // the workspace held, never used)
  for (int i = threadIdx.x; i < T * a.rank / 4; i += blockDim.x) {
    f32x4 v = reinterpret_cast<const f32x4*>(a.u)[i];
#pragma unroll 4
    for (int p = 1; p < a.parts; ++p) v += reinterpret_cast<const f32x4*>(a.u + p * a.part_stride)[i];
    reinterpret_cast<f32x4*>(s_u)[i] = v;
  }
  f32x4 acc[1][2], low[2];
  uint32_t aoff[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    acc[0][s] = low[s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    aoff[s] = s * 16 + m < T ? (uint32_t)((s * 16 + m) * ((int64_t)K * ABITS / 8)) + (uint32_t)(g * 4 * ABITS) : kOffNone;
  }
  const __amdgpu_buffer_rsrc_t cres = make_rsrc(codes, 0x7FFFFFFFu);
  if (T > 16) few_sweep<BITS, ABITS, 1, BLK, 2, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
  else few_sweep<BITS, ABITS, 1, BLK, 1, DEPTH>(W, ring, cres, aoff, c0, c1, acc);
  lds_barrier();
  if (n0 < N) {
    const int n = n0 + m;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = s * 16 + 4 * g + i;
        const int ad = t < T ? a.of[t] : -1;
        if ((uint32_t)ad >= (uint32_t)a.n_adapters) continue;
        const uint16_t* b = a.lora_b + ((int64_t)ad * N + n) * a.rank;
        const float* u = s_u + t * a.rank;
        for (int r = sk * 8; r < a.rank; r += SK * 8) {
          const u32x4 bv = *reinterpret_cast<const u32x4*>(b + r);
          const f32x4 u0 = *reinterpret_cast<const f32x4*>(u + r), u1 = *reinterpret_cast<const f32x4*>(u + r + 4);
          float d = low[s][i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __builtin_bit_cast(float, bv[j] << 16), hi = __builtin_bit_cast(float, bv[j] & 0xFFFF0000u);
            d = __builtin_fmaf(j < 2 ? u0[2 * j] : u1[2 * j - 4], lo, d);
            d = __builtin_fmaf(j < 2 ? u0[2 * j + 1] : u1[2 * j - 3], hi, d);
          }
          low[s][i] = d;
        }
      }
    }
  }
  f32x4 sums[4] = {acc[0][0], low[0], acc[0][1], low[1]};
  few_reduce<4>(red, cw, sk, SK, lane, sums);
  if (sk != 0 || n0 >= N) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = s * 16 + 4 * g + i;
      if (t < T) out[t * ldo + n0 + m] = __builtin_fmaf(scales[t], sums[2 * s][i], sums[2 * s + 1][i]);
    }
  }
}

// K is split until about 2048 waves share the sweep, while each keeps at least eight chunks (the
// splits' sums and the adapters' ranks cost a pass over LDS each): half as many waves, or
// sixteen chunks at least, take 10.4 and 10.2 us instead of 9.0 for 2560 -> 9728 at one token,
// and 12.6 instead of 12.9 for 9728 -> 2560 at 16; twice as many waves the same, four chunks at
// least the same, or 7.3 instead of 7.9 for 2560 -> 2560 at 16.
template <int BITS, int ABITS, bool BLK>
static hipError_t launch_few_adapter(const GemmArgs& a, const AdapterArgs& ad, hipStream_t stream) {
  const int tiles = a.N / 16, nchunks = (a.K + 127) / 128;
  int SK = 1;
  while (SK < 16 && (int64_t)tiles * SK < 2048 && SK * 8 <= nchunks) SK *= 2;
  const int CW = SK < 4 ? 4 / SK : 1;
  const dim3 grid((unsigned)((tiles + CW - 1) / CW)), block((unsigned)(64 * CW * SK));
  const size_t lds = (size_t)(SK - 1) * CW * 4 * 64 * sizeof(f32x4) + (size_t)a.n_rows * ad.rank * sizeof(float);
  hipLaunchKernelGGL((few_adapter_kernel<BITS, ABITS, BLK, 2>), grid, block, lds, stream, a.codes, a.scales, a.w[0],
                     (int)a.n_rows, a.N, a.K, a.blocked, ad, static_cast<float*>(a.out), a.ldo, CW, SK);
  return hipGetLastError();
}

// Parts of K in the first launch, at most: enough workgroups for a decode batch or a short
// prefill (one part: 16 tokens of K = 9728 23.5 us instead of 5.5, 333 tokens of rank 64 15.8
// instead of 9.6; sixteen save the latter 2.2 us and cost the projection 2.7); fewer beyond,
// where the token tiles fill the GPU (2048 tokens of K = 2560 in one part 8.8 instead of 8.5).
static int adapter_max_parts(int64_t T) { return T <= kFewRows ? 16 : T <= 1024 ? 4 : T <= 8192 ? 2 : 1; }

size_t adapter_workspace_bytes(int64_t T, int rank) {
  return ((size_t)T * rank * adapter_max_parts(T) * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_adapter_gemm(const GemmArgs& a, AdapterArgs ad, const uint16_t* x, int64_t ldx,
                               const uint16_t* lora_a, const float* adapter_scale, float* u, hipStream_t stream) {
  ad.u = u;
  const int64_t T = a.n_rows;
  const int rt = (ad.rank + 15) / 16;
  const int RT = rt >= 4 ? 4 : rt >= 2 ? 2 : 1, zr = (rt + RT - 1) / RT;
  // a decode batch's tile may hold 16 adapters, one a workgroup; in larger batches, where
  // requests mostly span tiles, a tile's four workgroups take turns (16 tokens with 16 adapters:
  // 5.5 us with 16 workgroups, 10.1 with four, 23.8 with one; 333 tokens 9.5, 9.6, 15.2)
  const int most = (int)(T < 16 ? T : T <= 256 ? 16 : 4), ny = ad.n_adapters < most ? ad.n_adapters : most;
  const int64_t tiles = (T + 15) / 16;
  // parts of at least 4 steps of 64 channels (one a wave)
  ad.parts = 1;
  while (ad.parts * 2 <= adapter_max_parts(T) && ad.parts * 2 * 4 <= (a.K + 63) / 64 && tiles * ny * zr * ad.parts < 1024) ad.parts *= 2;
  ad.part_stride = T * ad.rank;
  const dim3 grid((unsigned)tiles, (unsigned)ny, (unsigned)(zr * ad.parts));
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, ad, x, ldx, lora_a, adapter_scale, T, a.K, u);
  };
  const bool order = T > kFewRows;
  if (RT == 4) order ? launch(adapter_shrink_kernel<4, true>) : launch(adapter_shrink_kernel<4, false>);
  else if (RT == 2) order ? launch(adapter_shrink_kernel<2, true>) : launch(adapter_shrink_kernel<2, false>);
  else order ? launch(adapter_shrink_kernel<1, true>) : launch(adapter_shrink_kernel<1, false>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (T > kFewRows) return launch_mfma_prefill_adapter(a, ad, stream);
  if (a.act_bits == 4) {
    if (a.bits == 4) return launch_few_adapter<4, 4, false>(a, ad, stream);
    if (a.bits == 2) return launch_few_adapter<2, 4, false>(a, ad, stream);
    return a.blocked ? launch_few_adapter<3, 4, true>(a, ad, stream) : launch_few_adapter<3, 4, false>(a, ad, stream);
  }
  if (a.bits == 4) return launch_few_adapter<4, 8, false>(a, ad, stream);
  if (a.bits == 2) return launch_few_adapter<2, 8, false>(a, ad, stream);
  return a.blocked ? launch_few_adapter<3, 8, true>(a, ad, stream) : launch_few_adapter<3, 8, false>(a, ad, stream);
}

}  // namespace cbq
