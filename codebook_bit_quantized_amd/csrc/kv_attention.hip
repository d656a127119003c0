// Attention of a step's queries over the 4-bit key/value cache.
//
// The mathematics.  With a_j = scale <q, k_j> the result is sum_j exp(a_j) v_j / sum_j exp(a_j), in one
// pass over the keys with a running maximum.  A key is its scale ks_j times E2M1 codes, so
// a_j = ks_j <q', codes_j> with q' the rotated query times scale in fp16 (11 bits, where q came in 8: its rounding
// is far below that of q itself, and the range is seen to in convert_queries); codes are exact in fp16 and the
// products' sums are fp32.  A value's scale vs_j joins the weight:
//     b_j = a_j log2 e + log2 vs_j,   w_j = 2^(b_j - M),   M 2^7 below the running maximum of b,
//     result = sum_j w_j codes_j / sum_j (w_j / vs_j),
// so w_j in fp16 is always relative to its row's largest contribution, whatever the scales' range: 11 bits down to 2^-21 of
// it, fewer below, none below 2^-32.  The sum of weights takes them before that rounding, down to 2^-133 of the largest.
//
// The tiles.  A wave takes 64 keys at a time.  Scores are computed transposed, keys times queries
// (16x16x32 MFMA: 16 keys, 16 query rows), so that lane (row r = lane % 16, g = lane / 16) ends
// with the scores of row r and keys 4g .. 4g+3 of each 16: statistics are per lane and two
// swaps, and the weights are, where they lie, the second operand of values (channels) times weights. That
// product wants 8 keys of one channel in a lane: the values go to LDS as they are, and
// ds_read_b64_tr_b4 hands each lane 16 keys' codes of its channel.  Codes become fp16 by
// v_cvt_scalef32_pk_f16_fp4, two at a time.
//
// What bounds it.  With few query rows (decode, drafted tokens) the cache is read once and the bytes count: the
// kernel reads at 5.9 TB/s once under way, on top of 3.5 us until the first keys are there (length, schedule, page, key: four
// dependent loads), some 3 us in which the last workgroups end, and 4 us for the launch that joins.  64 ragged
// sequences of up to 32768 tokens: 48 us, 187 MB; one of 131072: 38 us, 143 MB.  Beyond that the vector instructions
// count: 64 keys by 32 rows take 387 of them (weights, conversions of codes) next to 64 matrix instructions, which are busy
// 29 to 41 % of the time.  The last 512 tokens of 16384: 159 us, 850 TFLOP/s; four prompts: 287 us, 824 TFLOP/s.
#include <algorithm>

#include "kv_device.hpp"

namespace cbq {
namespace {

constexpr int kTile = 64;          // keys a wave takes at a time
// Waves that share a row block of 16 rows.  Four, two workgroups on a compute unit, leave more parts to join: one sequence of
// 131072 tokens 38.8 against 38.1 us, 16 of 4000 36.1 against 34.3; 32 windows of 4096 23.5 against 25.5.
constexpr int kWaves = 8;
// Workgroups of a split call, as many as the chip holds at once (with the registers of a wave at their most): 256 of eight
// waves, 512 of four.
constexpr int max_groups(int rows) { return rows == 128 ? 512 : 256; }

// A sequence's part of the step, all values uniform over the workgroup.
struct Seq {
  int t0, rows;                    // its first token; tokens * G (-1: see kv_seq)
  int pos0;                        // position of the first token
  int len;                         // positions that can hold anything
};

struct Range { int lo, hi; };      // [lo, hi)

// What the workgroups of a split call leave for the join: a row block that starts in group w and goes on in the next `more`:
// its sequence's first token, its head, its first row and its rows.
struct alignas(16) Desc { int t0, kvh, r0, rows, more; };

struct SplitArgs {
  int groups;                      // workgroups
  int split;                       // 1: units are key tiles; 0: whole row blocks
  int shift;                       // split: a unit is 2^shift key tiles, so that all units fit 31 bits
  int start_cost;                  // split: units that the start of a row block counts for
  int min_units;                   // units a workgroup takes at least
  int G;                           // query heads a key/value head
  uint32_t g_mul, g_shift;         // r / G = r * g_mul >> g_shift for r < 2^31
  int join_rows;                   // rows of a row block that any has
  float c_q, c_v;                  // 1/sqrt(D) where queries are rotated / values rotated back, else 1
  Desc* desc;                      // [groups]
  float2* ml;                      // [2 * groups][ROWS]: M and sum of each part's rows
  float* o;                        // [2 * groups][ROWS][D]
};

__device__ __forceinline__ int div_g(const SplitArgs& sp, int r) {
  return (int)(((uint64_t)(uint32_t)r * sp.g_mul) >> sp.g_shift);
}

__device__ __forceinline__ Seq kv_seq(const KvArgs& a, int b, int G) {
  const int T = (int)a.T, cap = a.max_pages << a.logp, len = a.lens[b];
  int o0, o1;
  if (a.offsets) { o0 = a.offsets[b]; o1 = a.offsets[b + 1]; }
  else { o0 = b * a.per_seq; o1 = o0 + a.per_seq; }
  const int s = max(o0, 0), e = min(o1, T);
  Seq q;
  q.t0 = s;
  q.rows = e > s ? (e - s) * G : o1 < o0 ? -1 : 0;    // T * n_q < 2^31; -1: offsets that do not ascend
  const int64_t pos0 = (int64_t)len - o1 + s;         // pos0 + i < len for its tokens i: no sum below leaves 32 bits
  q.pos0 = (int)max(pos0, (int64_t)-0x80000000LL);
  q.len = min(max(len, 0), cap);
  return q;
}

// Positions that token i of the sequence attends.
__device__ __forceinline__ Range kv_range(const Seq& q, int i, int causal, int window) {
  const int pos = q.pos0 + i;
  Range r{0, q.len};
  if (causal) {
    r.hi = min(max(pos + 1, 0), q.len);
    if (window && pos >= window) r.lo = pos - window + 1;
  }
  return r;
}

// Key tiles [lo, hi) of query rows r0 .. r1 (at least one tile: a row that attends nothing is written too).
__device__ __forceinline__ Range kv_tiles(const KvAttnArgs& g, const SplitArgs& sp, const Seq& q, int r0, int r1) {
  const int lo = kv_range(q, div_g(sp, r0), g.causal, g.window).lo / kTile;
  const int hi = (int)(((uint32_t)kv_range(q, div_g(sp, r1), g.causal, g.window).hi + kTile - 1) / kTile);
  return Range{lo, max(hi, lo + 1)};
}

// ceil(x / y) for 0 <= x, 0 < y, quotients up to 2^16, by a reciprocal: what its rounding may miss is one step.
__device__ __forceinline__ int div_up(int x, int y) {
  const int q = (int)((float)x * __builtin_amdgcn_rcpf((float)y));
  return (int64_t)q * y < x ? q + 1 : q;
}

// How units are counted: `start` of them for a row block's start, and each row block rounded up to a multiple of `whole`.
struct Count { int start, whole; };

__device__ __forceinline__ int units_of(const SplitArgs& sp, const Count& c, const Range& t) {
  const int n = ((t.hi - t.lo - 1) >> sp.shift) + 1 + c.start;
  return c.whole > 1 ? div_up(n, c.whole) * c.whole : n;
}

// Units of row block rb of a sequence.
template <int ROWS>
__device__ __forceinline__ int rb_units(const KvAttnArgs& g, const SplitArgs& sp, const Count& c, const Seq& q, int rb) {
  if (rb >= (q.rows + ROWS - 1) / ROWS) return 0;
  if (!sp.split) return 1;
  return units_of(sp, c, kv_tiles(g, sp, q, rb * ROWS, min((rb + 1) * ROWS, q.rows) - 1));
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // lane 15 of a row into the next row
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // lane 31 into the upper half
  return x;
}

// The row blocks, or parts of them, that a workgroup works through.  All sequences' units in a row (a
// sequence's in the order head, row block, key tile; whole row blocks in the order row block, head) are dealt out evenly,
// `per` to a workgroup; each wave counts them for itself, from the lengths, so the lengths stay on the device and the
// work is even whatever they are.  A lane counts its sequences' row blocks where they are few, else
// the wave does it together.
template <int ROWS>
struct Walk {
  Seq q;
  int b, kvh, r0, off, left, per;  // r0: the next row block, off: units of it that are not this workgroup's
  // the current part: units [u0, u1) of `units` of row block `row0` of head `h` of sequence `seq`
  int seq, h, row0, u0, u1, units;
  Range tiles;                     // its key tiles
  Count count;
  Seq lane_q;                      // up to 64 sequences: the lane's own, so that no start waits for a length

  // whether and for how many groups the current part goes on: only the last part of a group does
  __device__ __forceinline__ int following(const SplitArgs& sp) const {
    const uint32_t n = ((uint32_t)(units - u1) + per - 1) / (uint32_t)per;
    return (int)min(n, (uint32_t)sp.groups - 1 - blockIdx.x);
  }

  __device__ __forceinline__ Seq get(const KvArgs& a, const SplitArgs& sp, int i) const {
    return a.B > 64 ? kv_seq(a, i, sp.G) : lane_seq(lane_q, i);
  }
  static __device__ __forceinline__ Seq lane_seq(const Seq& s, int i) {
    return Seq{__builtin_amdgcn_readlane(s.t0, i), __builtin_amdgcn_readlane(s.rows, i),
               __builtin_amdgcn_readlane(s.pos0, i), __builtin_amdgcn_readlane(s.len, i)};
  }

  // Units of one key/value head, by the whole wave; with at: the row block that holds unit *at, and what of it comes before.
  __device__ __forceinline__ int head_units(const KvAttnArgs& g, const SplitArgs& sp, const Seq& s, int* at, int* row) const {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int rb = 0; rb * ROWS < s.rows; rb += 64) {
      const int mine = rb_units<ROWS>(g, sp, count, s, rb + lane), inc = wave_scan(mine);
      const int all = __builtin_amdgcn_readlane(inc, 63);
      if (at && *at < n + all) {
        const int l = (int)__builtin_ctzll(__ballot(*at < n + inc));
        *row = (rb + l) * ROWS;
        *at -= n + __builtin_amdgcn_readlane(inc - mine, l);
        return n;
      }
      n += all;
    }
    return n;
  }

  __device__ __forceinline__ void start(const KvAttnArgs& g, const SplitArgs& sp) {
    const KvArgs& a = g.kv;
    const int lane = threadIdx.x & 63;
    const int each = (a.B + 63) >> 6;                 // sequences a lane counts
    constexpr int kFew = 4;                           // row blocks that a lane counts by itself
    int mine, head = 0, inc, total, blocks;
    bool ascending = true;
    count = Count{sp.start_cost, 1};
    per = 0;
    for (;;) {
      mine = blocks = 0;
      for (int k = 0; k < each; ++k) {
        const int i = lane * each + k;
        if (each > 1 || per == 0) {
          lane_q = Seq{0, 0, 0, 0};
          if (i < a.B) lane_q = kv_seq(a, i, sp.G);
        }
        ascending = ascending && lane_q.rows >= 0;
        const int n = (int)((uint32_t)(lane_q.rows + ROWS - 1) / ROWS);
        head = n;
        if (sp.split) {
          head = 0;
          if (n <= kFew)
            for (int rb = 0; rb < n; ++rb) head += rb_units<ROWS>(g, sp, count, lane_q, rb);
          for (uint64_t many = __ballot(n > kFew); many; many &= many - 1) {
            const int l = (int)__builtin_ctzll(many);
            const int u = head_units(g, sp, lane_seq(lane_q, l), nullptr, nullptr);
            if (lane == l) head = u;
          }
        }
        mine += head * a.n_kv;
        blocks += n * a.n_kv;
      }
      inc = wave_scan(mine);
      total = __builtin_amdgcn_readlane(inc, 63);
      if (per) break;
      const int n = ROWS == 16 ? __builtin_amdgcn_readlane(wave_scan(blocks), 63) : 0;
      per = max((int)(((uint32_t)total + sp.groups - 1) / (uint32_t)sp.groups), sp.min_units);
      // Where it takes no longer, a workgroup takes units of one row block only (the sum of the rounded-up quotients is at
      // most groups): a second row block in it would cost 1 to 3 us (4 heads, one sequence of 1200: 12.2 against 14.1 us, of
      // 4096, where the even split happens to fit, 13.6 against 12.7; 8 heads, 8 of 3000: 16.2 against 18.5).
      if (ROWS > 16 || !sp.split || n >= sp.groups) break;
      const int rest = total - n * sp.start_cost, free = sp.groups - n;
      const int own = max((int)(((uint32_t)rest + free - 1) / (uint32_t)free), sp.min_units);
      if (own > per) break;
      per = own;
      count = Count{0, own};
    }
    // unsplit calls start with the last units: a sequence's last rows attend the most keys
    const int64_t at = sp.split ? (int64_t)blockIdx.x : (int64_t)sp.groups - 1 - blockIdx.x;
    left = 0;
    b = a.B;
    // sequences whose tokens overlap could have more row blocks than the host has counted: nothing is done
    if (__any(!ascending) || at * per >= total) return;
    const int first = (int)at * per;
    left = min(total - first, per);
    const uint64_t past = __ballot(first < inc);
    const int f = past ? (int)__builtin_ctzll(past) : 63;
    b = f * each;
    off = first - (__builtin_amdgcn_readlane(inc, f) - __builtin_amdgcn_readlane(mine, f));
    kvh = 0;
    r0 = 0;
    for (; b < a.B; ++b) {                            // at most `each` times
      q = get(a, sp, b);
      const int hu = each == 1 ? __builtin_amdgcn_readlane(head, f) : head_units(g, sp, q, nullptr, nullptr);
      if (off < hu * a.n_kv) {
        if (!sp.split) {
          r0 = off / a.n_kv * ROWS;
          kvh = off % a.n_kv;
          off = 0;
        } else {
          kvh = off / hu;
          off -= kvh * hu;
          head_units(g, sp, q, &off, &r0);
        }
        return;
      }
      off -= hu * a.n_kv;
    }
    left = 0;
  }

  __device__ __forceinline__ bool next(const KvAttnArgs& g, const SplitArgs& sp) {
    if (left <= 0) return false;
    if (!sp.split) {
      while (r0 >= q.rows) {
        if (++b >= g.kv.B) return false;
        q = get(g.kv, sp, b);
        r0 = 0;
      }
      tiles = kv_tiles(g, sp, q, r0, min(r0 + ROWS, q.rows) - 1);
      seq = b;
      h = kvh;
      row0 = r0;
      u0 = 0;
      u1 = units = 1;
      --left;
      if (++kvh == g.kv.n_kv) { kvh = 0; r0 += ROWS; }
      return true;
    }
    if (r0 >= q.rows) {
      r0 = 0;
      if (++kvh >= g.kv.n_kv) {
        kvh = 0;
        do {
          if (++b >= g.kv.B) return false;
          q = get(g.kv, sp, b);
        } while (q.rows == 0);
      }
    }
    tiles = kv_tiles(g, sp, q, r0, min(r0 + ROWS, q.rows) - 1);
    units = units_of(sp, count, tiles);
    row0 = r0;
    r0 += ROWS;
    seq = b;
    h = kvh;
    u0 = off;
    u1 = min(units, off + left);
    left -= u1 - u0;
    off = 0;
    // the units that count for the start hold no keys
    const int lo = tiles.lo + (max(u0 - count.start, 0) << sp.shift);
    tiles.hi = min(tiles.hi, tiles.lo + (max(u1 - count.start, 0) << sp.shift));
    tiles.lo = lo;
    return true;
  }
};

template <int D>
struct Lds {
  static constexpr int P = D + 4;                     // padded row: 16 rows start in 16 different bank groups
  union {
    struct {
      alignas(16) uint8_t v[kWaves][kTile * D / 2];                  // values' codes, 16-byte (8-byte) quarters of a row swizzled
      alignas(16) float ks[kWaves][kTile], lv[kWaves][kTile], iv[kWaves][kTile];
    } t;
    alignas(16) float o[kWaves][16 * P];
  };
  float m[kWaves][16], l[kWaves][16];
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The bits of a value, by value: a bit cast of a vector's element reads the vector's first one.
__device__ __forceinline__ uint32_t float_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.0f : m; }

// x of the lanes 16 (32) apart: a of the even row (lower half), b of the odd row (upper half), in
// both lanes.  The swap's second operand is hidden from the compiler, which takes the two
// results of a swap of equal operands for one.
template <bool SWAP32>
__device__ __forceinline__ void swap_pair(float x, float& a, float& b) {
  uint32_t u = __builtin_bit_cast(uint32_t, x), v = u;
  asm("" : "+v"(v));
  u32x2 r;
  if constexpr (SWAP32) { const auto t = __builtin_amdgcn_permlane32_swap(u, v, false, false); r = u32x2{t[0], t[1]}; }
  else { const auto t = __builtin_amdgcn_permlane16_swap(u, v, false, false); r = u32x2{t[0], t[1]}; }
  a = __builtin_bit_cast(float, (uint32_t)r[0]);
  b = __builtin_bit_cast(float, (uint32_t)r[1]);
}

// over the four lanes that hold a row
__device__ __forceinline__ float row_max(float x) {
  float a, b;
  swap_pair<false>(x, a, b);
  swap_pair<true>(fmaxf(a, b), a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t x) {
  float a, b;
  swap_pair<false>(__builtin_bit_cast(float, x), a, b);
  x = max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
  swap_pair<true>(__builtin_bit_cast(float, x), a, b);
  return max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
__device__ __forceinline__ float row_add(float x) {
  float a, b;
  swap_pair<false>(x, a, b);
  swap_pair<true>(a + b, a, b);
  return a + b;
}

// 16 query rows as the MFMA's second operand: lane (row, g) holds channels g*D/4 ... of its row.
template <int D>
struct Queries { u32x4 x[D / 32]; };

template <int D>
__device__ __forceinline__ Queries<D> fetch_queries(const KvAttnArgs& g, const SplitArgs& sp, const Seq& q, int kvh, int r, bool row) {
  const int lane = threadIdx.x & 63, i = div_g(sp, r), h = r - i * sp.G;
  const uint16_t* src = g.q + (int64_t)(q.t0 + i) * g.ldq + (kvh * sp.G + h) * D + (lane >> 4) * (D / 4);
  Queries<D> f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) f.x[k] = row ? *reinterpret_cast<const u32x4*>(src + 8 * k) : u32x4{0, 0, 0, 0};
  return f;
}

// Rotated if asked, times c_scale in fp16.  A row whose largest value is then within 2^-4 ... 2^15 stays as it is (what
// lies below 2^-14 is off by at most 2^-25 there, 2^-21 of the largest); another is divided by a power of two near that
// value instead of times c_scale, and *rs, which its scores are multiplied by, makes up for both.
// The rotation is a product with the +-1 matrix on the matrix cores (bf16 inputs exact, fp32 sums): its row m of tile c
// is output channel D/4 (m / 4) + 4c + m % 4, so that lane (row, g) gets the channels it needs.  An entry's sign is
// the parity of the bits that input and output channel share; with input channel D/4 g + 8k + j
// it falls into parities of j with (m % 4, c % 2), of k with c / 2, and of g with m / 4.
template <int D>
__device__ __forceinline__ void convert_queries(const Queries<D>& f, bool rotate, float c_scale, f16x8* out, float* rs) {
  const int lane = threadIdx.x & 63;
  f32x4 x[D / 16];
  if (rotate) {
    const uint32_t m4 = lane & 3, gm = (lane >> 4) & ((lane >> 2) & 3);
    const uint32_t all = (gm ^ (gm >> 1)) & 1 ? 0x80008000u : 0u;
    uint32_t h[4];                                    // c even, k without shared bits: dword d holds j = 2d, 2d + 1
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t p = (m4 >> 1) & d & 1;           // j's bit 1 is d's bit 0
      h[d] = 0x3F803F80u ^ all ^ (p ? 0x80008000u : 0u) ^ (m4 & 1 ? 0x80000000u : 0u);
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      x[c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const int kc = k & (c >> 1);
        const uint32_t lo = (kc ^ (kc >> 1)) & 1 ? 0x80008000u : 0u, hi = c & 1 ? lo ^ 0x80008000u : lo;
        const u32x4 hm = {h[0] ^ lo, h[1] ^ lo, h[2] ^ hi, h[3] ^ hi};
        x[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hm), __builtin_bit_cast(bf16x8, f.x[k]), x[c], 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const uint32_t a = f.x[c / 2][2 * (c & 1)], b = f.x[c / 2][2 * (c & 1) + 1];
      x[c] = f32x4{__builtin_bit_cast(float, a << 16), __builtin_bit_cast(float, a & 0xFFFF0000u),
                   __builtin_bit_cast(float, b << 16), __builtin_bit_cast(float, b & 0xFFFF0000u)};
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, float_bits(x[c][j]) & 0x7FFFFFFFu);
  m = row_max_u32(m);
  const float top = __builtin_bit_cast(float, m) * fabsf(c_scale);
  const bool unit = (top >= 0x1p-4f && top < 0x1p15f) || m == 0;
  const uint32_t e = min(m >> 23, 253u);              // 2^(e-127) <= largest value, or smaller
  const float mul = unit ? c_scale : __builtin_bit_cast(float, (254u - e) << 23);
  const float p = m >= 0x7F800000u ? NAN : e ? __builtin_bit_cast(float, e << 23) : 0x1p-127f;
  *rs = unit ? 1.0f : p * c_scale;
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) out[c / 2][4 * (c & 1) + j] = (_Float16)(x[c][j] * mul);
}

// 8 codes -> 8 fp16
__device__ __forceinline__ f16x8 e2m1_f16x8(uint32_t x) {
  const f16x2 a = e2m1_pair<0>(x), b = e2m1_pair<1>(x), c = e2m1_pair<2>(x), d = e2m1_pair<3>(x);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Row of D values held 8 to a lane, normalised and rotated back, to bf16.
template <int D>
__device__ __forceinline__ void finish_row(float* v, float l, bool rotate, float c_v, int lane, uint16_t* dst) {
  if (rotate) kv_transform<D>(v, lane);
  const float f = l != 0.0f ? c_v / l : 0.0f;
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = (uint32_t)f32_to_bf16_rne(v[2 * i] * f) | ((uint32_t)f32_to_bf16_rne(v[2 * i + 1] * f) << 16);
  *reinterpret_cast<u32x4*>(dst) = out;
}

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

// A key's scales as soft_weights takes them.
__device__ __forceinline__ void stage_key(float ks, bool some, float* at) { *at = some ? ks : 0.0f; }
__device__ __forceinline__ void stage_value(float vs, bool some, float* lv, float* iv) {
  const float v = vs < 0x1p-64f ? 0x1p-64f : vs;
  *lv = some ? __builtin_amdgcn_logf(v) : -INFINITY;
  *iv = some ? __builtin_amdgcn_rcpf(v) : 0.0f;
}

// Scores of 64 keys to weights: sc[n][i][j] is row lane % 16 of row tile n and key 16i + 4 (lane / 16) + j of the tile at
// position t0.  Keys that no row attends come with ks = 0, lv = -inf and iv = 0 (stage_key, stage_value), which masks them at no
// cost here, but for scores that are NaN; same: all rows attend the same of the others, at least one of them.  The running
// maximum moves only when a score passes it by 2^kSlack: most tiles then need neither an exchange between lanes nor a
// rescaling.  M lies kTop below the maximum, so that weights use fp16's range to 2^15: with M the maximum itself they were
// lost from 2^-25 of the largest on, and 2^20 keys that far below another lost 2 % of the row's sum.
constexpr float kSlack = 8.0f, kTop = 7.0f;

template <int D, int NB>
__device__ __forceinline__ void soft_weights(const float* ks, const float* lv, const float* iv, int t0, bool same,
                                             bool unit, const float* rs, const int* lo, const int* hi, f32x4 (*sc)[4], float* M, float* l,
                                             f32x4 (*o)[D / 16], f16x8 (*w)[2]) {
  const int lane = threadIdx.x & 63, key = 4 * (lane >> 4);
  // A query that is not finite has an rs that is not 1, and scores that are NaN: they would survive lv = -inf, and a row may
  // attend none of the tile's keys that are held.  Called where its code costs the other calls least: with one row tile
  // before the masks (windows of 4096 19.8 us behind the scaling or at the masks, 19.1 in it), with two at the masks of rows
  // that attend different keys (four prompts 286 us; in the scaling 290, for every key's mask 293).  by: what the scores are
  // multiplied by besides, or null.
  auto clear_unheld = [&](const float* by) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool held = lv[16 * i + key + j] != -INFINITY;
#pragma unroll
        for (int n = 0; n < NB; ++n) sc[n][i][j] = held ? sc[n][i][j] * (by ? by[n] : 1.0f) : by ? 0.0f : -INFINITY;
      }
  };
  if (!unit) {
    if constexpr (NB == 1) {
      clear_unheld(rs);
    } else {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] *= rs[n];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 k = *reinterpret_cast<const f32x4*>(ks + 16 * i + key), v = *reinterpret_cast<const f32x4*>(lv + 16 * i + key);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[n][i][j] = __builtin_fmaf(sc[n][i][j], k[j], v[j]);
  }
  if (!same) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int at = t0 + key - lo[n];
      const uint32_t len = (uint32_t)max(hi[n] - lo[n], 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[n][i][j] = (uint32_t)(at + 16 * i + j) < len ? sc[n][i][j] : -INFINITY;
      }
    }
    if (NB > 1 && !unit) clear_unheld(nullptr);
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = fmaxf(mx, sc[n][i][j]);
    // by differences, as the weights' arguments: M + 15 is rounded by more where scores pass 2^24, and a weight past 2^16 is
    // infinite in fp16
    if (__any(mx - M[n] > kTop + kSlack)) {
      const float rm = row_max(mx), m = rm - M[n] > kTop + kSlack ? rm - kTop : M[n];   // a row moves for its own scores alone
      const float keep = __builtin_amdgcn_exp2f(M[n] - safe_max(m));
      l[n] *= keep;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[n][c] *= keep;
      M[n] = m;
    }
    const float ref = safe_max(M[n]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = __builtin_amdgcn_exp2f(sc[n][i][j] - ref);
        sc[n][i][j] = p;
        w[n][i >> 1][4 * (i & 1) + j] = (_Float16)p;
      }
  }
  if (same) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(iv + 16 * i + key);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) l[n] = __builtin_fmaf(sc[n][i][j], v[j], l[n]);
    }
  } else {                                            // 1 / vs of a key that the row does not attend may be NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(iv + 16 * i + key);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) l[n] = sc[n][i][j] != 0.0f ? __builtin_fmaf(sc[n][i][j], v[j], l[n]) : l[n];
    }
  }
}

// 16 keys' codes of channel 16c + lane % 16: keys 16i + 4 (lane / 16) + j, nibble 4i + j.  v: the tile's codes by key,
// quarters of a row swizzled by the key's i.
template <int D>
__device__ __forceinline__ i32x2 value_codes(const uint8_t* v, int c) {
  const int lane = threadIdx.x & 63, r = lane & 15, key = 16 * (r >> 2) + 4 * (lane >> 4) + (r & 3);
  const int chunk = c * 8 / (D / 8), in = c * 8 % (D / 8);
  return __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2*)(v + key * (D / 2) + (chunk ^ (r >> 2)) * (D / 8) + in));
}

template <int D> struct Chunk;                        // a quarter of a row of codes
template <> struct Chunk<128> { typedef u32x4 T; };
template <> struct Chunk<64> { typedef u32x2 T; };

template <int D>
struct TileRegs {                                     // one tile's codes and scales on their way
  typename Chunk<D>::T k[4], v[4];
  float ks, vs;
  uint32_t held;                                      // bit i: keys 16i .. 16i+15 lie in a page
};

// Pages of a wave's tiles: lane 4k + i holds the page of keys 16i ... of the k-th tile to come (every WV-th from `tile` on).
template <int WV>
__device__ __forceinline__ int tile_pages(const KvArgs& a, int b, int64_t tile) {
  const int lane = threadIdx.x & 63;
  return kv_page(a, b, (tile + (int64_t)(lane >> 2) * WV) * kTile + (lane & 3) * 16);
}

template <int D>
__device__ __forceinline__ void load_tile(const KvArgs& a, int kvh, int tile, int pages, int at, TileRegs<D>& r) {
  typedef typename Chunk<D>::T C;
  const int lane = threadIdx.x & 63;
  const uint32_t mask = (1u << a.logp) - 1;
  uint32_t held = 0;
  int pg[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pg[i] = __builtin_amdgcn_readlane(pages, 4 * at + i);
    held |= pg[i] >= 0 ? 1u << i : 0;
    pg[i] = pg[i] >= 0 ? pg[i] : 0;                   // keys in no page: any page is read, and masked
    const int64_t row = (((int64_t)(pg[i] * a.n_kv + kvh) << a.logp) + ((tile * kTile + 16 * i) & mask)) * (D / 2);
    r.k[i] = *reinterpret_cast<const C*>(a.codes[0] + row + (lane & 15) * (D / 2) + (lane >> 4) * (D / 8));
    r.v[i] = *reinterpret_cast<const C*>(a.codes[1] + row + (lane >> 2) * (D / 2) + (lane & 3) * (D / 8));
  }
  const int g = lane >> 4;
  const int p = g & 2 ? (g & 1 ? pg[3] : pg[2]) : (g & 1 ? pg[1] : pg[0]);
  const int64_t row = ((int64_t)(p * a.n_kv + kvh) << a.logp) + ((tile * kTile + lane) & mask);
  r.ks = a.scales[0][row];
  r.vs = a.scales[1][row];
  r.held = held;
}

template <int D>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_attention_kernel(KvAttnArgs g, SplitArgs sp) {
  constexpr int ROWS = 16, WV = kWaves, P = Lds<D>::P, L = D / 8;
  __shared__ Lds<D> s;
  const KvArgs& a = g.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid == 0 && sp.split) sp.desc[blockIdx.x].more = 0;
  Walk<ROWS> u;
  u.start(g, sp);
  const float c_scale = g.scale * sp.c_q * 1.44269504088896341f;

  Seq q;                                              // the part in hand
  int row0 = 0, n_rows = 0, kvh = 0;
  bool have = false, starts = false, ends = false;
  float M[1], l[1];
  f32x4 o[1][D / 16];
  for (;;) {
    // ---- the next part: its first keys are on their way before the last part's sums are joined
    const bool more = u.next(g, sp);
    int tile = u.tiles.lo + wave, at = 0, pages = 0;
    const bool mine = more && tile < u.tiles.hi;
    TileRegs<D> nx;
    if (mine) pages = tile_pages<WV>(a, u.seq, tile);
    if (have) {
      __syncthreads();
      const int row = lane & 15;
      const float lsum = row_add(l[0]);
      if (lane < 16) {
        s.m[wave][row] = M[0];
        s.l[wave][row] = lsum;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        *reinterpret_cast<f32x4*>(&s.o[wave][row * P + 16 * c + 4 * (lane >> 4)]) = o[0][c];
      __syncthreads();
    }
    Queries<D> fq;
    if (more) {
      const int r = u.row0 + (lane & 15);
      fq = fetch_queries<D>(g, sp, u.q, u.h, min(r, u.q.rows - 1), r < u.q.rows);
    }
    if (mine) load_tile<D>(a, u.h, tile, pages, 0, nx);
    if (have) {
      const int64_t part = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
      const int sub = tid % L;
      const int row = tid / L;
      if (row < n_rows) {                             // whole groups of L lanes
        float m = -INFINITY, sum = 0, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WV; ++w) m = fmaxf(m, s.m[w][row]);
        const float ref = safe_max(m);
#pragma unroll
        for (int w = 0; w < WV; ++w) {
          const float f = __builtin_amdgcn_exp2f(s.m[w][row] - ref);
          sum = __builtin_fmaf(s.l[w][row], f, sum);
          const f32x4 x0 = *reinterpret_cast<const f32x4*>(&s.o[w][row * P + 8 * sub]);
          const f32x4 x1 = *reinterpret_cast<const f32x4*>(&s.o[w][row * P + 8 * sub + 4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = __builtin_fmaf(x0[j], f, v[j]);
            v[4 + j] = __builtin_fmaf(x1[j], f, v[4 + j]);
          }
        }
        if (starts && ends) {
          const int r = row0 + row, i = div_g(sp, r), h = r - i * sp.G;
          finish_row<D>(v, sum, a.rotate & 2, sp.c_v, sub, g.out + (int64_t)(q.t0 + i) * g.ldo + (kvh * sp.G + h) * D + 8 * sub);
        } else {
          float* dst = sp.o + (part * ROWS + row) * D + 8 * sub;
          *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
          if (sub == 0) sp.ml[part * ROWS + row] = float2{m, sum};
        }
      }
    }
    if (!more) return;
    q = u.q;
    row0 = u.row0;
    kvh = u.h;
    n_rows = min(ROWS, q.rows - row0);
    starts = u.u0 == 0;
    ends = u.u1 == u.units;
    have = true;
    if (starts && !ends && tid == 0)
      sp.desc[blockIdx.x] = Desc{q.t0, kvh, row0, n_rows, u.following(sp)};

    // ---- the queries, and what each row attends
    f16x8 qf[D / 32];
    float rs[1];
    convert_queries<D>(fq, a.rotate & 1, c_scale, qf, rs);
    const bool row = (lane & 15) < n_rows;
    const Range attended = kv_range(q, div_g(sp, row ? row0 + (lane & 15) : row0), g.causal, g.window);
    const int lo[1] = {attended.lo}, hi[1] = {row ? attended.hi : 0};
    M[0] = -INFINITY;
    l[0] = 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[0][c] = f32x4{0, 0, 0, 0};
    // positions that some row attends, and that every row does
    const Range first = kv_range(q, div_g(sp, row0), g.causal, g.window);
    const Range last = kv_range(q, div_g(sp, row0 + n_rows - 1), g.causal, g.window);
    const Range any{first.lo, last.hi}, every{last.lo, first.hi};
    const int t_hi = u.tiles.hi;
    const bool unit = !__any(rs[0] != 1.0f);
    __syncthreads();                                  // the last part's sums have been read

    // ---- the wave's tiles
    for (; tile < t_hi; tile += WV) {
      TileRegs<D> cu = nx;
      uint8_t* vl = s.t.v[wave];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<typename Chunk<D>::T*>(vl + (16 * i + (lane >> 2)) * (D / 2) + ((lane & 3) ^ i) * (D / 8)) = cu.v[i];
      const int t0 = tile * kTile;
      const bool some = ((cu.held >> (lane >> 4)) & 1) && t0 + lane >= any.lo && t0 + lane < any.hi;
      stage_key(cu.ks, some, &s.t.ks[wave][lane]);
      stage_value(cu.vs, some, &s.t.lv[wave][lane], &s.t.iv[wave][lane]);
      if (tile + WV < t_hi) {
        if (++at == 16) { pages = tile_pages<WV>(a, u.seq, tile + WV); at = 0; }
        load_tile<D>(a, kvh, tile + WV, pages, at, nx);
      }
      if (!__ballot(some)) continue;                  // (a row that attends nothing gets zeros, whatever its query)
      // scores of 64 keys
      f32x4 sc[1][4];
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 kf = e2m1_f16x8(cu.k[i][k]);
          sc[0][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[k], k ? sc[0][i] : f32x4{0, 0, 0, 0}, 0, 0, 0);
        }
      __builtin_amdgcn_wave_barrier();
      const bool same = (t0 >= every.lo || any.lo == every.lo) && (t0 + kTile <= every.hi || any.hi == every.hi);
      i32x2 vc[D / 16];
#pragma unroll
      for (int c = 0; c < D / 16; ++c) vc[c] = value_codes<D>(vl, c);
      f16x8 w[1][2];
      soft_weights<D, 1>(s.t.ks[wave], s.t.lv[wave], s.t.iv[wave], t0, same, unit, rs, lo, hi, sc, M, l, o, w);
      // values times weights, 16 channels at a time
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const f16x8 vf = e2m1_f16x8((uint32_t)vc[c][k]);
          o[0][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, w[0][k], o[0][c], 0, 0, 0);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// ---------------------------------------------------------------------------
// Many query rows (prefill): a workgroup takes 128 rows of one key/value head, each wave 32 of its own,
// and all four read the same key tiles.  A tile (64 keys: codes as they are, 8 KB, and the scales)
// goes through LDS in two buffers with one barrier a tile, the next one's loads in flight meanwhile; each wave
// converts what it multiplies.

template <int D>
struct PrefillLds {
  struct Buf {
    alignas(16) uint8_t k[kTile * D / 2], v[kTile * D / 2];
    alignas(16) float ks[kTile], lv[kTile], iv[kTile];
    int held[4];                                      // whether each 16 keys lie in a page
  } buf[2];
};

// A row's channels lie at 16c + 4g + j in o[c][j] of lane group g: rotated over c and j in the lane and over g between
// lanes, one of a pair of registers going to each lane (or, not rotated, only exchanged).  Four registers' exchange leaves
// lane group g with channels 16 (4i + g) ... 16 (4i + g) + 15 in o[4i] ... o[4i + 3].
template <int D>
__device__ __forceinline__ void transform_tile(f32x4* o, bool rotate) {
  if (rotate) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const f32x4 x = o[c];
      const float a = x[0] + x[1], b = x[0] - x[1], d = x[2] + x[3], e = x[2] - x[3];
      o[c] = f32x4{a + d, b + e, a - d, b - e};
    }
#pragma unroll
    for (int h = 1; h < D / 16; h *= 2)
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        if (!(c & h)) {
          const f32x4 x = o[c], y = o[c + h];
          o[c] = x + y;
          o[c + h] = x - y;
        }
  }
  // lane pairs 16 apart trade within (c, c + 1), pairs 32 apart within (c, c + 2)
#pragma unroll
  for (int far = 0; far < 2; ++far)
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      if (!(c & (1 << far)))
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d = c + (1 << far);
          const uint32_t u = float_bits(o[c][j]), v = float_bits(o[d][j]);
          u32x2 t;
          if (far) { const auto r = __builtin_amdgcn_permlane32_swap(u, v, false, false); t = u32x2{r[0], r[1]}; }
          else { const auto r = __builtin_amdgcn_permlane16_swap(u, v, false, false); t = u32x2{r[0], r[1]}; }
          const float x = __builtin_bit_cast(float, (uint32_t)t[0]), y = __builtin_bit_cast(float, (uint32_t)t[1]);
          o[c][j] = rotate ? x + y : x;
          o[d][j] = rotate ? x - y : y;
        }
}

template <int D>
__global__ __launch_bounds__(256, 2) void kv_prefill_kernel(KvAttnArgs g, SplitArgs sp) {
  constexpr int NB = 2, ROWS = 64 * NB;               // tiles of 16 query rows a wave; rows of a workgroup
  typedef typename Chunk<D>::T C;
  __shared__ PrefillLds<D> s;
  const KvArgs& a = g.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t mask = (1u << a.logp) - 1;
  if (tid == 0 && sp.split) sp.desc[blockIdx.x].more = 0;
  Walk<ROWS> u;
  u.start(g, sp);
  const float c_scale = g.scale * sp.c_q * 1.44269504088896341f;
  while (u.next(g, sp)) {
    const Seq q = u.q;
    const int r0 = u.row0, kvh = u.h, b = u.seq;
    const int t_lo = u.tiles.lo, t_hi = u.tiles.hi;

    // ---- the wave's queries
    const int w0 = r0 + 16 * NB * wave;           // its first row
    const int w_rows = min(16 * NB, q.rows - w0); // may be <= 0
    f16x8 qf[NB][D / 32];
    float rs[NB], M[NB], l[NB];
    int lo[NB], hi[NB];
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int rr = 16 * n + (lane & 15);
      const bool row = rr < w_rows;
      const int r = row ? w0 + rr : r0;
      convert_queries<D>(fetch_queries<D>(g, sp, q, kvh, r, row), a.rotate & 1, c_scale, qf[n], &rs[n]);
      const Range w = kv_range(q, div_g(sp, r), g.causal, g.window);
      lo[n] = w.lo;
      hi[n] = row ? w.hi : 0;
      M[n] = -INFINITY;
      l[n] = 0;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[n][c] = f32x4{0, 0, 0, 0};
    }
    // positions that some row of the block attends, that some and that every row of the wave does
    const Range block{kv_range(q, div_g(sp, r0), g.causal, g.window).lo,
                      kv_range(q, div_g(sp, min(r0 + ROWS, q.rows) - 1), g.causal, g.window).hi};
    Range any{0, 0}, every{0, 0};
    if (w_rows > 0) {
      const Range r_first = kv_range(q, div_g(sp, w0), g.causal, g.window);
      const Range r_last = kv_range(q, div_g(sp, w0 + w_rows - 1), g.causal, g.window);
      any = Range{r_first.lo, r_last.hi};
      every = Range{r_last.lo, r_first.hi};
    }
    bool unit = true;
#pragma unroll
    for (int n = 0; n < NB; ++n) unit = unit && !__any(rs[n] != 1.0f);

    // ---- the tiles: each wave brings 16 keys of each
    C kr, vr;
    const float* scales = ((lane & 16) ? a.scales[1] : a.scales[0]) + (lane & 15);
    float scale = 0;
    int held = 0, pages = 0;
    auto fetch = [&](int tile, int at) {
      const int p0 = __builtin_amdgcn_readlane(pages, at);
      held = p0 >= 0;
      const int p = p0 >= 0 ? p0 : 0;             // keys in no page: any page is read, and masked
      const int64_t row = ((int64_t)(p * a.n_kv + kvh) << a.logp) + ((tile * kTile + 16 * wave) & mask);
      kr = *reinterpret_cast<const C*>(a.codes[0] + row * (D / 2) + lane * (D / 8));
      vr = *reinterpret_cast<const C*>(a.codes[1] + row * (D / 2) + lane * (D / 8));
      scale = scales[row];
    };
    auto page_batch = [&](int tile) { pages = kv_page(a, b, (int64_t)(tile + lane) * kTile + 16 * wave); };
    page_batch(t_lo);
    fetch(t_lo, 0);
    lds_barrier();                                // the last block's tiles have been read
    int at = 0;
    for (int tile = t_lo; tile < t_hi; ++tile) {
      auto& B = s.buf[(tile - t_lo) & 1];
      {
        const int key = 16 * wave + (lane >> 2);
        *reinterpret_cast<C*>(B.k + key * (D / 2) + ((lane & 3) ^ ((lane >> 4) & 3)) * (D / 8)) = kr;
        *reinterpret_cast<C*>(B.v + key * (D / 2) + ((lane & 3) ^ wave) * (D / 8)) = vr;
        const int at16 = 16 * wave + (lane & 15), pos = tile * kTile + at16;
        const bool some = held && pos >= block.lo && pos < block.hi;
        if (lane < 16) stage_key(scale, some, &B.ks[at16]);
        if (lane >= 16 && lane < 32) stage_value(scale, some, &B.lv[at16], &B.iv[at16]);
        if (lane == 0) B.held[wave] = held;
      }
      lds_barrier();
      if (tile + 1 < t_hi) {
        if (++at == 64) { page_batch(tile + 1); at = 0; }
        fetch(tile + 1, at);
      }
      const int t0 = tile * kTile;
      if (t0 >= any.hi || t0 + kTile <= any.lo) continue;
      f32x4 sc[NB][4];
      // The softmax at a lower priority than the rest: what feeds the matrix cores goes first, and the other wave's
      // vector work fills in (chunk of 512: 164 us; 180 without).
      __builtin_amdgcn_s_setprio(1);
      C kc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        kc[i] = *reinterpret_cast<const C*>(B.k + (16 * i + (lane & 15)) * (D / 2) + ((lane >> 4) ^ ((lane >> 2) & 3)) * (D / 8));
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 kf = e2m1_f16x8(kc[i][k]);
#pragma unroll
          for (int n = 0; n < NB; ++n)
            sc[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][k], k ? sc[n][i] : f32x4{0, 0, 0, 0}, 0, 0, 0);
        }
      __builtin_amdgcn_s_setprio(0);
      if (!(B.held[0] | B.held[1] | B.held[2] | B.held[3])) continue;
      const bool same = t0 >= every.lo && t0 + kTile <= every.hi;
      i32x2 vc[D / 16];
#pragma unroll
      for (int c = 0; c < D / 16; ++c) vc[c] = value_codes<D>(B.v, c);
      f16x8 w[NB][2];
      soft_weights<D, NB>(B.ks, B.lv, B.iv, t0, same, unit, rs, lo, hi, sc, M, l, o, w);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const f16x8 vf = e2m1_f16x8((uint32_t)vc[c][k]);
#pragma unroll
          for (int n = 0; n < NB; ++n) o[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, w[n][k], o[n][c], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_s_setprio(0);

    // ---- the rows, each in its wave
    const bool starts = u.u0 == 0, ends = u.u1 == u.units;
    const int64_t part = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int rr = 16 * n + (lane & 15);
      const float sum = row_add(l[n]);
      if (starts && ends) {
        transform_tile<D>(o[n], a.rotate & 2);
        const float f = sum != 0.0f ? sp.c_v / sum : 0.0f;
        if (rr < w_rows) {
          const int r = w0 + rr, i = div_g(sp, r), h = r - i * sp.G;
          uint16_t* dst = g.out + (int64_t)(q.t0 + i) * g.ldo + (kvh * sp.G + h) * D + 16 * (lane >> 4);
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            u32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f32x4 v = o[n][c + e / 2];
              x[e] = (uint32_t)f32_to_bf16_rne(v[2 * (e & 1)] * f) | ((uint32_t)f32_to_bf16_rne(v[2 * (e & 1) + 1] * f) << 16);
            }
            *reinterpret_cast<u32x4*>(dst + 64 * (c / 4) + 4 * (c & 3)) = x;
          }
        }
      } else if (rr < w_rows) {
        const int64_t at_row = part * ROWS + 16 * NB * wave + rr;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) *reinterpret_cast<f32x4*>(sp.o + at_row * D + 16 * c + 4 * (lane >> 4)) = o[n][c];
        if (lane < 16) sp.ml[at_row] = float2{M[n], sum};
      }
    }
    if (starts && !ends && tid == 0)
      sp.desc[blockIdx.x] = Desc{q.t0, kvh, r0, min(ROWS, q.rows - r0), u.following(sp)};
  }
}

// Joins the parts of a row block that starts in group blockIdx.x and goes on in the next ones.  RB rows a workgroup, from
// RB * blockIdx.y on, and a row's parts dealt out to NG groups of D/8 lanes.
template <int D, int ROWS, int RB>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttnArgs g, SplitArgs sp) {
  constexpr int L = D / 8, NG = 256 / L / RB;
  const int tid = threadIdx.x, sub = tid % L, grp = tid / L % NG, rb = tid / L / NG;
  const int w = blockIdx.x, row = blockIdx.y * RB + rb;
  const Desc d = sp.desc[w];
  if (d.more == 0) return;
  const bool mine = row < d.rows;
  if (RB == 1 && !mine) return;
  __shared__ float so[RB][NG][D], sm[RB][NG], sl[RB][NG];
  // part 0 is the block's start (second slot of w), part p the first slot of w + p
  float m = -INFINITY, sum = 0, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int p = grp; mine && p <= d.more; p += NG) {
    const int64_t part = (p == 0 ? 2 * (int64_t)w + 1 : 2 * (int64_t)(w + p)) * ROWS + row;
    const float2 ml = sp.ml[part];
    const f32x4 x0 = *reinterpret_cast<const f32x4*>(sp.o + part * D + 8 * sub);
    const f32x4 x1 = *reinterpret_cast<const f32x4*>(sp.o + part * D + 8 * sub + 4);
    const float mn = fmaxf(m, ml.x), ref = safe_max(mn);
    const float f0 = __builtin_amdgcn_exp2f(m - ref), f1 = __builtin_amdgcn_exp2f(ml.x - ref);
    sum = sum * f0 + ml.y * f1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = v[j] * f0 + x0[j] * f1;
      v[4 + j] = v[4 + j] * f0 + x1[j] * f1;
    }
    m = mn;
  }
  if constexpr (NG > 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) so[rb][grp][8 * sub + j] = v[j];
    if (sub == 0) { sm[rb][grp] = m; sl[rb][grp] = sum; }
    __syncthreads();
    if (grp != 0) return;
    const int n = d.more + 1 < NG ? d.more + 1 : NG;
    for (int p = 1; p < n; ++p) m = fmaxf(m, sm[rb][p]);
    const float ref = safe_max(m);
    sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
    for (int p = 0; p < n; ++p) {
      const float f = __builtin_amdgcn_exp2f(sm[rb][p] - ref);
      sum = __builtin_fmaf(sl[rb][p], f, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(so[rb][p][8 * sub + j], f, v[j]);
    }
  }
  if (!mine) return;                                  // whole groups of lanes
  const int r = d.r0 + row, i = div_g(sp, r), h = r - i * sp.G;
  finish_row<D>(v, sum, g.kv.rotate & 2, sp.c_v, sub, g.out + (int64_t)(d.t0 + i) * g.ldo + (d.kvh * sp.G + h) * D + 8 * sub);
}

// Query rows of a row block, by the rows a sequence has on average and all rows together.  16 rows share keys among eight
// waves and start sooner, 128 rows read them once for all.  Which is faster goes by rows times keys, about 25 million
// of them; the keys' number stays on the device, so long sequences just within the limits take the slower form (8 of 4096 with
// 128 rows, one of 16384 with 512), and so do sequences whose rows are far from the average (512 tokens of 16384 among 63 single
// tokens of 1000 to 4000: 306 us in one call, 160 and 41 in two).  Both forms, 8 key/value heads, rows a sequence:
//   1 sequence  of  1000: 512 rows 12 and 28 us; of 4096: 256 24 and 31, 512 35 and 40; of 16384: 256 47 and 54, 512 78 and 66
//   2 sequences of  8192: 256 43 and 48, 384 68 and 56
//   4 sequences of  2048: 128 16 and 32, 256 28 and 40, 512 50 and 48; of 8192: 96 46 and 44, 128 54 and 49, 256 95 and 65
//   8 sequences of  4096: 64 32 and 40, 96 49 and 44, 128 57 and 48, 256 100 and 65
//   16 sequences of 2048: 96 39 and 43, 128 52 and 48, 256 97 and 67
bool few_rows(int64_t T, int n_q) { return T * n_q <= 4096; }
int row_block(int64_t T, int B, int n_q, int n_kv) {
  const int64_t rows = (T + B - 1) / B * (n_q / n_kv);
  return rows <= 128 || few_rows(T, n_q) ? 16 : 128;
}

size_t workspace_of(int rows, int D) {
  return (size_t)max_groups(rows) * (sizeof(Desc) + 2 * rows * (sizeof(float2) + D * sizeof(float)));
}

// Whether row blocks are cut, for a second launch that joins them (about 4 us and the parts' traffic).
//  16 rows: a whole block takes 7.5 us and 0.23 a key tile; cutting pays
//   - from 1536 positions (8 heads, one sequence of 1203: 11.3 against 12.3 us; of 2011: 14.4 against 12.7, of 4096: 22
//     against 13);
//   - with 64 row blocks from 2560 (16 heads, 4 of 2011: 12.2 against 12.9; of 4096: 17.8 against 15.0);
//   - with 128 from 4096 (8 heads, 16 of 2011: 15.9 against 19.2; of 4096: the same; of 16384: 68 against 54);
//   - beyond 256 from 2048 (8 heads, 40 of 8 to 1500: 21.9 against 23.3; to 3000: 33 against 27; 256 of 8 to 1500: 79
//     against 75, to 4000: 164 against 127).  Sequences of equal length lose by that, less than ragged ones gain (8 heads, 64
//     of 2500: 35.8 against 38.3, of 3100: 42.8 against 44.5; 16 heads of 64, 64 of 2500: 43.0 against 46.1).
//   All of it by the table's width, which is what the host knows of the lengths: under a table for far longer ones short
//   sequences are cut too (16 of 1203 under one for 131072 positions 14.6 instead of 11.7, with 5 tokens each 21.8 instead of
//   12.6; 16 of 300 with 64 tokens each 35 instead of 19).
//   With a window, and as many tokens in each sequence (no offsets, or one each), row blocks are alike but for sequences
//   shorter than it, and whole ones lose only what the last 256 leave idle (8 heads of 64, window 4096, 16 sequences: 18.2
//   against 21.0; 32: 19.3 against 27.3, some of them as short as 200: 17.5 against 23.5; 40: 32.1 against 30.9, 48:
//   32.4 against 34.4; window 8192: 28.6 against 25.9, 29.3 against 34.2, 52.7 against 40.4, 52.7 against 44.4).
//  128 rows: whole blocks take 8 us and 1.75 a key tile, in rounds of 512 where the longest go first; cut ones 22 us and
//  half as much again, evenly (64 new tokens, 8 heads, one sequence of 1024: 35.5 against 25 us; 16 of them: 37 against 51;
//  a prompt of 2048: 70 against 91).
bool split_pays(const KvAttnArgs& g, int rows, int64_t blocks, int64_t cap) {
  if (blocks >= 1 << 24) return false;                // enough work for any chip, and the units of fewer fit 31 bits
  const KvArgs& a = g.kv;
  if (rows == 16) {
    const int64_t idle = -blocks & (max_groups(16) - 1);
    if (g.window && (!a.offsets || a.T == a.B) && blocks >= 128 && idle <= (cap > 80 ? 64 : 128)) return false;
    return cap > (blocks > 256 ? 33 : blocks >= 128 ? 65 : blocks >= 64 ? 41 : 25);
  }
  const int64_t G = g.n_q / a.n_kv;
  const double n = a.n_kv * (a.offsets ? (double)(a.T * G / rows) + 0.5 * a.B
                                       : (double)a.B * ((a.per_seq * G + rows - 1) / rows));
  const double mean = g.causal ? std::max((double)cap - (double)(a.T / a.B) / (2 * kTile), 0.5 * cap) : (double)cap;
  const double whole = std::max(8 + 1.75 * cap, n * (8 + 1.75 * mean) / 512);
  return 22 + 1.5 * n * 1.75 * mean / 512 < whole;
}

template <int D>
hipError_t launch_decode(const KvAttnArgs& g, SplitArgs sp, hipStream_t stream) {
  kv_attention_kernel<D><<<sp.groups, 64 * kWaves, 0, stream>>>(g, sp);
  if (hipError_t e = hipGetLastError()) return e;
  if (!sp.split) return hipSuccess;
  kv_join_kernel<D, 16, 1><<<dim3(sp.groups, sp.join_rows), 256, 0, stream>>>(g, sp);
  return hipGetLastError();
}

template <int D>
hipError_t launch_prefill(const KvAttnArgs& g, SplitArgs sp, hipStream_t stream) {
  kv_prefill_kernel<D><<<sp.groups, 256, 0, stream>>>(g, sp);
  if (hipError_t e = hipGetLastError()) return e;
  if (!sp.split) return hipSuccess;
  kv_join_kernel<D, 128, 8><<<dim3(sp.groups, (sp.join_rows + 7) / 8), 256, 0, stream>>>(g, sp);
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t T, int B, int n_q, int n_kv, int D) {
  return workspace_of(row_block(T, B, n_q, n_kv), D);
}

size_t kv_attention_workspace_most(int64_t T, int n_q, int D) { return workspace_of(few_rows(T, n_q) ? 16 : 128, D); }

hipError_t launch_kv_attention(const KvAttnArgs& g, hipStream_t stream) {
  const KvArgs& a = g.kv;
  const int G = g.n_q / a.n_kv, rows = row_block(a.T, a.B, g.n_q, a.n_kv), most = max_groups(rows);
  SplitArgs sp{};
  const float c = (float)(1.0 / std::sqrt((double)a.D));
  sp.c_q = a.rotate & 1 ? c : 1.0f;
  sp.c_v = a.rotate & 2 ? c : 1.0f;
  sp.desc = static_cast<Desc*>(g.ws);
  sp.ml = reinterpret_cast<float2*>(sp.desc + most);
  sp.o = reinterpret_cast<float*>(sp.ml + (size_t)2 * most * rows);
  sp.G = G;
  const uint32_t lg = G > 1 ? 32 - __builtin_clz(G - 1) : 0;                // 2^lg >= G
  sp.g_shift = 31 + lg;
  sp.g_mul = (uint32_t)(((uint64_t(1) << sp.g_shift) + G - 1) / G);
  const int64_t own = (int64_t)a.per_seq * G;
  sp.join_rows = a.offsets || own > rows ? rows : (int)own;
  // Row blocks at most.  With offsets: a sequence of n tokens has ceil(n G / rows) <= n ceil(G / rows), and its last block
  // lacks rows - 1 rows at most; with one token a sequence that is the number without offsets, so the call is the same.
  const int64_t ragged = std::min(a.T * ((G + rows - 1) / rows), (a.T * G + (rows - 1) * std::min<int64_t>(a.T, a.B)) / rows);
  const int64_t blocks = (a.offsets ? ragged : a.B * ((own + rows - 1) / rows)) * a.n_kv;
  int64_t cap = ((int64_t)a.max_pages << a.logp) / kTile + 1;               // key tiles of one at most
  if (g.window) cap = std::min(cap, ((int64_t)g.window + rows / G + 1) / kTile + 2);
  sp.split = split_pays(g, rows, blocks, cap);
  sp.min_units = 1;
  int64_t want = blocks;
  if (sp.split) {
    // Fewer than 4 key tiles to a workgroup only make more parts: one head, one sequence of 4096, at least 1: 19 us, 4: 13, 16: 16.
    sp.min_units = 4;
    // Queries, sums over the waves and results of a row block against key tiles.  64 ragged sequences: 48 us; counted as 8
    // 56, as 64 54; drafted tokens 30, 35 and 33.  128 rows: 0 and 4 take what 1 does, within 1 %.
    sp.start_cost = rows == 128 ? 1 : 24;
    while (blocks * ((cap >> sp.shift) + 1 + sp.start_cost) >= 0x7FFFFFFF - most) ++sp.shift;
    want = (blocks * ((cap >> sp.shift) + 1 + sp.start_cost) + sp.min_units - 1) / sp.min_units;
  }
  const int64_t limit = rows == 128 && !sp.split ? 1 << 22 : most;
  sp.groups = (int)(want < limit ? want : limit);
  if (rows == 128) return a.D == 64 ? launch_prefill<64>(g, sp, stream) : launch_prefill<128>(g, sp, stream);
  return a.D == 64 ? launch_decode<64>(g, sp, stream) : launch_decode<128>(g, sp, stream);
}

}  // namespace cbq
