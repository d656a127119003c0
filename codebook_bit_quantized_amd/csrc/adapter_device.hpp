// The order in which tiles take the tokens of many adapters (gfx950, wave64).
#pragma once
#include "cbq_internal.hpp"

namespace cbq {

// Places for the tokens of a group of G (n of them exist) by adapter, so that tiles cut from it
// hold few adapters each in whatever order the tokens come: equal adapters lie together, in
// token order, tokens without one behind them (of: the group's entries).  Where the group
// changes adapters in at most G / 16 places, as where requests are contiguous, tokens keep
// theirs.  Workgroups of at least G threads; every thread calls it.  Calls put(place, token,
// adapter) for every token below n (adapter -1: none); the caller waits before it reads what
// that wrote.  Costs G compares a token, a fraction of a microsecond.
template <int G, typename Put>
__device__ __forceinline__ void order_by_adapter(const int32_t* of, int n, int n_adapters, int tid, uint32_t* s_key, Put put) {
  constexpr uint32_t kNone = 0x7FFFFFFFu, kBehind = 0xFFFFFFFFu;
  uint32_t key = kBehind;
  if (tid < n) {
    const int a = of[tid];
    key = (uint32_t)a < (uint32_t)n_adapters ? (uint32_t)a : kNone;
  }
  if (tid < G) s_key[tid] = key;
  lds_barrier();
  int changes = 0;
#pragma unroll
  for (int i = 0; i < G; i += 64) {
    const int j = i + (tid & 63);
    changes += __popcll(__ballot(s_key[j] != s_key[j > 0 ? j - 1 : 0]));
  }
  int place = tid;
  if (changes > G / 16) {                    // the same for every wave
    place = 0;
#pragma unroll 4
    for (int j = 0; j < G; j += 4) {
      const u32x4 k = *reinterpret_cast<const u32x4*>(s_key + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) place += k[i] < key || (k[i] == key && j + i < tid) ? 1 : 0;
    }
  }
  if (tid < n) put(place, tid, key == kNone ? -1 : (int)key);
}

}  // namespace cbq
