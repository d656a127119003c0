// Attention of a step's queries over the 4-bit key/value cache.
//
// One workgroup a query row and head, one pass over its keys in blocks of 256 with the running
// maximum and sum of the softmax: thread i holds key i's score, then channel i's sum.
#include "kv_device.hpp"

namespace cbq {
namespace {

template <int D>
__device__ __forceinline__ void head_transform_lds(float* x, int tid) {
  for (int h = 1; h < D; h *= 2) {
    __syncthreads();
    float r = 0;
    if (tid < D) r = (tid & h) ? x[tid ^ h] - x[tid] : x[tid] + x[tid ^ h];
    __syncthreads();
    if (tid < D) x[tid] = r;
  }
  __syncthreads();
}

__device__ __forceinline__ float e2m1_value(uint32_t n) {
  const float m = (n & 6) ? (1.0f + 0.5f * (n & 1)) * (float)(1 << (((n >> 1) & 3) - 1)) : 0.5f * (n & 1);
  return (n & 8) ? -m : m;
}

template <int D>
__global__ __launch_bounds__(256) void kv_attention_kernel(KvAttnArgs g, float c_b) {
  const KvArgs& a = g.kv;
  __shared__ float q[D], o[D], w[256], red[256];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, kvh = h / (g.n_q / a.n_kv);
  const int b = kv_seq_of(a, t);
  if (b < 0) return;
  const int64_t pos = kv_position(a, b, t);
  if (tid < D) {
    q[tid] = bf16_to_f32(g.q[t * g.ldq + (int64_t)h * D + tid]);
    o[tid] = 0;
  }
  if (a.rotate & 1) head_transform_lds<D>(q, tid);
  __syncthreads();
  const int64_t cap = (int64_t)a.max_pages << a.logp;
  int64_t hi = a.lens[b] < cap ? a.lens[b] : cap, lo = 0;
  if (g.causal && pos + 1 < hi) hi = pos + 1;
  if (g.window && pos - g.window + 1 > 0) lo = pos - g.window + 1;
  const float sc = g.scale * ((a.rotate & 1) ? c_b : 1.0f);
  float m = -INFINITY, l = 0;
  for (int64_t j0 = lo; j0 < hi; j0 += 256) {
    const int64_t j = j0 + tid;
    const int page = j < hi ? kv_page(a, b, j) : -1;
    float s = -INFINITY, vs = 0;
    if (page >= 0) {
      const int64_t at = kv_row(a, page, kvh, j);
      const uint8_t* c = a.codes[0] + at * (D / 2);
      float d = 0;
      for (int i = 0; i < D / 2; ++i)
        d += q[2 * i] * e2m1_value(c[i] & 15) + q[2 * i + 1] * e2m1_value(c[i] >> 4);
      s = d * a.scales[0][at] * sc;
      vs = a.scales[1][at];
    }
    __syncthreads();
    red[tid] = s;
    __syncthreads();
    float mn = m;
    for (int i = 0; i < 256; ++i) mn = fmaxf(mn, red[i]);
    const float ms = mn == -INFINITY ? 0 : mn;
    const float p = page >= 0 ? expf(s - ms) : 0;
    __syncthreads();
    red[tid] = p;
    w[tid] = page >= 0 ? p * vs : 0;
    __syncthreads();
    const float keep = expf(m - ms);
    l *= keep;
    for (int i = 0; i < 256; ++i) l += red[i];
    if (tid < D) {
      float x = o[tid] * keep;
      for (int i = 0; i < 256 && j0 + i < hi; ++i) {
        const int pg = kv_page(a, b, j0 + i);
        if (pg < 0) continue;
        const uint8_t c = a.codes[1][kv_row(a, pg, kvh, j0 + i) * (D / 2) + tid / 2];
        x += w[i] * e2m1_value((tid & 1) ? c >> 4 : c & 15);
      }
      o[tid] = x;
    }
    m = mn;
  }
  __syncthreads();
  if (a.rotate & 2) head_transform_lds<D>(o, tid);
  __syncthreads();
  if (tid < D) {
    const float x = l != 0 ? o[tid] / l * ((a.rotate & 2) ? c_b : 1.0f) : 0;
    g.out[t * g.ldo + (int64_t)h * D + tid] = f32_to_bf16_rne(x);
  }
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t T, int B, int n_q, int n_kv, int D) { return 16; }

hipError_t launch_kv_attention(const KvAttnArgs& g, hipStream_t stream) {
  const float c_b = (float)(1.0 / std::sqrt((double)g.kv.D));
  auto f = g.kv.D == 64 ? kv_attention_kernel<64> : kv_attention_kernel<128>;
  f<<<dim3((uint32_t)g.kv.T, g.n_q), 256, 0, stream>>>(g, c_b);
  return hipGetLastError();
}

}  // namespace cbq
