// Internal launch interface between the C ABI layer and the HIP kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "cbq_device.hpp"

namespace cbq {

// Where 2- and 3-bit codebooks are looked up: each path's default, register tables or
// LDS pair tables.
enum { kTablesDefault = 0, kTablesReg = 1, kTablesLds = 2 };

// Device view of one weight set (see cbq_weights in cbq.h).
struct GemmW {
  const uint8_t* idx;
  const uint16_t* codebook;
};

struct GemmArgs {
  const uint8_t* codes;
  const float* scales;
  int act_bits;
  int64_t n_rows;
  const int32_t* offsets;   // nullptr: dense
  const int32_t* row_token; // nullptr: identity
  GemmW w[2];
  int n_w;
  int E, N, K, bits;
  bool swiglu;
  int tables;               // kTables*: placement of 2- and 3-bit codebook tables
  int blocked;              // 1: indices in the blocked layout (cbq_prepack_weights)
  void* out;
  int64_t ldo;
  void* ws;                 // optional workspace (K-split partial sums of the MFMA path)
  size_t ws_bytes;
};

hipError_t launch_rotate_quantize(const uint16_t* x, int64_t T, int K, int64_t ldx, int b,
                                  int act_bits, const float* smooth, const uint8_t* signs,
                                  uint8_t* codes, float* scales, uint32_t* precond,
                                  hipStream_t stream);

// Norms around a block (norm_quantize.hip).  Pointers may be null where the comment says so.
// What is normed: x, or combined rows of that type; or fp32 rows rotated and quantised as they
// are (no norm; codes then gets the few-row GEMM's fp16 codes, few_device.hpp).
enum { kNormX = 0, kNormF32 = 1, kNormBF16 = 2, kRotateF32 = 3 };
struct NormArgs {
  const uint16_t* x;          // bf16 [T][ldx]: the row, or the residual stream beside rows
  int64_t ldx;
  const void* rows;           // fp32 or bf16 [T*topk + n_shared*T][ldr]
  int64_t ldr;
  const int32_t* slot_of;     // [T][topk]
  const float* topk_w;        // [T][topk]
  int topk, n_shared;
  const float* post_weight;   // [K] or null: no norm of the combined row
  float post_eps;
  const uint16_t* gate;       // bf16 [T][ldg] (ldg 0: one row for all) or null
  int64_t ldg;
  float scale;
  uint16_t* out;              // bf16 [T][ldo]
  int64_t ldo;
  const float* weight;        // [K] or null: nothing after out
  float eps;
  uint16_t* normed;           // bf16 [T][ldn] or null
  int64_t ldn;
  uint8_t* codes;             // packed codes or null
  float* scales;
  int act_bits;
  int64_t T;
  int K;
  int logb;                   // set by the launcher, as the next three
  float c_b;
  double inv_K;
  int64_t t0;                 // first token of the launch
};
hipError_t launch_norm_quantize(NormArgs a, int src, int b, hipStream_t stream);

// The few-token MoE layer (moe_few.hip).  FewArgs: one of its grouped GEMMs.
struct FewArgs {
  const float* logits;        // [T][E]
  int32_t* ids;               // [T][topk]
  int T, E, topk, n_shared;
  const uint8_t* codes;       // code rows: tokens (gate/up) or choices (down)
  const float* scales;
  GemmW w[2];
  int N, K, blocked;
  float* out;                 // fp32 [T*topk + n_shared*T][N]
};
struct FewDownArgs {
  const float* h;             // fp32 [topk + n_shared][F]
  const int32_t* ids;         // [topk]
  const float* logits;        // [E]
  int E, topk, n_shared, renormalize, act_bits, H, F;
  GemmW w;
  int blocked;
  float c_b;                  // 1 / sqrt(rotation block)
  void* y;                    // [H]
  int y_bf16;
};
struct MoeFewArgs {
  const uint8_t* codes;
  const float* scales;
  const float* logits;
  int T, E, topk, n_shared, renormalize, act_bits, H, F;
  GemmW gate, up, down;
  int bits_gu, bits_d, blocked_gu, blocked_d;
  void* y;
  int64_t ldy;
  int y_bf16;
  void* ws;
};
size_t moe_few_workspace_bytes(int64_t T, int topk, int n_shared, int H, int F);
hipError_t launch_moe_few(const MoeFewArgs& m, hipStream_t stream);

// Low-rank adapters beside a projection (adapter_gemm.hip): what the projection's epilogue
// reads.  Token t of adapter a = of[t] (none outside [0, n_adapters)) adds
// sum_r u[t][r] lora_b[a][n][r] to column n.
struct AdapterArgs {
  const int32_t* of;          // [T]
  int n_adapters, rank;       // rank: a multiple of 8
  const uint16_t* lora_b;     // bf16 [n_adapters][N][rank]
  const float* u;             // fp32 [parts][T][rank], to be summed in order
  int parts;
  int64_t part_stride;        // T * rank
};
size_t adapter_workspace_bytes(int64_t T, int rank);
hipError_t launch_adapter_gemm(const GemmArgs& a, AdapterArgs ad, const uint16_t* x, int64_t ldx,
                               const uint16_t* lora_a, const float* adapter_scale, float* u, hipStream_t stream);
// The MFMA path with the adapters in its epilogue: one weight set, dense rows.
hipError_t launch_mfma_prefill_adapter(const GemmArgs& a, const AdapterArgs& ad, hipStream_t stream);

// The 4-bit key/value cache and the sequences of a step (kv_cache.hip, kv_attention.hip).
struct KvArgs {
  uint8_t* codes[2];          // keys, values
  float* scales[2];
  int n_pages, n_kv, logp, D; // logp: log2 of the page's tokens
  int rotate;                 // bit 0 keys, bit 1 values
  const int32_t* table;       // or null: sequence b's pages are b*max_pages ...
  int64_t ld_table;
  int max_pages;
  const int32_t* lens;
  const int32_t* offsets;     // or null: per_seq tokens each
  int B, per_seq;
  int64_t T;
};
hipError_t launch_kv_write(const KvArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                           hipStream_t stream);
hipError_t launch_kv_read(const KvArgs& a, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv, hipStream_t stream);
struct KvAttnArgs {
  KvArgs kv;
  const uint16_t* q;
  int64_t ldq;
  int n_q;
  float scale;
  int causal, window;
  uint16_t* out;
  int64_t ldo;
  void* ws;
};
size_t kv_attention_workspace_bytes(int64_t T, int B, int n_q, int n_kv, int D);   // of one call
size_t kv_attention_workspace_most(int64_t T, int n_q, int D);                     // of any with at most T tokens
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream);

// Compute units of the current device (cached per device after the first query).
hipError_t device_cu_count(int* out);

size_t route_workspace_bytes(int64_t T, int E);
// The library's own route scratch (no allocation): its size, and its device address on
// the current device (looked up on that device's first call).
size_t route_scratch_bytes();
hipError_t route_scratch(int32_t** out);
hipError_t launch_route(const float* logits, int64_t T, int E, int topk, int renormalize,
                        int n_shared, int32_t* ids, float* w, int32_t* offsets,
                        int32_t* sorted_tokens, int32_t* slot_of, int32_t* ws, hipStream_t stream);

// LUT (decode) path.  max_rows >= 0: experts with more rows are skipped (AUTO split).
hipError_t launch_lut_decode(const GemmArgs& a, int max_rows, hipStream_t stream);

// MFMA (prefill) path.  Experts with at most min_rows rows are skipped (AUTO split).
hipError_t launch_mfma_prefill(const GemmArgs& a, int min_rows, hipStream_t stream);

// Workspace bytes with which a single-matrix MFMA call of these sizes may split K in two
// (0: it never splits).  The launcher splits when the workspace holds that many bytes and
// the call's 256-row tiles would leave CUs idle.
size_t mfma_split_workspace_bytes(int n_w, int bits, int64_t n_rows, int N, int K);

// The pages' table forms (4-bit codebooks, A4): mode 0 per-row product tables with sign
// folding, mode 1 per-row integer buckets of the activation codes.
hipError_t launch_lut_pages(const GemmArgs& a, int mode, hipStream_t stream);

// Regroups a row-layout index block [E][N][K*bits/8] into the blocked layout.
hipError_t launch_prepack(const uint8_t* src, uint8_t* dst, int E, int N, int K, int bits,
                          hipStream_t stream);

// Bytes per row of one expert's index block: K (rows layout) or K rounded up to a
// multiple of 128 (blocked layout), times bits / 8.
__host__ __device__ inline int64_t index_row_bytes(int K, int bits, bool blocked) {
  const int64_t kp = blocked ? (int64_t)(K + 127) / 128 * 128 : K;
  return kp * bits / 8;
}

hipError_t launch_kmeans(const uint16_t* w, int64_t R, int K, int64_t ldw, int bits, int max_iters,
                         uint8_t* idx, uint16_t* codebook, int32_t* iters_done,
                         hipStream_t stream);

hipError_t launch_refit(const uint16_t* w, int64_t R, int K, int64_t ldw, int bits, const uint8_t* idx,
                        const uint16_t* x, int n, int64_t ldx, uint16_t* codebook, hipStream_t stream);

size_t dense_rotation_workspace_bytes(int64_t T, int K);
hipError_t launch_rotate_dense(const uint16_t* x, int64_t T, int K, int64_t ldx, const uint16_t* R,
                               int act_bits, uint8_t* codes, float* scales, uint32_t* precond,
                               void* ws, hipStream_t stream);

hipError_t launch_combine(const float* expert_out, const int32_t* slot_of, const float* w,
                          int64_t T, int topk, int H, int n_shared, float* y, hipStream_t stream);

}  // namespace cbq
