// Launch arguments of the kernels of the 4-bit KV cache (kv4.cu, kv4_attention.cu,
// kv4_attention_tc.cu, kv4_weights.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dflash.h"

namespace df {

constexpr int kKv4Codes = 64;   // bytes of codes of one cache row (128 values of 4 bits)
constexpr int kKv4Scales = 8;   // bytes of scales of one cache row (one for 16 values)

// The planes of one layer, or of all layers.
struct Kv4Planes {
  uint8_t *kc, *ks, *vc, *vs;   // [.. b][Hkv][cap][64 or 8]
};

struct Kv4AppendArgs {
  Kv4Planes p;                  // one layer
  int b, Hkv, cap, n;
  const df_bf16 *k, *v;         // [b][n][Hkv][128]
  const int32_t *n_new, *cache_len;
  df_bf16 *k_held, *v_held;     // may be null
  int k_exp, v_exp;
  int* status;
};
int launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st);

struct Kv4AttnArgs {
  Kv4Planes p;                  // one layer
  int b, T, Hq, Hkv, cap;
  const df_bf16* q;             // [b][T][Hq][128]
  const int32_t* cache_len;
  const uint32_t* anc;          // [b][T][ceil(T/32)], or null: row i sees tree slots 0 .. i
  float scale;
  int k_exp, v_exp;
  df_bf16* out;                 // [b][T][Hq][128]
  float* lse;                   // [b][T][Hq], may be null
  void* scratch;                // kv4_attn_scratch_bytes
  int* status;
};
size_t kv4_attn_scratch_bytes(int b, int T, int Hq, int Hkv);
int launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t st);

struct Kv4WeightsArgs {
  Kv4Planes p;                  // one layer (keys only)
  int b, T, Hq, Hkv, cap;
  const df_bf16* q;             // [b][T][Hq][128]
  const float* lse;             // [b][T][Hq]
  const int32_t *cache_len, *n_rows, *src_slot;
  int max_src;
  float scale, decay;
  int k_exp;
  const float* score;           // [b][Hkv][cap] of the layer
  float* score_out;
  int* status;
};
int launch_kv4_weights(const Kv4WeightsArgs& a, cudaStream_t st);

struct Kv4CompactArgs {
  Kv4Planes p;                  // all layers
  int n_layers, b, Hkv, cap;
  const int32_t *src_slot, *n_acc, *cache_len;
  int max_src;
  int* status;
};
int launch_kv4_compact(const Kv4CompactArgs& a, cudaStream_t st);

struct Kv4EvictArgs {
  Kv4Planes src, dst;           // all layers
  int n_layers, b, Hkv, cap, dst_cap;
  const float* score;           // [n_layers][b][Hkv][cap]
  const int32_t* cache_len;
  int budget, n_sink, n_recent;
  float* score_out;             // [n_layers][b][Hkv][dst_cap], may be null
  int32_t* new_len;             // [b]
  int32_t* kept;                // [n_layers][b][Hkv][budget]
  int* status;
};
int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t st);

}  // namespace df
