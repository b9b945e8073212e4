// C ABI entry points of the 4-bit KV cache (include/dflash.h): argument checks and workspaces.
#include <cmath>

#include "common.cuh"
#include "kv4.h"
#include "nvtx.h"
#include "workspace.h"

namespace df {
namespace {

constexpr long long kGridLimit = 2147483647LL;   // blocks of a grid's x

int cache_ok(const df_kv4_cache* c) {
  if (!c || c->n_layers < 1 || c->b < 0 || c->Hkv < 1 || c->cap < 1) return DF_ERR_ARG;
  if (c->k_exp < -32 || c->k_exp > 32 || c->v_exp < -32 || c->v_exp > 32) return DF_ERR_ARG;
  if (c->hd != 128 || c->cap % 8) return DF_ERR_SHAPE;
  if (c->b == 0) return DF_OK;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return DF_ERR_ARG;
  if (!al16(c->k_codes) || !al16(c->k_scales) || !al16(c->v_codes) || !al16(c->v_scales)) return DF_ERR_ALIGN;
  return DF_OK;
}

size_t layer_rows(const df_kv4_cache* c) { return (size_t)c->b * c->Hkv * c->cap; }

Kv4Planes planes(const df_kv4_cache* c, int layer) {
  const size_t r = layer_rows(c) * layer;
  return Kv4Planes{c->k_codes + r * kKv4Codes, c->k_scales + r * kKv4Scales, c->v_codes + r * kKv4Codes,
                   c->v_scales + r * kKv4Scales};
}

bool apart(const void* x, size_t nx, const void* y, size_t ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a + nx <= b || b + ny <= a;
}

// Every array of one cache apart from every array of the other.
bool caches_apart(const df_kv4_cache* x, const df_kv4_cache* y) {
  const size_t nx = layer_rows(x) * x->n_layers, ny = layer_rows(y) * y->n_layers;
  const void* xp[] = {x->k_codes, x->v_codes, x->k_scales, x->v_scales};
  const void* yp[] = {y->k_codes, y->v_codes, y->k_scales, y->v_scales};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (!apart(xp[i], nx * (i < 2 ? kKv4Codes : kKv4Scales), yp[j], ny * (j < 2 ? kKv4Codes : kKv4Scales))) return false;
  return true;
}

// A softmax scale that stays a number when the keys' exponent goes into it.
bool scale_ok(float scale, int k_exp) {
  const float x = std::ldexp(scale * 1.4426950408889634f, k_exp);
  return scale > 0.f && std::isnormal(x);
}

}  // namespace
}  // namespace df

using namespace df;

extern "C" {

size_t dflash_kv4_append_workspace_size(void) { return kAlign; }

int dflash_kv4_append(const df_kv4_cache* c, int layer, const df_bf16* k, const df_bf16* v, int n,
                      const int32_t* n_new, const int32_t* cache_len, df_bf16* k_held, df_bf16* v_held, void* ws,
                      size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_kv4_append");
  DF_TRY(cache_ok(c));
  if (layer < 0 || layer >= c->n_layers || n < 0 || (k_held == nullptr) != (v_held == nullptr)) return DF_ERR_ARG;
  if (c->b == 0 || n == 0) return DF_OK;
  if (!k || !v || !cache_len) return DF_ERR_ARG;
  if (!al16(k) || !al16(v) || (k_held && (!al16(k_held) || !al16(v_held)))) return DF_ERR_ALIGN;
  if ((long long)c->b * c->Hkv * ((n + 63) / 64) > kGridLimit) return DF_ERR_SHAPE;
  if (!ws || ws_bytes < dflash_kv4_append_workspace_size()) return DF_ERR_WORKSPACE;
  Kv4AppendArgs a{};
  a.p = planes(c, layer); a.b = c->b; a.Hkv = c->Hkv; a.cap = c->cap; a.n = n;
  a.k = k; a.v = v; a.n_new = n_new; a.cache_len = cache_len; a.k_held = k_held; a.v_held = v_held;
  a.k_exp = c->k_exp; a.v_exp = c->v_exp; a.status = status_of(ws);
  return launch_kv4_append(a, (cudaStream_t)stream);
}

size_t dflash_kv4_attention_workspace_size(const df_kv4_cache* c, int n_tree, int Hq) {
  if (!c || c->b < 1 || c->Hkv < 1 || n_tree < 1 || Hq < 1 || Hq % c->Hkv) return kAlign;
  Carver cv(nullptr);
  cv.take<unsigned char>(kv4_attn_scratch_bytes(c->b, n_tree, Hq, c->Hkv));
  return cv.off;
}

int dflash_kv4_attention(const df_kv4_cache* c, int layer, int n_tree, int Hq, const df_bf16* q,
                         const int32_t* cache_len, const uint32_t* anc, float scale, df_bf16* out, float* lse,
                         void* ws, size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_kv4_attention");
  DF_TRY(cache_ok(c));
  if (layer < 0 || layer >= c->n_layers || n_tree < 1 || Hq < 1 || Hq % c->Hkv || !scale_ok(scale, c->k_exp))
    return DF_ERR_ARG;
  if (c->b == 0) return DF_OK;
  if (!q || !cache_len || !out) return DF_ERR_ARG;
  if (!al16(q) || !al16(out) || (anc && !al16(anc))) return DF_ERR_ALIGN;
  // 32-bit row numbers, and stages (of 32 slots and a tile of rows) of the whole call
  if (c->cap > 1 << 20 || Hq / c->Hkv > 4096 || (long long)n_tree * Hq > (1 << 30) || (long long)c->b * (((long long)n_tree * Hq + 7) / 8) > kGridLimit ||
      (double)c->b * c->Hkv * (c->cap / 32 + 2) * ((double)n_tree * (Hq / c->Hkv) / 256 + 1) > 1e9)
    return DF_ERR_SHAPE;
  if (!ws || ws_bytes < dflash_kv4_attention_workspace_size(c, n_tree, Hq)) return DF_ERR_WORKSPACE;
  Carver cv(ws);
  Kv4AttnArgs a{};
  a.p = planes(c, layer); a.b = c->b; a.T = n_tree; a.Hq = Hq; a.Hkv = c->Hkv; a.cap = c->cap;
  a.q = q; a.cache_len = cache_len; a.anc = anc; a.scale = scale; a.k_exp = c->k_exp; a.v_exp = c->v_exp;
  a.out = out; a.lse = lse; a.status = status_of(ws);
  a.scratch = cv.take<unsigned char>(kv4_attn_scratch_bytes(c->b, n_tree, Hq, c->Hkv));
  return launch_kv4_attention(a, (cudaStream_t)stream);
}

size_t dflash_kv4_attention_weights_workspace_size(const df_kv4_cache* c, int n_tree, int Hq) {
  (void)c; (void)n_tree; (void)Hq;
  return kAlign;
}

int dflash_kv4_attention_weights(const df_kv4_cache* c, int layer, int n_tree, int Hq, const df_bf16* q,
                                 const float* lse, const int32_t* cache_len, const int32_t* n_rows,
                                 const int32_t* src_slot, int max_src, float scale, float decay, const float* score,
                                 float* score_out, void* ws, size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_kv4_attention_weights");
  DF_TRY(cache_ok(c));
  if (layer < 0 || layer >= c->n_layers || n_tree < 1 || Hq < 1 || Hq % c->Hkv || !scale_ok(scale, c->k_exp) ||
      !(decay >= 0.f && decay <= 1.f) || max_src < 0)
    return DF_ERR_ARG;
  if (c->b == 0) return DF_OK;
  if (!q || !lse || !cache_len || !score || !score_out) return DF_ERR_ARG;
  if (!al16(q) || !al16(score) || !al16(score_out)) return DF_ERR_ALIGN;
  if (c->cap > 1 << 20 || (long long)n_tree * Hq > (1 << 30) || (double)c->b * c->Hkv * (c->cap / 128 + 2) > 1e9) return DF_ERR_SHAPE;
  if (!ws || ws_bytes < dflash_kv4_attention_weights_workspace_size(c, n_tree, Hq)) return DF_ERR_WORKSPACE;
  Kv4WeightsArgs a{};
  a.p = planes(c, layer); a.b = c->b; a.T = n_tree; a.Hq = Hq; a.Hkv = c->Hkv; a.cap = c->cap;
  a.q = q; a.lse = lse; a.cache_len = cache_len; a.n_rows = n_rows; a.src_slot = src_slot; a.max_src = max_src;
  a.scale = scale; a.decay = decay; a.k_exp = c->k_exp;
  a.score = score + layer_rows(c) * layer; a.score_out = score_out + layer_rows(c) * layer;
  a.status = status_of(ws);
  return launch_kv4_weights(a, (cudaStream_t)stream);
}

size_t dflash_kv4_compact_workspace_size(void) { return kAlign; }

int dflash_kv4_compact(const df_kv4_cache* c, const int32_t* src_slot, int max_src, const int32_t* n_acc,
                       const int32_t* cache_len, void* ws, size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_kv4_compact");
  DF_TRY(cache_ok(c));
  if (max_src < 0) return DF_ERR_ARG;
  if (c->b == 0 || max_src == 0) return DF_OK;
  if (!src_slot || !n_acc || !cache_len) return DF_ERR_ARG;
  if ((long long)c->n_layers * c->b * c->Hkv > kGridLimit) return DF_ERR_SHAPE;
  if (!ws || ws_bytes < dflash_kv4_compact_workspace_size()) return DF_ERR_WORKSPACE;
  Kv4CompactArgs a{};
  a.p = planes(c, 0); a.n_layers = c->n_layers; a.b = c->b; a.Hkv = c->Hkv; a.cap = c->cap;
  a.src_slot = src_slot; a.n_acc = n_acc; a.cache_len = cache_len; a.max_src = max_src; a.status = status_of(ws);
  return launch_kv4_compact(a, (cudaStream_t)stream);
}

size_t dflash_kv4_evict_workspace_size(const df_kv4_cache* c, int budget) {
  (void)c; (void)budget;
  return kAlign;
}

int dflash_kv4_evict(const df_kv4_cache* c, const float* score, const int32_t* cache_len, int budget, int n_sink,
                     int n_recent, const df_kv4_cache* to, float* score_out, int32_t* new_len, int32_t* kept,
                     void* ws, size_t ws_bytes, df_stream stream) {
  DF_NVTX("dflash_kv4_evict");
  DF_TRY(cache_ok(c));
  DF_TRY(cache_ok(to));
  if (to->n_layers != c->n_layers || to->b != c->b || to->Hkv != c->Hkv || to->k_exp != c->k_exp ||
      to->v_exp != c->v_exp || budget < 1 || n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > budget)
    return DF_ERR_ARG;
  if (budget > to->cap) return DF_ERR_CAPACITY;
  if (c->b == 0) return DF_OK;
  if (!score || !cache_len || !new_len || !kept) return DF_ERR_ARG;
  if (!al16(score) || (score_out && !al16(score_out)) || !al16(kept)) return DF_ERR_ALIGN;
  const size_t planes_n = (size_t)c->n_layers * c->b * c->Hkv;
  if (!caches_apart(c, to) ||
      (score_out && !apart(score, planes_n * c->cap * 4, score_out, planes_n * to->cap * 4)))
    return DF_ERR_ARG;
  if (planes_n * ((budget + 63) / 64) > (size_t)kGridLimit) return DF_ERR_SHAPE;
  if (!ws || ws_bytes < dflash_kv4_evict_workspace_size(c, budget)) return DF_ERR_WORKSPACE;
  Kv4EvictArgs a{};
  a.src = planes(c, 0); a.dst = planes(to, 0);
  a.n_layers = c->n_layers; a.b = c->b; a.Hkv = c->Hkv; a.cap = c->cap; a.dst_cap = to->cap;
  a.score = score; a.cache_len = cache_len; a.budget = budget; a.n_sink = n_sink; a.n_recent = n_recent;
  a.score_out = score_out; a.new_len = new_len; a.kept = kept; a.status = status_of(ws);
  return launch_kv4_evict(a, (cudaStream_t)stream);
}

}  // extern "C"
