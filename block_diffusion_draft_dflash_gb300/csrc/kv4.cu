// The 4-bit KV cache: rounding rows into it, moving an accepted path, evicting slots.
//
// A row (one slot of one kv head) is 64 bytes of e2m1 codes and 8 bytes of e4m3 scales.  The
// scale of 16 values whose largest magnitude is a is s = e4m3(a / (6 * 2^exp)) and a value's
// code e2m1(x / (s * 2^exp)), both rounded to nearest even and saturated.  The inputs are bf16
// (8 significant bits), the borders between codes have at most 7 after multiplication with s
// and the divisor 2^exp only shifts, so fp32 quotients that are correctly rounded at the
// borders give the codes that exact arithmetic gives.
#include <cuda_fp8.h>
#include <math.h>

#include "kv4.cuh"
#include "kv4.h"
#include "trace.h"

namespace df {

// ------------------------------------------------------------------------------ append
constexpr int kAppTokens = 64;   // tokens of one kv head per CTA: 8 warps x 4 pairs

// 16 lanes hold one row (8 values each, 16-byte loads); the two lanes of a block of 16 agree
// on its scale with one shuffle.  A CTA takes consecutive tokens of one head, so that its
// code and scale stores fill whole sectors of the cache.
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4AppendArgs a, float k_down, float v_down) {
  pdl_wait();
  pdl_trigger();
  const int chunks = (a.n + kAppTokens - 1) / kAppTokens;
  int u = blockIdx.x;
  const int chunk = u % chunks; u /= chunks;
  const int h = u % a.Hkv, s = u / a.Hkv;
  const bool is_v = blockIdx.y == 1;
  const int nn = a.n_new ? a.n_new[s] : a.n;
  if (nn < 0 || nn > a.n) {
    set_status(a.status, DF_ERR_ARG, s);
    return;
  }
  const int len = kv4_len(a.cache_len, s, nn, a.cap, a.status);
  if (len < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 15;
  const df_bf16* in = is_v ? a.v : a.k;
  df_bf16* held = is_v ? a.v_held : a.k_held;
  const float down = is_v ? v_down : k_down, up = 1.f / down;   // 2^-exp, 2^exp
  uint8_t* codes = is_v ? a.p.vc : a.p.kc;
  uint8_t* scales = is_v ? a.p.vs : a.p.ks;
  const size_t plane = ((size_t)s * a.Hkv + h) * a.cap;
  const int j0 = chunk * kAppTokens + warp * 8 + (lane >> 4);
  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 2 * i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (j < nn) raw[i] = *reinterpret_cast<const uint4*>(in + (((size_t)s * a.n + j) * a.Hkv + h) * 128 + sub * 8);
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 2 * i;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[8], amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
      if (v != v) { bad = true; v = 0.f; }               // recorded, and stored as 0
      v *= down;
      x[e] = fminf(fmaxf(v, -4096.f), 4096.f);           // beyond 448 * 6 both saturate
      amax = fmaxf(amax, fabsf(x[e]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const __nv_fp8_storage_t sb = __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f), __NV_SATFINITE, __NV_E4M3);
    const float sc = e4m3_to_f(sb);
    uint32_t code = 0;
    if (sc > 0.f) {
      // x / s to the nearest fp32 number: one step of correction of x * (1 / s), whose
      // remainder the fma computes exactly
      const float r = __frcp_rn(sc);
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = x[e] * r;
        q[e] = fmaf(fmaf(-t, sc, x[e]), r, t);
      }
      asm("{\n .reg .b8 a, b, c, d;\n"
          " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
          " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
          " mov.b32 %0, {a, b, c, d};\n}"
          : "=r"(code)
          : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    }
    if (j < nn) {
      const size_t row = plane + len + j;
      *reinterpret_cast<uint32_t*>(codes + row * kKv4Codes + sub * 4) = code;
      if ((sub & 1) == 0) scales[row * kKv4Scales + (sub >> 1)] = sb;
      if (held) {
        uint32_t f[4], o[4];
        e2m1x8_to_f16(code, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f[e]));
          o[e] = pack_bf16x2(v.x * sc * up, v.y * sc * up);   // six significant bits: exact
        }
        *reinterpret_cast<uint4*>(held + (((size_t)s * a.n + j) * a.Hkv + h) * 128 + sub * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (bad) set_status(a.status, DF_ERR_NAN, s);
}

int launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
  DF_TRACE("kv4_append", st);
  const int chunks = (a.n + kAppTokens - 1) / kAppTokens;
  launch_k(kv4_append_kernel, dim3((unsigned)(a.b * a.Hkv * chunks), 2), dim3(256), 0, st, a, ldexpf(1.f, -a.k_exp),
           ldexpf(1.f, -a.v_exp));
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

// ----------------------------------------------------------------------------- compact
constexpr int kCmpRows = 32;   // rows of one round: a path of accept_and_compact fits one

// One warp per (layer, sequence, kv head).  Sources ascend and lie at or behind their
// destinations, so a round's stores touch no later round's source; inside a round every
// load precedes every store.
__global__ void __launch_bounds__(256) kv4_compact_kernel(const Kv4CompactArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long plane = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (plane >= (long long)a.n_layers * a.b * a.Hkv) return;
  const int s = (int)((plane / a.Hkv) % a.b);
  const int n = a.n_acc[s], len = a.cache_len[s];
  const int32_t* src = a.src_slot + (size_t)s * a.max_src;
  const int dst0 = len - n;
  bool ok = n >= 0 && n <= a.max_src && dst0 >= 0 && len <= a.cap;
  int last = -1;
  for (int r0 = 0; ok && r0 < n; r0 += kCmpRows) {   // the whole list is looked at before anything moves
    const int j = r0 + lane;
    const int mine = j < n ? src[j] : a.cap;
    int prev = __shfl_up_sync(0xffffffffu, mine, 1);
    if (lane == 0) prev = last;
    ok = __all_sync(0xffffffffu, j >= n || (mine > prev && mine >= dst0 + j && mine < a.cap));
    last = __shfl_sync(0xffffffffu, mine, 31);
  }
  if (!ok) {
    if (lane == 0) set_status(a.status, DF_ERR_ARG, s);
    return;
  }
  uint8_t* kc = a.p.kc + plane * a.cap * kKv4Codes;
  uint8_t* vc = a.p.vc + plane * a.cap * kKv4Codes;
  uint8_t* ks = a.p.ks + plane * a.cap * kKv4Scales;
  uint8_t* vs = a.p.vs + plane * a.cap * kKv4Scales;
  for (int r0 = 0; r0 < n; r0 += kCmpRows) {
    const int mine = r0 + lane < n ? src[r0 + lane] : 0;
    uint4 k[4], v[4];
    uint2 ksc = make_uint2(0u, 0u), vsc = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 8 + (lane >> 2);
      const size_t at = (size_t)__shfl_sync(0xffffffffu, mine, row) * kKv4Codes + (lane & 3) * 16;
      if (r0 + row < n) {
        k[i] = *reinterpret_cast<const uint4*>(kc + at);
        v[i] = *reinterpret_cast<const uint4*>(vc + at);
      }
    }
    if (r0 + lane < n) {
      ksc = *reinterpret_cast<const uint2*>(ks + (size_t)mine * kKv4Scales);
      vsc = *reinterpret_cast<const uint2*>(vs + (size_t)mine * kKv4Scales);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 8 + (lane >> 2);
      const size_t at = (size_t)(dst0 + r0 + row) * kKv4Codes + (lane & 3) * 16;
      if (r0 + row < n) {
        *reinterpret_cast<uint4*>(kc + at) = k[i];
        *reinterpret_cast<uint4*>(vc + at) = v[i];
      }
    }
    if (r0 + lane < n) {
      *reinterpret_cast<uint2*>(ks + (size_t)(dst0 + r0 + lane) * kKv4Scales) = ksc;
      *reinterpret_cast<uint2*>(vs + (size_t)(dst0 + r0 + lane) * kKv4Scales) = vsc;
    }
    __syncwarp();
  }
}

int launch_kv4_compact(const Kv4CompactArgs& a, cudaStream_t st) {
  DF_TRACE("kv4_compact", st);
  const long long planes = (long long)a.n_layers * a.b * a.Hkv;
  launch_k(kv4_compact_kernel, dim3((unsigned)((planes + 7) / 8)), dim3(256), 0, st, a);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

// ------------------------------------------------------------------------------- evict
constexpr int kSelThreads = 1024;

// Order of slots for eviction: larger is kept first.  The first n_sink and the last n_recent
// slots stand above every score; a NaN stands below.
DF_DEV uint32_t evict_key(float score, int slot, int lo, int hi) {
  if (slot < lo || slot >= hi) return 0xFFFFFFFFu;
  return score == score ? float_key(score + 0.f) : 0u;   // + 0: one zero
}

// One CTA per (layer, sequence, kv head): the key of the last kept slot by radix selection
// (four digits of 8 bits), then the kept slots in order, the lowest slots first among equal
// keys.  Every count is a whole number: no order of additions changes the choice.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int hist[256];
  __shared__ int sh_bin, sh_want;
  __shared__ int warp_gt[32], warp_eq[32];
  const size_t plane = blockIdx.x;
  const int s = (int)((plane / a.Hkv) % a.b);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.cache_len[s];
  if (len < 0 || len > a.cap) {
    if (tid == 0) set_status(a.status, DF_ERR_CAPACITY, s);
    len = 0;
  }
  const float* score = a.score + plane * a.cap;
  float* score_out = a.score_out ? a.score_out + plane * a.dst_cap : nullptr;
  int32_t* kept = a.kept + plane * a.budget;
  if (len <= a.budget) {
    for (int j = tid; j < a.budget; j += kSelThreads) {
      kept[j] = j < len ? j : -1;
      if (score_out && j < len) score_out[j] = score[j];
    }
    return;
  }
  const int lo = a.n_sink, hi = len - a.n_recent;
  uint32_t prefix = 0;
  int want = a.budget;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t key = evict_key(score[i], i, lo, hi);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {   // lane l: bins 8l .. 8l+7; the bin that holds the want-th largest key
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) { c[e] = hist[lane * 8 + e]; sum += c[e]; }
      int above = sum;   // inclusive sum over lanes from the top
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += t;
      }
      above -= sum;
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        if (above < want && want <= above + c[e]) { sh_bin = lane * 8 + e; sh_want = want - above; }
        above += c[e];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh_bin << shift;
    want = sh_want;
  }
  // kept: keys above prefix, and the first `want` slots whose key equals it
  int run_gt = 0, run_eq = 0;
  for (int i0 = 0; i0 < len; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float sc = i < len ? score[i] : 0.f;
    const uint32_t key = i < len ? evict_key(sc, i, lo, hi) : 0u;
    const bool gt = i < len && key > prefix, eq = i < len && key == prefix;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) { warp_gt[warp] = __popc(bg); warp_eq[warp] = __popc(be); }
    __syncthreads();
    int g = run_gt + __popc(bg & below), e = run_eq + __popc(be & below);
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      if (w < warp) { g += warp_gt[w]; e += warp_eq[w]; }
      run_gt += warp_gt[w];
      run_eq += warp_eq[w];
    }
    if (gt || (eq && e < want)) {
      const int j = g + min(e, want);
      kept[j] = i;
      if (score_out) score_out[j] = sc;
    }
  }
}

constexpr int kGatherRows = 64;

// Copies kept rows: a CTA moves kGatherRows rows of one plane, 16 bytes of keys' and values'
// codes per thread.  new_len is written here, after every CTA of the selection has read the
// lengths, so it may be the same array.
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4EvictArgs a, int chunks) {
  pdl_wait();
  pdl_trigger();
  const size_t plane = blockIdx.x / chunks;
  const int j0 = (int)(blockIdx.x % chunks) * kGatherRows;
  const int tid = threadIdx.x;
  const int32_t* kept = a.kept + plane * a.budget;
  if (j0 == 0 && plane % a.Hkv == 0 && plane < (size_t)a.b * a.Hkv && tid == 0) {
    // the list holds -1 behind its last slot: its length by bisection
    int lo = 0, hi = a.budget;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (kept[mid] >= 0) lo = mid + 1; else hi = mid;
    }
    a.new_len[plane / a.Hkv] = lo;
  }
  const size_t from = plane * a.cap, to = plane * a.dst_cap;
  const int j = j0 + (tid >> 2), part = tid & 3;
  const int i = j < a.budget ? kept[j] : -1;
  if (i < 0) return;
  const size_t ci = (from + i) * kKv4Codes + part * 16, co = (to + j) * kKv4Codes + part * 16;
  const uint4 k = *reinterpret_cast<const uint4*>(a.src.kc + ci), v = *reinterpret_cast<const uint4*>(a.src.vc + ci);
  const uint8_t* sp = part < 2 ? a.src.ks : a.src.vs;
  uint8_t* dp = part < 2 ? a.dst.ks : a.dst.vs;
  const uint32_t sc = *reinterpret_cast<const uint32_t*>(sp + (from + i) * kKv4Scales + (part & 1) * 4);
  *reinterpret_cast<uint4*>(a.dst.kc + co) = k;
  *reinterpret_cast<uint4*>(a.dst.vc + co) = v;
  *reinterpret_cast<uint32_t*>(dp + (to + j) * kKv4Scales + (part & 1) * 4) = sc;
}

int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t st) {
  const long long planes = (long long)a.n_layers * a.b * a.Hkv;
  {
    DF_TRACE("kv4_select", st);
    launch_k(kv4_select_kernel, dim3((unsigned)planes), dim3(kSelThreads), 0, st, a);
  }
  DF_TRACE("kv4_gather", st);
  const int chunks = (a.budget + kGatherRows - 1) / kGatherRows;
  launch_k(kv4_gather_kernel, dim3((unsigned)(planes * chunks)), dim3(256), 0, st, a, chunks);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
