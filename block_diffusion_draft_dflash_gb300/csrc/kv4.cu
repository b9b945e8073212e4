// The 4-bit KV cache: rounding rows into it, moving an accepted path, evicting slots.
//
// A row (one slot of one kv head) is 64 bytes of e2m1 codes and 8 bytes of e4m3 scales.  The
// scale of 16 values whose largest magnitude is a is s = e4m3(a / (6 * 2^exp)) and a value's
// code e2m1(x / (s * 2^exp)), both rounded to nearest even and saturated.  The inputs are bf16
// (8 significant bits), the borders between codes have at most 7 after multiplication with s
// and the divisor 2^exp only shifts, so fp32 quotients that are exact at the borders give the
// codes that exact arithmetic gives.
#include <cuda_fp8.h>
#include <math.h>

#include "kv4.cuh"
#include "kv4.h"
#include "runtime.h"
#include "trace.h"

namespace df {

// ------------------------------------------------------------------------------ append
constexpr int kAppTokens = 64;   // tokens of one kv head per CTA: 8 warps x 4 pairs

// max(|a|, |b|) of two bf16 pairs; a NaN stays one.
DF_DEV uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}
DF_DEV uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
DF_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

DF_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
DF_DEV float reciprocal(float x) {   // within 2^-22
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// x / d with r = 1 / d but for a few last bits: one step of correction of x r, whose remainder
// the fma computes exactly.  A quotient of few bits, a border between two codes or scales, comes
// out exactly: the step brings it there but for 2^-40 of its value.
DF_DEV float divide(float x, float d, float r) {
  const float t = x * r;
  return fmaf(fmaf(t, -d, x), r, t);
}

// 16 lanes hold one row (8 values each, 16-byte loads); the two lanes of a block of 16 agree
// on its scale with one shuffle.  A CTA takes consecutive tokens of one head, so that its
// code and scale stores fill whole sectors of the cache.  Bound by its bytes: 4 x 4096 tokens
// of 8 heads (153 MB with the held values) in 25 us.
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4AppendArgs a, float k_up, float v_up) {
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
  const float up = is_v ? v_up : k_up, limit = 4096.f * up;   // 2^exp; beyond 448 * 6 * 2^exp all saturate
  const float six = 6.f * up, six_r = reciprocal(six);
  uint8_t* codes = is_v ? a.p.vc : a.p.kc;
  uint8_t* scales = is_v ? a.p.vs : a.p.ks;
  const int j0 = chunk * kAppTokens + warp * 8 + (lane >> 4);
  const df_bf16* src = in + (((size_t)s * a.n + j0) * a.Hkv + h) * 128 + sub * 8;
  const size_t step = (size_t)2 * a.Hkv * 128;
  const size_t row0 = ((size_t)s * a.Hkv + h) * a.cap + len + j0;
  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (j0 + 2 * i < nn) raw[i] = *reinterpret_cast<const uint4*>(src + i * step);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    const uint32_t m2 = absmax2(absmax2(w[0], w[1]), absmax2(w[2], w[3]));
    float amax = max_nan(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xFFFF0000u));
    if (__any_sync(0xffffffffu, !(amax <= limit))) {   // rare: a NaN, or beyond the scales' range
      if (amax != amax) set_status(a.status, DF_ERR_NAN, s);
      amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = x[e] == x[e] ? fminf(fmaxf(x[e], -limit), limit) : 0.f;   // a NaN is stored as 0
        amax = fmaxf(amax, fabsf(x[e]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const __nv_fp8_storage_t sb = __nv_cvt_float_to_fp8(divide(amax, six, six_r), __NV_SATFINITE, __NV_E4M3);
    const float sc = e4m3_to_f(sb) * up;   // the block's scale with 2^exp
    uint32_t code = 0;
    const uint64_t z2 = pack_f32x2(-0.f, -0.f), sc2 = pack_f32x2(sc, sc);
    if (sc > 0.f) {
      const float r = reciprocal(sc);   // then as divide() does
      const uint64_t r2 = pack_f32x2(r, r), n2 = pack_f32x2(-sc, -sc);
      float q[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t v = pack_f32x2(x[2 * e], x[2 * e + 1]);
        const uint64_t t = fma_f32x2(v, r2, z2);
        const uint64_t y = fma_f32x2(fma_f32x2(t, n2, v), r2, t);
        asm("mov.b64 {%0, %1}, %2;" : "=f"(q[2 * e]), "=f"(q[2 * e + 1]) : "l"(y));
      }
      asm("{\n .reg .b8 a, b, c, d;\n"
          " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
          " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
          " mov.b32 %0, {a, b, c, d};\n}"
          : "=r"(code)
          : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    }
    if (j0 + 2 * i < nn) {
      const size_t row = row0 + 2 * i;
      *reinterpret_cast<uint32_t*>(codes + row * kKv4Codes + sub * 4) = code;
      if ((sub & 1) == 0) scales[row * kKv4Scales + (sub >> 1)] = sb;
      if (held) {
        uint32_t f[4], o[4];
        e2m1x8_to_f16(code, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f[e]));
          const uint64_t y = fma_f32x2(pack_f32x2(v.x, v.y), sc2, z2);   // six significant bits: exact
          float lo, hi;
          asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(y));
          o[e] = pack_bf16x2(lo, hi);
        }
        *reinterpret_cast<uint4*>(held + (src - in) + i * step) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

int launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
  DF_TRACE("kv4_append", st);
  const int chunks = (a.n + kAppTokens - 1) / kAppTokens;
  launch_k(kv4_append_kernel, dim3((unsigned)(a.b * a.Hkv * chunks), 2), dim3(256), 0, st, a, ldexpf(1.f, a.k_exp),
           ldexpf(1.f, a.v_exp));
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

// 16 bytes of a row's 64 codes.  Rows are picked here and there: without the hint L2 fetches the
// neighbouring row with each (half of 36 x 8 x 8449 rows kept: 277 MB read instead of 204, 65 us
// instead of 54).
DF_DEV uint4 load_picked(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
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
        k[i] = load_picked(kc + at);
        v[i] = load_picked(vc + at);
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
constexpr int kSelThreads = 512;
constexpr int kSelHeld = 49152;   // keys held in shared memory; a longer row's are made anew in every step

// Order of slots for eviction: larger is kept first.  The first n_sink and the last n_recent
// slots stand above every score; a NaN stands below.
DF_DEV uint32_t evict_key(float score, int slot, int lo, int hi) {
  if (slot < lo || slot >= hi) return 0xFFFFFFFFu;
  return score == score ? float_key(score + 0.f) : 0u;   // + 0: one zero
}

// One CTA per (layer, sequence, kv head): the key of the last kept slot, two bits a step (the
// largest key that `budget` slots reach), then the kept slots in order, the lowest slots first
// among equal keys.  What bounds it is the comparisons, three of every key in a step, so the steps
// begin behind the bits that the smallest and the largest score share, and once the bracket holds
// kSelFew keys at most every warp goes on by itself with a list of those. 288 rows of 8449 scores
// take 23 us, 25 us with all 16 steps over whole rows, and more with a histogram of digits: 52 us
// with atomic counters, 47 us with counters in registers.  Every count is a whole number: no order
// of additions, and no order in that list, changes the choice.
constexpr int kSelFew = 256;   // eight keys a lane
__global__ void __launch_bounds__(kSelThreads, 2) kv4_select_kernel(const Kv4EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kSelWarps = kSelThreads / 32;
  __shared__ __align__(16) int4 sums[2][kSelWarps];
  __shared__ int2 counts[kSelWarps];
  __shared__ uint32_t least[kSelWarps], most[kSelWarps];
  __shared__ __align__(16) uint32_t few[kSelFew];
  __shared__ int n_few;
  const size_t plane = blockIdx.x;
  const int s = (int)((plane / a.Hkv) % a.b);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.cache_len[s];
  if (len < 0 || len > a.cap) {
    if (tid == 0) set_status(a.status, DF_ERR_CAPACITY, s);
    len = 0;
  }
  const float* score = a.score + plane * a.cap;
  int32_t* kept = a.kept + plane * a.budget;
  if (len <= a.budget) {
    for (int j = tid; j < a.budget; j += kSelThreads) kept[j] = j < len ? j : -1;
    return;
  }
  const int lo = a.n_sink, hi = len - a.n_recent;   // the slots between are chosen by score
  if (tid == 0) n_few = 0;
  if (tid < kSelFew) few[tid] = 0u;
  extern __shared__ __align__(16) uint32_t keys[];
  const bool held = len <= kSelHeld;
  auto key_at = [&](int i) { return held ? keys[i] : i < len ? evict_key(score[i], i, lo, hi) : 0u; };
  uint32_t k_min = 0xFFFFFFFFu, k_max = 0u;
  auto see = [&](uint32_t k, int i) {
    if (i >= lo && i < hi) {
      k_min = min(k_min, k);
      k_max = max(k_max, k);
    }
  };
  if (held) {   // a row of scores is 16-byte aligned and as long as cap, a multiple of 8
#pragma unroll 4
    for (int i = tid; i < (len + 3) / 4; i += kSelThreads) {
      const float4 v = reinterpret_cast<const float4*>(score)[i];
      const int at = 4 * i;
      const uint4 k = make_uint4(evict_key(v.x, at, lo, hi), at + 1 < len ? evict_key(v.y, at + 1, lo, hi) : 0u,
                                 at + 2 < len ? evict_key(v.z, at + 2, lo, hi) : 0u, at + 3 < len ? evict_key(v.w, at + 3, lo, hi) : 0u);
      see(k.x, at); see(k.y, at + 1); see(k.z, at + 2); see(k.w, at + 3);
      reinterpret_cast<uint4*>(keys)[i] = k;
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < len; i += kSelThreads) see(evict_key(score[i], i, lo, hi), i);
  }
  __syncwarp();
  k_min = __reduce_min_sync(0xffffffffu, k_min);
  k_max = __reduce_max_sync(0xffffffffu, k_max);
  if (lane == 0) { least[warp] = k_min; most[warp] = k_max; }
  __syncthreads();
  k_min = __reduce_min_sync(0xffffffffu, least[lane % kSelWarps]);
  k_max = __reduce_max_sync(0xffffffffu, most[lane % kSelWarps]);
  // slots of the row whose key is at least k[0], k[1], k[2] > 0
  auto reach = [&](const uint32_t (&k)[3], int step, int (&n)[3]) {
    int c[3] = {0, 0, 0};
    if (held) {
#pragma unroll 2
      for (int i = tid; i < (len + 3) / 4; i += kSelThreads) {
        const uint4 v = reinterpret_cast<const uint4*>(keys)[i];
#pragma unroll
        for (int x = 0; x < 3; ++x)
          c[x] += (v.x >= k[x] ? 1 : 0) + (v.y >= k[x] ? 1 : 0) + (v.z >= k[x] ? 1 : 0) + (v.w >= k[x] ? 1 : 0);
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < len; i += kSelThreads) {
        const uint32_t v = evict_key(score[i], i, lo, hi);
#pragma unroll
        for (int x = 0; x < 3; ++x) c[x] += v >= k[x] ? 1 : 0;
      }
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 3; ++x) c[x] = __reduce_add_sync(0xffffffffu, c[x]);
    if (lane == 0) sums[step & 1][warp] = make_int4(c[0], c[1], c[2], 0);
    __syncthreads();
    const int4 all = lane < kSelWarps ? sums[step & 1][lane] : make_int4(0, 0, 0, 0);
    n[0] = __reduce_add_sync(0xffffffffu, all.x);
    n[1] = __reduce_add_sync(0xffffffffu, all.y);
    n[2] = __reduce_add_sync(0xffffffffu, all.z);
  };
  // The bracket: keys from prefix on with the bits above `shift + 1` the same.  It holds the last
  // kept key; `above` slots lie behind it, `inside` in it.
  const uint32_t differ = k_min ^ k_max;
  int above = lo + len - hi, inside = hi - lo;   // not kept by score: keys above all others
  uint32_t prefix = 0xFFFFFFFFu;
  bool exact = above >= a.budget;                // `budget` slots have at least the key prefix
  int shift = -2;
  if (!exact) {
    shift = differ ? (31 - __clz(differ)) & ~1 : -2;
    prefix = shift == 30 ? 0u : k_min >> (shift + 2) << (shift + 2);
  }
  // Keys that reach prefix plus 1, 2 and 3 times 2^shift are counted: the bracket shrinks to a quarter.
  auto narrow = [&](const int (&n)[3]) {
    const int d = (n[0] >= a.budget ? 1 : 0) + (n[1] >= a.budget ? 1 : 0) + (n[2] >= a.budget ? 1 : 0);
    prefix |= (uint32_t)d << shift;
    const int reached = d == 0 ? above + inside : d == 1 ? n[0] : d == 2 ? n[1] : n[2];
    above = d == 0 ? n[0] : d == 1 ? n[1] : d == 2 ? n[2] : above;
    inside = reached - above;
    exact = reached == a.budget;
    shift -= 2;
  };
#pragma unroll 1
  for (int step = 0; shift >= 0 && !exact && inside > kSelFew; ++step) {
    const uint32_t k[3] = {prefix | 1u << shift, prefix | 2u << shift, prefix | 3u << shift};
    int n[3];
    reach(k, step, n);
    narrow(n);
  }
  if (shift >= 0 && !exact) {
    // the keys inside, in any order: a lane marks those among 32 of its own, a warp takes their places at once
    const int quads = (len + 3) / 4;
    for (int base = warp * 32; base < quads; base += 8 * kSelThreads) {
      uint32_t mine = 0u;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int at = base + x * kSelThreads + lane, i = 4 * at;
        if (at < quads) {
          const uint4 v = held ? reinterpret_cast<const uint4*>(keys)[at]
                               : make_uint4(key_at(i), key_at(i + 1), key_at(i + 2), key_at(i + 3));
          const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = shift == 30 || (k[e] ^ prefix) >> (shift + 2) == 0u;
            if (in && i + e >= lo && i + e < hi) mine |= 1u << (4 * x + e);
          }
        }
      }
      __syncwarp();
      const int n = __popc(mine);
      int at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += x;
      }
      int first = 0;
      if (lane == 31 && at > 0) first = atomicAdd(&n_few, at);
      at += __shfl_sync(0xffffffffu, first, 31) - n;
      for (; mine; mine &= mine - 1) {
        const int b = __ffs(mine) - 1;
        few[at++] = key_at(4 * (base + (b >> 2) * kSelThreads + lane) + (b & 3));
      }
      __syncwarp();
    }
    __syncthreads();
    uint32_t k8[kSelFew / 32];
#pragma unroll
    for (int x = 0; x < kSelFew / 32; ++x) k8[x] = few[x * 32 + lane];
    const int listed_above = above;
#pragma unroll 1
    while (shift >= 0 && !exact) {
      int n[3];
#pragma unroll
      for (int y = 0; y < 3; ++y) {
        const uint32_t k = prefix | (uint32_t)(y + 1) << shift;
        n[y] = 0;
#pragma unroll
        for (int x = 0; x < kSelFew / 32; ++x) n[y] += k8[x] >= k ? 1 : 0;
        n[y] = __reduce_add_sync(0xffffffffu, n[y]) + listed_above;
      }
      narrow(n);
    }
  }
  const int want = a.budget - above;   // where it is not exact: of the slots whose key equals prefix
  // kept: keys above prefix, and the first `want` slots whose key equals it.  A warp takes a
  // piece of the row: it counts both kinds, then, knowing the counts before it, writes its part.
  const int piece = ((len + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int p0 = min(len, warp * piece), p1 = min(len, p0 + piece);
  const uint32_t below = (1u << lane) - 1u;
  const uint32_t over = exact ? prefix - 1u : prefix;   // kept whatever its slot: a key above this (exact: prefix > 0)
  int g = 0, e = 0;
#pragma unroll 4
  for (int i = p0 + lane; i < p1; i += 32) {
    const uint32_t k = key_at(i);
    g += k > over ? 1 : 0;
    e += k == over ? 1 : 0;
  }
  __syncwarp();
  g = __reduce_add_sync(0xffffffffu, g);
  e = __reduce_add_sync(0xffffffffu, e);
  if (lane == 0) counts[warp] = make_int2(g, e);
  __syncthreads();
  const int2 before = lane < warp ? counts[lane] : make_int2(0, 0);   // of the warps before this one
  g = __reduce_add_sync(0xffffffffu, before.x);
  e = __reduce_add_sync(0xffffffffu, before.y);
  if (exact) {
#pragma unroll 4
    for (int i0 = p0; i0 < p1; i0 += 32) {
      const int i = i0 + lane;
      const bool keep = i < p1 && key_at(i) > over;
      const uint32_t bits = __ballot_sync(0xffffffffu, keep);
      if (keep) kept[g + __popc(bits & below)] = i;
      g += __popc(bits);
    }
    return;
  }
#pragma unroll 2
  for (int i0 = p0; i0 < p1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < p1 ? key_at(i) : 0u;
    const bool gt = i < p1 && k > prefix, eq = i < p1 && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const int me = e + __popc(be & below);
    if (gt || (eq && me < want)) kept[g + __popc(bg & below) + min(me, want)] = i;
    g += __popc(bg);
    e += __popc(be);
  }
}

constexpr int kGatherRows = 64;

// Copies kept rows and their scores (36 layers x 8 heads x 4096 rows in 54 us: 339 MB read and
// written, 6.3 TB/s, the rate of a copy): a CTA moves kGatherRows rows of one plane, 16 bytes of keys' and values'
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
  const uint4 k = load_picked(a.src.kc + ci), v = load_picked(a.src.vc + ci);
  const uint8_t* sp = part < 2 ? a.src.ks : a.src.vs;
  uint8_t* dp = part < 2 ? a.dst.ks : a.dst.vs;
  const uint32_t sc = *reinterpret_cast<const uint32_t*>(sp + (from + i) * kKv4Scales + (part & 1) * 4);
  const bool scored = a.score_out && part == 0;
  const float w = scored ? a.score[from + i] : 0.f;   // every load before the first store
  *reinterpret_cast<uint4*>(a.dst.kc + co) = k;
  *reinterpret_cast<uint4*>(a.dst.vc + co) = v;
  *reinterpret_cast<uint32_t*>(dp + (to + j) * kKv4Scales + (part & 1) * 4) = sc;
  if (scored) a.score_out[to + j] = w;
}

int launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t st) {
  const long long planes = (long long)a.n_layers * a.b * a.Hkv;
  {
    DF_TRACE("kv4_select", st);
    const size_t smem = (size_t)(a.cap < kSelHeld ? a.cap : kSelHeld) * 4;
    if (ensure_dynamic_smem(kv4_select_kernel, smem) != cudaSuccess) return DF_ERR_CUDA;
    launch_k(kv4_select_kernel, dim3((unsigned)planes), dim3(kSelThreads), smem, st, a);
  }
  DF_TRACE("kv4_gather", st);
  const int chunks = (a.budget + kGatherRows - 1) / kGatherRows;
  launch_k(kv4_gather_kernel, dim3((unsigned)(planes * chunks)), dim3(256), 0, st, a, chunks);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
