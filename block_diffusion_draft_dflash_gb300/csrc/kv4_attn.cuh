// What the two attention kernels over the 4-bit cache share: parameters, the cutting of the
// work into shares, the mask, and the form in which partial results reach the combine kernel.
//
// A unit is one (sequence, kv head, tile of R query rows); its keys come in stages.  All
// stages of a call lie in one line (sequence-major), which the CTAs cut into equal shares
// whatever the sequences' lengths.  A unit that lies inside one share is finished by its CTA;
// the parts of a cut unit go to slots that the combine kernel reads in the order of the CTAs.
#pragma once
#include "kv4.cuh"
#include "kv4.h"

#ifndef KV4_COLD
#define KV4_COLD static __device__ __noinline__   // rarely run: out of the way of the loops
#endif

namespace df {

struct Kv4AttnParams {
  Kv4Planes p;
  int b, T, Hq, Hkv, G, cap, W;
  uint32_t g_magic;      // ceil(2^32 / G): x / G = umulhi(x, g_magic) for x G < 2^32; 0 for G = 1
  const df_bf16* q;
  const int32_t* cache_len;
  const uint32_t* anc;
  float scale2;          // scale * log2(e) * 2^k_exp
  float v_mul;           // 2^v_exp
  df_bf16* out;
  float* lse;
  int R, nrt;            // rows of a tile, tiles of a (sequence, kv head)
  bool last_single;      // kv4_single of the last tile
  int stage_log2;        // keys of a stage
  int min_stages;        // no share is smaller, while there are several
  int n_cta;
  float shift;           // probabilities carry 2^shift
  float* o_part;         // [n_cta + units][R][128]: slot CTA + unit
  float2* ml_part;       // [n_cta + units][R]: maximum in log2 units, sum
  int2* range;           // [units]: first and last CTA
  int* status;
};

// A tile of the tcgen05 kernel with at most half its rows (the last one, then): both halves work
// on the same rows, on every other block of keys, and its stages are twice as long.
DF_DEV bool kv4_single(const Kv4AttnParams& p, int rt) { return p.last_single && rt == p.nrt - 1; }

// Stages of `keys` slots; a tile that sees nothing has one.
DF_DEV int kv4_stages(const Kv4AttnParams& p, int keys, bool single) {
  const int shift = p.stage_log2 + (single ? 1 : 0);
  return max(1, (keys + (1 << shift) - 1) >> shift);
}
// Slots that a sequence shows (0 where its length does not fit), and a chain's tile of it.
DF_DEV int kv4_all(const Kv4AttnParams& p, int N) { return N >= 0 && N <= p.cap - p.T ? N + p.T : 0; }
DF_DEV int kv4_chain(const Kv4AttnParams& p, int N, int rt) {
  return kv4_all(p, N) ? N + min(p.T, ((rt + 1) * p.R - 1) / p.G + 1) : 0;
}
// Tiles of a sequence differ in length where a chain has several: a row sees no later node.
DF_DEV bool kv4_even(const Kv4AttnParams& p) { return p.anc || p.nrt == 1; }

DF_DEV int kv4_head_stages(const Kv4AttnParams& p, int s) {   // of one kv head
  const int N = p.cache_len[s];
  if (kv4_even(p)) {
    const int len = kv4_all(p, N);
    return (p.nrt - 1) * kv4_stages(p, len, false) + kv4_stages(p, len, p.last_single);
  }
  int n = 0;
#pragma unroll 1
  for (int rt = 0; rt < p.nrt; ++rt) n += kv4_stages(p, kv4_chain(p, N, rt), kv4_single(p, rt));
  return n;
}

struct Kv4Seg {        // the part of one unit that lies in a share
  int s, kvh, rt, unit;
  int tile0, count;    // stages [tile0, tile0 + count)
  int N, len;          // cache_len (0 where it does not fit), slots seen
  int first, last;     // holds the unit's first, last stage
  int single;          // kv4_single
};

// A CTA's walk through its share.  One warp of the CTA walks (code that a kernel runs once
// costs some 50 cycles an instruction) and hands the units out by shared memory.
struct Kv4Walk {
  int t, t1, end;      // next stage, end of the share, end of sequence s
  int s, head;         // stages of one kv head of s

  // By a whole warp, like next(); false: no share.
  DF_DEV bool init(const Kv4AttnParams& p, int cta, int lane) {
    int total = 0;     // all stages, then those of the sequences already passed
    bool found = false;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {   // one copy of the code: the sum, then the place in it
#pragma unroll 1
      for (int base = 0; base < p.b && !found; base += 32) {
        const int h = base + lane < p.b ? kv4_head_stages(p, base + lane) : 0;
        int inc = h * p.Hkv;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (pass == 1) {
          const int k = __popc(__ballot_sync(0xffffffffu, base + lane < p.b && total + inc <= t));   // sequences before t
          if (k < 32) {
            s = base + k;
            head = __shfl_sync(0xffffffffu, h, k);
            end = total + __shfl_sync(0xffffffffu, inc, k);
            found = true;
          }
        }
        total += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (pass == 0) {
        const int n = min((total + p.min_stages - 1) / p.min_stages, p.n_cta);
        if (cta >= n) return false;
        const int q = total / n, rest = total - q * n;   // the first `rest` shares have one more
        t = q * cta + min(cta, rest);
        t1 = t + q + (cta < rest ? 1 : 0);
        total = 0;
      }
    }
    return true;
  }

  DF_DEV bool next(const Kv4AttnParams& p, Kv4Seg& g) {
    if (t >= t1) return false;
    if (t == end) {
      head = kv4_head_stages(p, ++s);
      end += head * p.Hkv;
    }
    int rel = t - (end - head * p.Hkv), rt = 0;
    const int N = p.cache_len[s];
    g.kvh = rel / head;
    rel -= g.kvh * head;
    int len = kv4_all(p, N), per_unit;
    if (kv4_even(p)) {   // all tiles but the last have the same stages
      per_unit = kv4_stages(p, len, false);
      rt = min(rel / per_unit, p.nrt - 1);
      rel -= rt * per_unit;
      if (kv4_single(p, rt)) per_unit = kv4_stages(p, len, true);
    } else {
#pragma unroll 1
      for (;; ++rt) {
        len = kv4_chain(p, N, rt);
        per_unit = kv4_stages(p, len, kv4_single(p, rt));
        if (rel < per_unit) break;
        rel -= per_unit;
      }
    }
    g.s = s;
    g.rt = rt;
    g.unit = (s * p.Hkv + g.kvh) * p.nrt + rt;
    g.tile0 = rel;
    g.count = min(t1 - t, per_unit - rel);
    g.len = len;
    g.N = len > 0 ? N : 0;
    g.single = kv4_single(p, rt);
    g.first = rel == 0;
    g.last = rel + g.count == per_unit;
    t += g.count;
    return true;
  }
};

// 32 bits of a row's visibility for keys j0 .. j0+31.
KV4_COLD uint32_t kv4_see_bits(const uint32_t* anc, int W, int N, int j0, int node, int len) {
  const int n = N - j0;
  uint32_t bits = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;   // the cache
  if (anc) {
    const int t0 = -n;                                                   // tree slot of bit 0
    const int w = t0 >= 0 ? t0 >> 5 : -((31 - t0) >> 5), sh = t0 - 32 * w;
    const uint32_t lo = w >= 0 && w < W ? anc[w] : 0u;
    const uint32_t hi = sh && w + 1 >= 0 && w + 1 < W ? anc[w + 1] : 0u;
    bits |= sh ? (lo >> sh) | (hi << (32 - sh)) : lo;
  } else {
    const int m = N + node + 1 - j0;                                      // chain: keys below N + node + 1
    bits = m >= 32 ? 0xFFFFFFFFu : m <= 0 ? 0u : (1u << m) - 1u;
  }
  const int l = len - j0;
  return l >= 32 ? bits : l <= 0 ? 0u : bits & ((1u << l) - 1u);
}

// mbar_wait in few instructions: the roles of a kernel share the instruction cache.
KV4_COLD bool kv4_wait_slow(uint64_t* bar, uint32_t parity, int* status, int where) {
  const uint64_t t0 = globaltimer(), limit = wait_limit(status);
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) != 0) continue;
    if (globaltimer() - t0 > limit) {
      set_status(status, DF_ERR_TIMEOUT, where);
      return false;
    }
    if (status && *(volatile int*)status == DF_ERR_TIMEOUT) return false;   // another role gave up
  }
}
DF_DEV bool kv4_wait(uint64_t* bar, uint32_t parity, int* status, int where) {
  return mbar_try_wait(bar, parity) || kv4_wait_slow(bar, parity, status, where);
}

// Probabilities of the tcgen05 kernel carry 2^7: with the 2^8 that a late maximum may add they stay below 2^15.
constexpr float kTcShift = 7.f;
constexpr float kLn2 = 0.6931471805599453f;

// ln of the softmax's sum from a maximum and a sum in log2 units.
DF_DEV float kv4_lse(float m, float l, float shift) { return l > 0.f ? (m - shift + log2f(l)) * kLn2 : -INFINITY; }

int launch_kv4_attn_few(Kv4AttnParams p, cudaStream_t st);    // kv4_attention.cu: mma.sync, few rows
int launch_kv4_attn_tc(Kv4AttnParams p, cudaStream_t st);     // kv4_attention_tc.cu: tcgen05, tiles of 128 rows

}  // namespace df
