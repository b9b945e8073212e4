// What the two attention kernels over the 4-bit cache share: parameters, the cutting of the
// work into shares, the mask, and the form in which partial results reach the combine kernel.
//
// A unit is one (sequence, kv head, tile of R query rows); its keys come in stages.  All
// stages of a call lie in one line (sequence-major), which the CTAs cut into equal shares
// whatever the sequences' lengths.  A unit that lies inside one share is finished by its CTA;
// the parts of a cut unit go to slots that the combine kernel reads in the order of the CTAs.
// A share cuts two units at most, the one it begins in and the one it ends in.
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
  int change_step;       // a seventh of what going over to another unit costs, in stages
  int n_cta;
  float shift;           // probabilities carry 2^shift
  float* o_part;         // [slots][R][128], two slots of each CTA
  float2* ml_part;       // [slots][R]: maximum in log2 units, sum
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

// ceil(x / d) by a multiplication: magic = floor((2^32 - 1) / d) + 1, d > 1, exact for (x + d) d < 2^32.
DF_DEV int kv4_parts(int x, int d, uint32_t magic) { return (int)__umulhi((uint32_t)(x + d - 1), magic); }

// The line's length over one kv head of a sequence of N slots: stages, or (per > 1) parts of at
// most `per` stages.
DF_DEV int kv4_head_line(const Kv4AttnParams& p, int N, int per, uint32_t magic) {
  auto line = [&](int stages) { return per == 1 ? stages : kv4_parts(stages, per, magic); };
  if (kv4_even(p)) {
    const int len = kv4_all(p, N);
    const int last = line(kv4_stages(p, len, p.last_single));
    return p.nrt == 1 ? last : (p.nrt - 1) * line(kv4_stages(p, len, false)) + last;
  }
  int n = 0;
#pragma unroll 1
  for (int rt = 0; rt < p.nrt; ++rt) n += line(kv4_stages(p, kv4_chain(p, N, rt), kv4_single(p, rt)));
  return n;
}

struct Kv4Seg {        // the part of one unit that a CTA works on
  int s, kvh, rt, unit;
  int tile0, count;    // stages [tile0, tile0 + count)
  int N, len;          // cache_len (0 where it does not fit), slots seen
  int first, last;     // holds the unit's first, last stage
  int single;          // kv4_single
  int held;            // kv4_held, where a warp hands units out
};

// The workspace's hold word, which makes a call give up (tests of the failure path).  Read beside
// the lengths: it costs no time of its own.
DF_DEV int kv4_held(const int* status) { return *(const volatile int*)(status + 4); }
// By a whole warp.
KV4_COLD bool kv4_hold_clear(int* status, int where, int lane) {
  return __all_sync(0xffffffffu, lane != 0 || wait_hold_clear(status, where));
}

// A CTA's walk through its share.  One warp of the CTA walks (code that a kernel runs once
// costs some 50 cycles an instruction) and hands the units out by shared memory.
//
// Where there are enough CTAs every unit is cut into equal parts of at most `per` stages, one
// for each CTA, with the smallest `per` that the CTAs allow.  Going over to another unit costs
// as much as some stages (an epilogue, another Q), so this is done unless the largest part
// exceeds the mean share by more than 7 p.change_step.  Else the shares are equal pieces of the line of
// all stages, whatever units they cut.
struct Kv4Walk {
  int t, t1, end;      // next place in the line, end of the share, end of sequence s
  int s, head;         // line of one kv head of s
  int per;             // 1: the line counts stages; else parts
  uint32_t magic;      // of kv4_parts

  DF_DEV static uint32_t magic_of(int d) { return 0xFFFFFFFFu / (uint32_t)d + 1u; }   // 0 for d = 1: not used

  // By a whole warp, like next(); false: no share.
  DF_DEV bool init(const Kv4AttnParams& p, int cta, int lane) {
    const int N0 = lane < p.b ? p.cache_len[lane] : 0;   // of the first 32 sequences
    // Pass 0: the sum of all stages.  Pass 1: for 8 lengths of a part, a lane each, the parts
    // that they make of four sequences at a time.  Then the place in the line that was chosen.
    int total = 0, mean = 0;
    per = 1;
    magic = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      const int d = max(2, mean) + (lane & 7) * p.change_step;
      const uint32_t m = pass ? magic_of(d) : 0u;
      const int step = pass ? 4 : 32, first = pass ? lane >> 3 : lane;
      int n = 0;
#pragma unroll 1
      for (int base = 0; base < p.b; base += step) {
        const int i = base + first;
        const int N = base < 32 ? __shfl_sync(0xffffffffu, N0, i & 31) : i < p.b ? p.cache_len[i] : 0;
        if (i < p.b) n += kv4_head_line(p, N, pass ? d : 1, m) * p.Hkv;
      }
      n += __shfl_xor_sync(0xffffffffu, n, 16);
      n += __shfl_xor_sync(0xffffffffu, n, 8);
      if (pass == 0) {
        total = __reduce_add_sync(0xffffffffu, lane < 8 ? n : 0);
        mean = max(p.min_stages, (total + p.n_cta - 1) / p.n_cta);
      } else {
        const uint32_t fits = __ballot_sync(0xffffffffu, n <= p.n_cta) & 0xFFu;
        if (fits) {
          const int k = __ffs(fits) - 1;
          per = __shfl_sync(0xffffffffu, d, k);
          magic = __shfl_sync(0xffffffffu, m, k);
          total = __shfl_sync(0xffffffffu, n, k);
        }
      }
    }
    if (per > 1) {
      if (cta >= total) return false;
      t = cta;
      t1 = cta + 1;
    } else {
      const int n = min((total + p.min_stages - 1) / p.min_stages, p.n_cta);
      if (cta >= n) return false;
      const int q = total / n, rest = total - q * n;   // the first `rest` shares have one more
      t = q * cta + min(cta, rest);
      t1 = t + q + (cta < rest ? 1 : 0);
    }
    int before = 0;
#pragma unroll 1
    for (int base = 0;; base += 32) {
      const int N = base == 0 ? N0 : base + lane < p.b ? p.cache_len[base + lane] : 0;
      const int h = base + lane < p.b ? kv4_head_line(p, N, per, magic) : 0;
      int inc = h * p.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int k = __popc(__ballot_sync(0xffffffffu, base + lane < p.b && before + inc <= t));   // sequences before t
      if (k < 32) {
        s = base + k;
        head = __shfl_sync(0xffffffffu, h, k);
        end = before + __shfl_sync(0xffffffffu, inc, k);
        return true;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
  }

  DF_DEV bool next(const Kv4AttnParams& p, Kv4Seg& g) {
    if (t >= t1) return false;
    if (t == end) {
      head = kv4_head_line(p, p.cache_len[++s], per, magic);
      end += head * p.Hkv;
    }
    int rel = t - (end - head * p.Hkv), rt = 0;
    const int N = p.cache_len[s];
    g.kvh = rel / head;
    rel -= g.kvh * head;
    // the tile, and the place in its own piece of the line
    int len = kv4_all(p, N), stages, piece;
#pragma unroll 1
    for (;; ++rt) {
      if (!kv4_even(p)) len = kv4_chain(p, N, rt);
      stages = kv4_stages(p, len, kv4_single(p, rt));
      piece = per == 1 ? stages : kv4_parts(stages, per, magic);
      if (kv4_even(p) && rt == 0 && p.nrt > 2) {   // all tiles but the last are alike
        const int skip = min(rel / piece, p.nrt - 1);
        rel -= skip * piece;
        rt = skip;
        if (rt < p.nrt - 1) break;
        --rt;
        continue;
      }
      if (rel < piece) break;
      rel -= piece;
    }
    g.s = s;
    g.rt = rt;
    g.unit = (s * p.Hkv + g.kvh) * p.nrt + rt;
    if (per == 1) {
      g.tile0 = rel;
      g.count = min(t1 - t, stages - rel);
      t += g.count;
    } else {   // equal parts
      const int q = stages / piece, rest = stages - q * piece;
      g.tile0 = q * rel + min(rel, rest);
      g.count = q + (rel < rest ? 1 : 0);
      ++t;
    }
    g.len = len;
    g.N = len > 0 ? N : 0;
    g.single = kv4_single(p, rt);
    g.first = g.tile0 == 0;
    g.last = g.tile0 + g.count == stages;
    return true;
  }
};

// Slot of a cut unit's part: 2 CTA + 1 for the one that begins the unit, 2 CTA for any other.
DF_DEV int kv4_slot(int cta, bool first) { return 2 * cta + (first ? 1 : 0); }

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

// A query row's share of a lane: dimensions 32 t4 .. + 31 as fp16 (brought there by a power of
// two that the quad agrees on, `back` its inverse), two registers for each of 8 steps.
DF_DEV void load_q(const df_bf16* src, bool on, int t4, uint32_t (&f)[8][2], float& back) {
  uint4 raw[4];
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) raw[c] = on ? reinterpret_cast<const uint4*>(src + t4 * 32)[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const float s = f16_row_factor(amax, back);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[2 * c + (e >> 1)][e & 1] = pack_f16x2(__uint_as_float(w[e] << 16) * s, __uint_as_float(w[e] & 0xFFFF0000u) * s);
  }
}

// Probabilities of the tcgen05 kernel carry 2^7: with the 2^8 that a late maximum may add they stay below 2^15.
constexpr float kTcShift = 7.f;
constexpr float kLn2 = 0.6931471805599453f;

// ln of the softmax's sum from a maximum and a sum in log2 units; a sum of NaN gives NaN.
DF_DEV float kv4_lse(float m, float l, float shift) { return l == 0.f ? -INFINITY : (m - shift + log2f(l)) * kLn2; }

int launch_kv4_attn_few(Kv4AttnParams p, cudaStream_t st);    // kv4_attention.cu: mma.sync, few rows
int launch_kv4_attn_tc(Kv4AttnParams p, cudaStream_t st);     // kv4_attention_tc.cu: tcgen05, tiles of 128 rows

}  // namespace df
