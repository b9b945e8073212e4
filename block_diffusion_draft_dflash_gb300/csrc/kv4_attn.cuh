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

namespace df {

struct Kv4AttnParams {
  Kv4Planes p;
  int b, T, Hq, Hkv, G, cap, W;
  const df_bf16* q;
  const int32_t* cache_len;
  const uint32_t* anc;
  float scale2;          // scale * log2(e) * 2^k_exp
  float v_mul;           // 2^v_exp
  df_bf16* out;
  float* lse;
  int R, nrt;            // rows of a tile, tiles of a (sequence, kv head)
  int stage;             // keys of a stage
  int min_stages;        // no share is smaller, while there are several
  int n_cta;
  float shift;           // probabilities carry 2^shift
  float* o_part;         // [n_cta + units][R][128]: slot CTA + unit
  float2* ml_part;       // [n_cta + units][R]: maximum in log2 units, sum
  int2* range;           // [units]: first and last CTA
  int* status;
};

// Slots that a tile's rows see at most.
DF_DEV int kv4_tile_len(const Kv4AttnParams& p, int N, int rt) {
  if (N < 0 || N > p.cap - p.T) return 0;   // left out
  return p.anc ? N + p.T : N + min(p.T, ((rt + 1) * p.R - 1) / p.G + 1);
}
DF_DEV int kv4_tile_stages(const Kv4AttnParams& p, int N, int rt) {   // a tile that sees nothing has one
  return max(1, (kv4_tile_len(p, N, rt) + p.stage - 1) / p.stage);
}
DF_DEV int kv4_head_stages(const Kv4AttnParams& p, int s) {   // of one kv head
  const int N = p.cache_len[s];
  if (p.anc || p.nrt == 1) return p.nrt * kv4_tile_stages(p, N, p.nrt - 1);
  int n = 0;
  for (int rt = 0; rt < p.nrt; ++rt) n += kv4_tile_stages(p, N, rt);
  return n;
}

struct Kv4Seg {        // the part of one unit that lies in a share
  int s, kvh, rt, unit;
  int tile0, count;    // stages [tile0, tile0 + count)
  int N, len;          // cache_len (0 where it does not fit), slots seen
  bool first, last;    // holds the unit's first, last stage
};

// A CTA's walk through its share; every call by a whole warp, with the same result in each.
struct Kv4Walk {
  long long t, t1, seq0;   // next stage, end of the share, first stage of sequence s
  int s, head;             // stages of one kv head of s

  DF_DEV bool init(const Kv4AttnParams& p, int cta, int lane) {
    long long total = 0;
    for (int i = lane; i < p.b; i += 32) total += (long long)kv4_head_stages(p, i) * p.Hkv;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long most = (total + p.min_stages - 1) / p.min_stages;
    const int n = most < p.n_cta ? (int)most : p.n_cta;
    if (cta >= n) return false;
    t = total * cta / n;
    t1 = total * (cta + 1) / n;
    s = 0;
    seq0 = 0;
    for (int base = 0; base < p.b; base += 32) {
      long long inc = base + lane < p.b ? (long long)kv4_head_stages(p, base + lane) * p.Hkv : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int k = __popc(__ballot_sync(0xffffffffu, base + lane < p.b && seq0 + inc <= t));   // whole sequences before t
      s += k;
      if (k > 0) seq0 += __shfl_sync(0xffffffffu, inc, k - 1);
      if (k < 32) break;
    }
    head = kv4_head_stages(p, s);
    return true;
  }

  DF_DEV bool next(const Kv4AttnParams& p, Kv4Seg& g) {
    if (t >= t1) return false;
    const int rel = (int)(t - seq0);
    g.s = s;
    g.kvh = rel / head;
    int in_head = rel % head, per_unit;
    const int N = p.cache_len[s];
    if (p.anc || p.nrt == 1) {
      per_unit = head / p.nrt;
      g.rt = in_head / per_unit;
      in_head %= per_unit;
    } else {
      g.rt = 0;
      per_unit = kv4_tile_stages(p, N, 0);
      while (in_head >= per_unit) {
        in_head -= per_unit;
        per_unit = kv4_tile_stages(p, N, ++g.rt);
      }
    }
    g.unit = (s * p.Hkv + g.kvh) * p.nrt + g.rt;
    g.tile0 = in_head;
    g.count = (int)min(t1 - t, (long long)(per_unit - in_head));
    g.len = kv4_tile_len(p, N, g.rt);
    g.N = g.len > 0 ? N : 0;
    g.first = in_head == 0;
    g.last = in_head + g.count == per_unit;
    t += g.count;
    if (t == seq0 + (long long)head * p.Hkv && s + 1 < p.b) {
      seq0 = t;
      head = kv4_head_stages(p, ++s);
    }
    return true;
  }
};

// Probabilities of the tcgen05 kernel carry 2^7: with the 2^8 that a late maximum may add they stay below 2^15.
constexpr float kTcShift = 7.f;
constexpr float kLn2 = 0.6931471805599453f;

// ln of the softmax's sum from a maximum and a sum in log2 units.
DF_DEV float kv4_lse(float m, float l, float shift) { return l > 0.f ? (m - shift + log2f(l)) * kLn2 : -INFINITY; }

int launch_kv4_attn_few(Kv4AttnParams p, cudaStream_t st);    // kv4_attention.cu: mma.sync, few rows
int launch_kv4_attn_tc(Kv4AttnParams p, cudaStream_t st);     // kv4_attention_tc.cu: tcgen05, tiles of 128 rows

}  // namespace df
