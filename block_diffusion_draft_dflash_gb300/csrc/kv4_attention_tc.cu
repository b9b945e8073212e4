// Tree attention over a KV cache held in 4 bits on the tcgen05 tensor cores: tiles of 128 query
// rows (a node's heads of one kv head lie next to one another, so one decoded K/V tile feeds
// all of them).
//
// Per 128-key block:  S = Q K^T (fp16 operands, fp32 in TMEM, three buffers), softmax with a
// running maximum that moves only when a block raises it by more than 2^8, P as fp16 over its
// own S in TMEM, O += P V.  The cache's values are fp16 numbers (kv4.cuh), so decoding loses
// nothing and the products are exact.
//
// Warp roles: 8 softmax / epilogue warps (two per 32 rows, one per 64 columns), 4 decoding
// warps, one MMA issuer (owns TMEM) and one warp that brings the codes.  Codes arrive by
// untiled bulk copies (a block's rows are contiguous) in kNS stages; the decoding warps write K
// as [key][dim] and V as [dim][key] in 128-byte-swizzled rows, which is what the MMA reads as
// K-major operands.  V's codes lie [key][dim]: a decoding thread takes 8 keys x 16 dimensions
// and merges two keys' codes nibble by nibble, so that one conversion yields a pair of keys.
// A CTA walks through its share of all blocks (kv4_attn.cuh), unit by unit.
#include "kv4_attn.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {

constexpr int kCG = 2;                         // column groups (softmax warps per 32 rows)
constexpr int kCols = 128 / kCG;
constexpr int kSoft = 128 * kCG;               // softmax threads
constexpr int kDecWarps = 4;
constexpr int kDec0 = kSoft / 32;              // first decoding warp
constexpr int kMmaWarp = kDec0 + kDecWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
constexpr int kKB = 128;                       // keys of a block
constexpr int kSBufs = 3;                      // S/P buffers in TMEM
constexpr uint32_t kOCol = kSBufs * 128;
constexpr int kNS = 3;                         // stages of codes
constexpr uint32_t kTile = 128 * 128 * 2;      // one fp16 tile: two slabs of 64 columns
constexpr int kOctet = 8 * kKv4Codes + 16;     // V codes of 8 keys, padded: 8 octets start in 8 bank groups
constexpr int kStKc = 0, kStVc = kKB * kKv4Codes, kStKs = kStVc + 16 * kOctet, kStVs = kStKs + kKB * kKv4Scales;
constexpr int kStage = kStVs + kKB * kKv4Scales;
static_assert(kStage % 16 == 0, "bulk copies");

// Instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 bits of a row's visibility for keys j0 .. j0+31.
DF_DEV uint32_t see_bits(const uint32_t* anc, int W, int N, int j0, int node, int len) {
  const int n = N - j0;
  uint32_t bits = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;   // the cache
  const int t0 = -n;                                                     // tree slot of bit 0
  if (anc) {
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

DF_DEV bool soft_and(bool v) {   // over the softmax threads (barrier 1)
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r) : "r"((uint32_t)v), "r"(kSoft) : "memory");
  return r != 0;
}
DF_DEV void soft_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kSoft) : "memory"); }

__global__ void __launch_bounds__(kThreads, 1) kv4_attn_tc_kernel(const Kv4AttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* q_smem = smem;
  unsigned char* k_smem = q_smem + kTile;        // two tiles
  unsigned char* v_smem = k_smem + 2 * kTile;    // two tiles
  unsigned char* codes = v_smem + 2 * kTile;     // kNS stages
  __shared__ __align__(8) uint64_t c_full[kNS], c_empty[kNS], k_full[2], k_empty[2], v_full[2], v_empty[2];
  __shared__ __align__(8) uint64_t s_full[kSBufs], p_full[kSBufs], o_done[kSBufs], q_full, o_free, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ float red_max[2][kCG][128], red_sum[kCG][128];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNS; ++i) { mbar_init(&c_full[i], 1); mbar_init(&c_empty[i], kDecWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kDecWarps); mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kDecWarps); mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], kSoft); mbar_init(&o_done[i], 1); }
    mbar_init(&q_full, kSoft);
    mbar_init(&o_free, kSoft);
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) { tmem_alloc(&tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_slot;
  Kv4Walk walk;
  const bool any = walk.init(p, blockIdx.x, lane);
  Kv4Seg sg;

  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- bring codes
    int j = 0;          // block of this CTA
    bool ok = any;
    while (ok && walk.next(p, sg)) {
      const size_t plane = ((size_t)sg.s * p.Hkv + sg.kvh) * p.cap;
      for (int i = 0; i < sg.count && ok; ++i, ++j) {
        const int st = j % kNS;
        ok = __all_sync(0xffffffffu, mbar_wait(&c_empty[st], ((j / kNS) & 1) ^ 1, p.status, 60));
        if (!ok) break;
        const int key0 = (sg.tile0 + i) * kKB;
        const int n = min(kKB, p.cap - key0);   // a multiple of 8
        unsigned char* to = codes + st * kStage;
        const size_t row = plane + key0;
        if (lane == 0) {
          mbar_arrive_expect_tx(&c_full[st], n * 2 * (kKv4Codes + kKv4Scales));
          bulk_load(to + kStKc, p.p.kc + row * kKv4Codes, n * kKv4Codes, &c_full[st]);
          bulk_load(to + kStKs, p.p.ks + row * kKv4Scales, n * kKv4Scales, &c_full[st]);
          bulk_load(to + kStVs, p.p.vs + row * kKv4Scales, n * kKv4Scales, &c_full[st]);
        }
        __syncwarp();
        if (lane < n / 8) bulk_load(to + kStVc + lane * kOctet, p.p.vc + (row + lane * 8) * kKv4Codes, 8 * kKv4Codes, &c_full[st]);
      }
    }
    // every copy must have landed before the CTA may exit
    for (int i = j - kNS > 0 ? j - kNS : 0; i < j; ++i) mbar_wait(&c_full[i % kNS], (i / kNS) & 1, nullptr, 0);
  } else if (warp >= kDec0 && warp < kMmaWarp) {
    // ---------------------------------------------------------------- decode
    const int w = warp - kDec0;
    int j = 0;
    bool ok = any;
    while (ok && walk.next(p, sg)) {
      for (int i = 0; i < sg.count; ++i, ++j) {
        const int st = j % kNS, buf = j & 1;
        const uint32_t free_parity = ((j >> 1) & 1) ^ 1;
        ok = mbar_wait(&c_full[st], (j / kNS) & 1, p.status, 61) && mbar_wait(&k_empty[buf], free_parity, p.status, 62);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const unsigned char* from = codes + st * kStage;
        {
          // K: one key per lane; its four 16-byte pieces in an order that spreads the lanes
          // of a phase over all banks, both when reading and when writing
          const int key = w * 32 + lane;
          unsigned char* dst = k_smem + buf * kTile + key * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int cc = (c + (lane >> 1)) & 3;
            const uint4 x = *reinterpret_cast<const uint4*>(from + kStKc + key * kKv4Codes + cc * 16);
            const uint32_t two = *reinterpret_cast<const uint16_t*>(from + kStKs + key * kKv4Scales + cc * 2);
            const uint32_t s0 = e4m3x2_to_f16((two & 0xFFu) * 0x00010001u), s1 = e4m3x2_to_f16((two >> 8) * 0x00010001u);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t f[4];
              e2m1x8_to_f16(xs[e], f);
              const uint32_t sc = e < 2 ? s0 : s1;
              const int pos = ((cc & 1) * 4 + e) ^ (key & 7);
              *reinterpret_cast<uint4*>(dst + (cc >> 1) * (kTile / 2) + pos * 16) =
                  make_uint4(hmul2(f[0], sc), hmul2(f[1], sc), hmul2(f[2], sc), hmul2(f[3], sc));
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[buf]);
        ok = mbar_wait(&v_empty[buf], free_parity, p.status, 63);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        {
          // V: 8 keys (octet 8 (w / 2) + lane % 8) x 16 dimensions (block 4 (w % 2) + lane / 8)
          const int o8 = lane & 7, blk = (w & 1) * 4 + (lane >> 3), oct = (w >> 1) * 8 + o8;
          uint2 x[8];
          uint32_t sc[4];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const uint2*>(from + kStVc + oct * kOctet + k * kKv4Codes + blk * 8);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned char* sp = from + kStVs + (oct * 8 + 2 * k) * kKv4Scales + blk;
            sc[k] = e4m3x2_to_f16((uint32_t)sp[0] | ((uint32_t)sp[kKv4Scales] << 16));
          }
          unsigned char* dst = v_smem + buf * kTile + (w >> 1) * (kTile / 2) + blk * 16 * 128;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t ev[4][4], od[4][4];   // [pair of keys][even or odd dimension]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a = h ? x[2 * k].y : x[2 * k].x, b = h ? x[2 * k + 1].y : x[2 * k + 1].x;
              e2m1x8_to_f16((a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4), ev[k]);
              e2m1x8_to_f16(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), od[k]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int d0 = h * 8 + 2 * m;   // row of the tile, modulo 16
              *reinterpret_cast<uint4*>(dst + d0 * 128 + (o8 ^ (d0 & 7)) * 16) =
                  make_uint4(hmul2(ev[0][m], sc[0]), hmul2(ev[1][m], sc[1]), hmul2(ev[2][m], sc[2]), hmul2(ev[3][m], sc[3]));
              *reinterpret_cast<uint4*>(dst + (d0 + 1) * 128 + (o8 ^ ((d0 + 1) & 7)) * 16) =
                  make_uint4(hmul2(od[0][m], sc[0]), hmul2(od[1][m], sc[1]), hmul2(od[2][m], sc[2]), hmul2(od[3][m], sc[3]));
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[buf]);
          mbar_arrive(&c_empty[st]);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    // The warp runs in lockstep (every decision is a vote); one elected lane issues.
    constexpr uint32_t idesc = idesc_f16_f32(128, 128);
    const uint32_t qa = smem_u32(q_smem);
    const bool leader = elect_one();
    bool ok = any;
    int s_next = 0, pv_next = 0, n_seg = 0;
    while (ok && walk.next(p, sg)) {
      const int end = s_next + sg.count, first = s_next;
      ok = mbar_wait(&q_full, n_seg & 1, p.status, 64);
      // the epilogue has read the previous unit's O
      if (n_seg > 0) ok = mbar_wait(&o_free, (n_seg - 1) & 1, p.status, 65) && ok;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      ++n_seg;
      int idle = 0;
      uint64_t t_idle = 0;
      const uint64_t limit = wait_limit(p.status);
      while (ok && pv_next < end) {
        if (s_next < end && s_next - pv_next < kSBufs &&
            __any_sync(0xffffffffu, mbar_test_wait(&k_full[s_next & 1], (s_next >> 1) & 1))) {
          tc_fence_after();
          const uint32_t kb = smem_u32(k_smem + (s_next & 1) * kTile);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk >> 2) * (kTile / 2) + (kk & 3) * 32;
              mma_bf16(tmem + (s_next % kSBufs) * 128, sdesc_kmajor_sw128(qa + off), sdesc_kmajor_sw128(kb + off), idesc,
                       kk > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[s_next % kSBufs]);
            mma_commit(&k_empty[s_next & 1]);
          }
          __syncwarp();
          ++s_next;
        } else if (pv_next < s_next &&
                   __any_sync(0xffffffffu, mbar_test_wait(&p_full[pv_next % kSBufs], (pv_next / kSBufs) & 1) &&
                                               mbar_test_wait(&v_full[pv_next & 1], (pv_next >> 1) & 1))) {
          tc_fence_after();
          const uint32_t vb = smem_u32(v_smem + (pv_next & 1) * kTile);
          const uint32_t pt = tmem + (pv_next % kSBufs) * 128;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              constexpr int kPer = kCols / 16;   // 16-key steps of one column group
              const uint32_t off = (kk >> 2) * (kTile / 2) + (kk & 3) * 32;
              mma_bf16_ts(tmem + kOCol, pt + (kk / kPer) * kCols + (kk % kPer) * 8, sdesc_kmajor_sw128(vb + off), idesc,
                          (pv_next > first || kk > 0) ? 1u : 0u);
            }
            mma_commit(&o_done[pv_next % kSBufs]);
            mma_commit(&v_empty[pv_next & 1]);
          }
          __syncwarp();
          ++pv_next;
        } else {
          if ((++idle & 1023) == 0) {   // bounded: give up after the wait limit without progress
            const uint64_t now = __shfl_sync(0xffffffffu, globaltimer(), 0);
            if (t_idle == 0) t_idle = now;
            else if (now - t_idle > limit) {
              if (leader) set_status(p.status, DF_ERR_TIMEOUT, 66);
              ok = false;
            }
            if (__any_sync(0xffffffffu, p.status && *(volatile int*)p.status == DF_ERR_TIMEOUT)) ok = false;
          }
          continue;
        }
        idle = 0;
        t_idle = 0;
      }
    }
    if (!ok && s_next > 0) {   // giving up: the MMAs issued must finish before TMEM is freed
      if (leader) mma_commit(&drain);
      __syncwarp();
      mbar_wait(&drain, 0, nullptr, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax, epilogue
    // Warp w: TMEM lanes 32 (w % 4) .. + 31, one query row per thread, columns 64 (w / 4) .. + 63
    // of S (keys) and of O (dimensions).
    const int grp = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    constexpr float kRescale = 8.f;
    bool ok = any;
    int j = 0;
    while (ok && walk.next(p, sg)) {
      const int row = sg.rt * 128 + r, node = row / p.G;
      const bool row_ok = node < p.T;
      const bool live = __any_sync(0xffffffffu, row_ok);
      if (sg.len == 0 && threadIdx.x == 0) set_status(p.status, DF_ERR_CAPACITY, sg.s);
      const size_t grow = ((size_t)sg.s * p.T + node) * p.Hq + sg.kvh * p.G + row % p.G;
      // Q: the row, brought to fp16 by a power of two, into its swizzled place; every S of the
      // previous unit is complete (its scores were read)
      float qs;
      {
        uint4 raw[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) raw[c] = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + grow * 128 + grp * 64);
#pragma unroll
          for (int c = 0; c < 8; ++c) raw[c] = src[c];
        }
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
        }
        red_sum[grp][r] = amax;
        soft_sync();
        float back;
        const float f = f16_row_factor(fmaxf(red_sum[0][r], red_sum[1][r]), back);
        qs = p.scale2 * back;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = pack_f16x2(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xFFFF0000u) * f);
          *reinterpret_cast<uint4*>(q_smem + grp * (kTile / 2) + r * 128 + ((c ^ (r & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async();
        mbar_arrive(&q_full);
      }
      const uint32_t* anc_row = p.anc && row_ok ? p.anc + ((size_t)sg.s * p.T + node) * p.W : nullptr;
      // no row of the tile has its mask before this key
      const int edge_key = sg.len == 0 ? 0 : p.anc ? sg.N : sg.N + min(p.T - 1, sg.rt * 128 / p.G) + 1;
      float m_run = -INFINITY, l_part = 0.f;   // the maximum in raw scores
      for (int i = 0; i < sg.count; ++i, ++j) {
        const bool w1 = __all_sync(0xffffffffu, mbar_wait(&s_full[j % kSBufs], (j / kSBufs) & 1, p.status, 67));
        float sv[kCols];
        float mpart = -INFINITY;
        const uint32_t sp = tmem + lane_base + (j % kSBufs) * 128 + grp * kCols;
        if (w1) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_ld16(sp + c, sv + c);
          tmem_ld_wait();
          const int key0 = (sg.tile0 + i) * kKB + grp * kCols;
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if ((sg.tile0 + i + 1) * kKB > edge_key) {
            uint32_t adm[kCols / 32];
#pragma unroll
            for (int x = 0; x < kCols / 32; ++x)
              adm[x] = row_ok && (anc_row || !p.anc) ? see_bits(anc_row, p.W, sg.N, key0 + 32 * x, node, sg.len) : 0u;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              if (!((adm[c >> 5] >> (c & 31)) & 1u)) sv[c] = -INFINITY;
              m4[c & 3] = fmaxf(m4[c & 3], sv[c]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kCols; ++c) m4[c & 3] = fmaxf(m4[c & 3], sv[c]);
          }
          mpart = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else {
#pragma unroll
          for (int c = 0; c < kCols; ++c) sv[c] = -INFINITY;
        }
        red_max[j & 1][grp][r] = mpart;
        if (!soft_and(w1 && ok)) { ok = false; break; }
        const float mx = fmaxf(red_max[j & 1][0][r], red_max[j & 1][1][r]);
        float alpha = 1.f;
        if ((mx - m_run) * qs > kRescale) {           // also on the first key a row sees
          alpha = ex2_approx((m_run - mx) * qs);
          m_run = mx;
        }
        uint32_t packed[kCols / 2];
        if (live && m_run != -INFINITY) {
          const float mb = kTcShift - m_run * qs;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float p0 = ex2_approx(fmaf(sv[c], qs, mb)), p1 = ex2_approx(fmaf(sv[c + 1], qs, mb));
            const float p2 = ex2_approx(fmaf(sv[c + 2], qs, mb)), p3 = ex2_approx(fmaf(sv[c + 3], qs, mb));
            s4[(c >> 2) & 3] += (p0 + p1) + (p2 + p3);
            packed[c >> 1] = pack_f16x2(p0, p1);
            packed[(c >> 1) + 1] = pack_f16x2(p2, p3);
          }
          l_part = l_part * alpha + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) packed[c] = 0u;
        }
        if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O must hold PV of every earlier block before it is rescaled
          ok = mbar_wait(&o_done[(j - 1) % kSBufs], ((j - 1) / kSBufs) & 1, p.status, 68) && ok;
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint32_t oaddr = tmem + lane_base + kOCol + grp * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float o[16];
            tmem_ld16(oaddr + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= alpha;
            tmem_st16(oaddr + c, o);
          }
        }
        tmem_st32(sp, packed);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[j % kSBufs]);
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      ok = mbar_wait(&o_done[(j - 1) % kSBufs], ((j - 1) / kSBufs) & 1, p.status, 69) && ok;
      red_sum[grp][r] = l_part;
      if (!soft_and(ok)) { ok = false; break; }
      tc_fence_after();
      const float l = red_sum[0][r] + red_sum[1][r];
      const float m2 = m_run == -INFINITY ? -INFINITY : m_run * qs;
      const uint32_t oaddr = tmem + lane_base + kOCol + grp * kCols;
      const bool whole = sg.first && sg.last;
      const float inv = l > 0.f ? p.v_mul / l : 0.f;
      const size_t at = (size_t)(blockIdx.x + sg.unit) * 128 + r;
      if (live) {
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          float o[16];
          tmem_ld16(oaddr + c, o);
          tmem_ld_wait();
          if (row_ok && whole) {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.out + grow * 128 + grp * kCols + c);
            dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
            dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
          } else if (row_ok) {
            float4* dst = reinterpret_cast<float4*>(p.o_part + at * 128 + grp * kCols + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (row_ok && grp == 0) {
          if (!whole) p.ml_part[at] = make_float2(m2, l);
          else if (p.lse) p.lse[grow] = kv4_lse(m2, l, kTcShift);
        }
      }
      if (threadIdx.x == 0) {
        if (whole) p.range[sg.unit] = make_int2(0, 0);
        else if (sg.first) p.range[sg.unit].x = blockIdx.x;
        else if (sg.last) p.range[sg.unit].y = blockIdx.x;
      }
      tc_fence_before();
      soft_sync();   // red_sum is read before the next unit writes it
      mbar_arrive(&o_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

int launch_kv4_attn_tc(Kv4AttnParams p, cudaStream_t st) {
  p.shift = kTcShift;
  const size_t smem = 1024 + 5 * kTile + kNS * kStage;
  if (ensure_dynamic_smem(kv4_attn_tc_kernel, smem) != cudaSuccess) return DF_ERR_CUDA;
  launch_k(kv4_attn_tc_kernel, dim3(p.n_cta), dim3(kThreads), smem, st, p);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
