// Attention over a KV cache held in 4 bits, for few query rows per kv head.
//
// Row (s, i, h) sees slots [0, N) and the tree slots N + j of its ancestors, N = cache_len[s]:
//   out = softmax(scale q K^T) V,  lse = log of the softmax's sum
// with K, V the values that the cache's codes and scales stand for (kv4.cuh: fp16 numbers, so
// the fp16 tensor-core products are exact; sums, softmax statistics and outputs are fp32).
//
// What bounds it with few rows is the cache, 144 bytes a slot and kv head, and then the
// instructions that decode it: one token of 16 sequences of 9803 to 32768 slots, 8 kv heads (393
// MB), takes 81 us, 4.8 TB/s, with an instruction issued in 65 % of the schedulers' cycles; 8 rows
// of one sequence of 2000 slots take 8 us, which is latency.  Every warp streams stages of 32 slots
// (bulk copies into a ring of its own, no CTA barrier), decodes codes straight into tensor-core
// fragments and keeps its own running maximum, sum and output; the warps are merged when the CTA's
// part of a unit ends.
//
// Both products are transposed, S^T = K Q^T and O^T = V^T P^T: the cache is the 16-row operand
// and the query rows are the 8 columns, so 8 rows (4 heads of a token, say) cost half of what
// they would as rows.  P goes from the one product's accumulators to the other's operand by
// an 8 x 8 transposition in registers.
#include <math.h>

#include "kv4_attn.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {

constexpr int kWarps = 8;
constexpr int kStageKeys = 32;   // launch: stage_log2
constexpr int kStages = 2;
constexpr int kStageBytes = kStageKeys * 2 * (kKv4Codes + kKv4Scales);   // K codes, V codes, K scales, V scales
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
// Probabilities are scaled by 2^12 before they are rounded to fp16 (the tensor cores' operand; 11
// significant bits, more than the bf16 output has; their sum is taken before): what lies 2^26 below
// the row's largest still has all its bits.
constexpr float kPShift = 12.f;

// 8 x 8 fp16 transposition: lane (g, t) has row g, columns 2t, 2t+1, before and after.
DF_DEV uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int NT>   // tiles of 8 query rows
__global__ void __launch_bounds__(kWarps * 32, 2) kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int R = 8 * NT;
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float2 ml[kWarps][R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  unsigned char* ring = smem + warp * kStages * kStageBytes;
  pdl_wait();
  pdl_trigger();
  Kv4Walk walk;
  if (!walk.init(p, blockIdx.x, lane)) return;
  Kv4Seg seg;
  uint32_t slot = 0, phase = 0;   // of the warp's next stage
  bool ok = true;
  while (walk.next(p, seg)) {
    const int s = seg.s, kvh = seg.kvh, tile0 = seg.tile0, count = seg.count, N = seg.N, len = seg.len;
    if (len == 0 && tid == 0) set_status(p.status, DF_ERR_CAPACITY, s);
    const size_t plane = ((size_t)s * p.Hkv + kvh) * p.cap;
    const int rows = min(R, p.T * p.G - seg.rt * R);   // live rows of the tile
    auto issue = [&](int i, uint32_t to) {   // this warp's i-th stage of the unit
      if (lane == 0) {
        unsigned char* st = ring + to * kStageBytes;
        uint64_t* bar = &bars[warp][to];
        const int key0 = (tile0 + warp + i * kWarps) * kStageKeys;
        const uint32_t n = min(kStageKeys, p.cap - key0);   // a multiple of 8
        const size_t row = plane + key0;
        mbar_arrive_expect_tx(bar, n * 2 * (kKv4Codes + kKv4Scales));
        bulk_load(st, p.p.kc + row * kKv4Codes, n * kKv4Codes, bar);
        bulk_load(st + 2 * kStageKeys * kKv4Codes, p.p.ks + row * kKv4Scales, n * kKv4Scales, bar);
        bulk_load(st + kStageKeys * kKv4Codes, p.p.vc + row * kKv4Codes, n * kKv4Codes, bar);
        bulk_load(st + kStageKeys * (2 * kKv4Codes + kKv4Scales), p.p.vs + row * kKv4Scales, n * kKv4Scales, bar);
      }
    };
    const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
    for (int i = 0; i < kStages && i < mine; ++i) issue(i, (slot + i) % kStages);
    const int held = kv4_held(p.status);   // on its way beside the rows
    // Q^T fragments: column n = g of tile q is row 8 q + g.  The products run over dimensions in
    // the order in which a lane finds its codes: 32 t4 .. + 31, four at a step.
    uint32_t qf[NT][8][2];
    float qs[NT][2];   // raw score -> log2 units, of rows 2 t4, 2 t4 + 1 (this lane's columns of S^T)
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int r = seg.rt * R + q * 8 + g, node = r / p.G;
      float back;
      load_q(p.q + (((size_t)s * p.T + node) * p.Hq + kvh * p.G + r - node * p.G) * 128, node < p.T, t4, qf[q], back);
      back *= p.scale2;
      qs[q][0] = __shfl_sync(0xffffffffu, back, t4 * 8);
      qs[q][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4);
    }
    if (held && ok) ok = kv4_hold_clear(p.status, 51, lane);   // held: give up with copies on their way
    float o[NT][8][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[q][j][0] = o[q][j][1] = o[q][j][2] = o[q][j][3] = 0.f;
      mx[q][0] = mx[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
    }
    int i = 0;
#pragma unroll 1
    for (; i < mine; ++i) {
      ok = __all_sync(0xffffffffu, ok && kv4_wait(&bars[warp][slot], phase, p.status, 50));
      if (!ok) break;
      const unsigned char* st = ring + slot * kStageBytes;
      const unsigned char *skc = st, *svc = st + kStageKeys * kKv4Codes;
      const unsigned char *sks = st + 2 * kStageKeys * kKv4Codes, *svs = sks + kStageKeys * kKv4Scales;
      const int key0 = (tile0 + warp + i * kWarps) * kStageKeys;
      // S^T: two tiles of 16 keys.  Row x of 8 (of a tile's upper or lower half) is key
      // 4 (x % 2) + x / 2, so that lane t4's columns of P belong to keys t4 + 4 e, whose value
      // rows it decodes below.
      float sc[NT][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < NT; ++q) sc[q][h][0] = sc[q][h][1] = sc[q][h][2] = sc[q][h][3] = 0.f;
        const int key = h * 16 + (g & 1) * 4 + (g >> 1);   // and 8 further
        const uint4 ca = *reinterpret_cast<const uint4*>(skc + key * kKv4Codes + t4 * 16);
        const uint4 cb = *reinterpret_cast<const uint4*>(skc + (key + 8) * kKv4Codes + t4 * 16);
        const uint32_t ta = *reinterpret_cast<const uint16_t*>(sks + key * kKv4Scales + t4 * 2);
        const uint32_t tb = *reinterpret_cast<const uint16_t*>(sks + (key + 8) * kKv4Scales + t4 * 2);
        // both blocks' scales of a key in one word, then either of them in both halves
        const uint32_t pa = e4m3x2_to_f16(__byte_perm(ta, 0, 0x4140)), pb = e4m3x2_to_f16(__byte_perm(tb, 0, 0x4140));
        const uint32_t sa[2] = {__byte_perm(pa, 0, 0x1010), __byte_perm(pa, 0, 0x3232)};
        const uint32_t sb[2] = {__byte_perm(pb, 0, 0x1010), __byte_perm(pb, 0, 0x3232)};
        const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t fa[4], fb[4];
          e2m1x8_to_f16(wa[e], fa);
          e2m1x8_to_f16(wb[e], fb);
#pragma unroll
          for (int x = 0; x < 4; ++x) { fa[x] = hmul2(fa[x], sa[e >> 1]); fb[x] = hmul2(fb[x], sb[e >> 1]); }
          const uint32_t a0[4] = {fa[0], fb[0], fa[1], fb[1]}, a1[4] = {fa[2], fb[2], fa[3], fb[3]};
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            mma_f16_16816(sc[q][h], a0, qf[q][2 * e][0], qf[q][2 * e][1]);
            mma_f16_16816(sc[q][h], a1, qf[q][2 * e + 1][0], qf[q][2 * e + 1][1]);
          }
        }
      }
      // log2 units, mask, running maximum
      const bool edge = key0 + kStageKeys > N;
      uint32_t pf[NT][2][2];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[q][h][e] *= qs[q][e & 1];
        if (edge) {
          uint32_t bits[2] = {0u, 0u};
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {   // one copy of the code
            const int r = seg.rt * R + q * 8 + t4 * 2 + c, node = r / p.G;
            const uint32_t* anc = p.anc && node < p.T ? p.anc + ((size_t)s * p.T + node) * p.W : nullptr;
            const uint32_t x = node < p.T ? kv4_see_bits(anc, p.W, N, key0, node, len) : 0u;
            bits[0] = c == 0 ? x : bits[0];
            bits[1] = x;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((bits[e & 1] >> (h * 16 + (e >> 1) * 8 + (g & 1) * 4 + (g >> 1))) & 1u)) sc[q][h][e] = -INFINITY;
        }
        float mt[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mt[c] = fmaxf(fmaxf(sc[q][0][c], sc[q][0][c + 2]), fmaxf(sc[q][1][c], sc[q][1][c + 2]));
          mt[c] = fmaxf(mt[c], __shfl_xor_sync(0xffffffffu, mt[c], 4));
          mt[c] = fmaxf(mt[c], __shfl_xor_sync(0xffffffffu, mt[c], 8));
          mt[c] = fmaxf(mt[c], __shfl_xor_sync(0xffffffffu, mt[c], 16));
          mt[c] = fmaxf(mt[c], mx[q][c]);
        }
        if (__any_sync(0xffffffffu, mt[0] > mx[q][0] || mt[1] > mx[q][1])) {
          const float a0 = mx[q][0] == -INFINITY ? 0.f : ex2_approx(mx[q][0] - mt[0]);
          const float a1 = mx[q][1] == -INFINITY ? 0.f : ex2_approx(mx[q][1] - mt[1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) { o[q][j][0] *= a0; o[q][j][1] *= a1; o[q][j][2] *= a0; o[q][j][3] *= a1; }
          l[q][0] *= a0;
          l[q][1] *= a1;
          mx[q][0] = mt[0];
          mx[q][1] = mt[1];
        }
        // a row that has seen nothing yet: every score is -inf, and 2^(-inf - 0) = 0
        const float b0 = kPShift - (mt[0] == -INFINITY ? 0.f : mt[0]), b1 = kPShift - (mt[1] == -INFINITY ? 0.f : mt[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = ex2_approx(sc[q][h][0] + b0), p1 = ex2_approx(sc[q][h][1] + b1);
          const float p2 = ex2_approx(sc[q][h][2] + b0), p3 = ex2_approx(sc[q][h][3] + b1);
          l[q][0] += p0 + p2;
          l[q][1] += p1 + p3;
          pf[q][h][0] = transpose8(pack_f16x2(p0, p1));
          pf[q][h][1] = transpose8(pack_f16x2(p2, p3));
        }
      }
      // O^T: lane g takes dimensions 16 g .. 16 g + 15 (one scale a key), tile j rows the 2j-th
      // and the 2j+1-th of them.  Two keys' codes are merged nibble by nibble, so that one
      // conversion gives the pair of keys that a fragment register holds.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 c[4];
        uint32_t sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = h * 16 + e * 4 + t4;
          c[e] = *reinterpret_cast<const uint2*>(svc + key * kKv4Codes + g * 8);
          sb[e] = svs[key * kKv4Scales + g];
        }
        const uint32_t s01 = e4m3x2_to_f16(__byte_perm(sb[0], sb[1], 0x5450)), s23 = e4m3x2_to_f16(__byte_perm(sb[2], sb[3], 0x5450));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t c0 = w ? c[0].y : c[0].x, c1 = w ? c[1].y : c[1].x, c2 = w ? c[2].y : c[2].x, c3 = w ? c[3].y : c[3].x;
          uint32_t e01[4], o01[4], e23[4], o23[4];
          e2m1x8_to_f16((c0 & 0x0F0F0F0Fu) | ((c1 << 4) & 0xF0F0F0F0u), e01);
          e2m1x8_to_f16(((c0 >> 4) & 0x0F0F0F0Fu) | (c1 & 0xF0F0F0F0u), o01);
          e2m1x8_to_f16((c2 & 0x0F0F0F0Fu) | ((c3 << 4) & 0xF0F0F0F0u), e23);
          e2m1x8_to_f16(((c2 >> 4) & 0x0F0F0F0Fu) | (c3 & 0xF0F0F0F0u), o23);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t a[4] = {hmul2(e01[x], s01), hmul2(o01[x], s01), hmul2(e23[x], s23), hmul2(o23[x], s23)};
#pragma unroll
            for (int q = 0; q < NT; ++q) mma_f16_16816(o[q][4 * w + x], a, pf[q][h][0], pf[q][h][1]);
          }
        }
      }
      __syncwarp();   // every lane has read the stage
      if (i + kStages < mine) issue(i + kStages, slot);
      if (++slot == kStages) { slot = 0; phase ^= 1; }
    }
    for (const int out = min(mine, i + kStages); i < out; ++i) {   // given up: the copies on their way must land
      kv4_wait(&bars[warp][slot], phase, nullptr, 0);
      if (++slot == kStages) { slot = 0; phase ^= 1; }
    }
    // ---------------------------------------------------------------- merge the warps
    __syncthreads();   // every ring is read, every copy of the unit has landed
    float* so = reinterpret_cast<float*>(smem) + warp * R * 128;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[q][c] += __shfl_xor_sync(0xffffffffu, l[q][c], 4);
        l[q][c] += __shfl_xor_sync(0xffffffffu, l[q][c], 8);
        l[q][c] += __shfl_xor_sync(0xffffffffu, l[q][c], 16);
        const int r = q * 8 + t4 * 2 + c;
        if (g == 0) ml[warp][r] = make_float2(mx[q][c], l[q][c]);
        // the row's dimensions 16 g .. + 15, their four pieces in an order that spreads the lanes
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(so + r * 128 + g * 16 + ((j ^ t4) * 4)) =
              make_float4(o[q][2 * j][c], o[q][2 * j][c + 2], o[q][2 * j + 1][c], o[q][2 * j + 1][c + 2]);
      }
    }
    __syncthreads();
    const bool whole = seg.first && seg.last;
    if (tid == 0) {
      if (seg.first) p.range[seg.unit].x = blockIdx.x;
      if (seg.last) p.range[seg.unit].y = blockIdx.x;
    }
    for (int x = tid; x < rows * 32; x += kWarps * 32) {   // four dimensions of one row
      const int r = x >> 5, d = (x & 31) * 4;
      const int at_d = (x & 31) >> 2, piece = ((x & 3) ^ ((r >> 1) & 3)) * 4;   // where they lie
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][r].x);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml[w][r];
        const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
        const float4 ov = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (w * R + r) * 128 + at_d * 16 + piece);
        L += f * v.y;
        acc.x += f * ov.x; acc.y += f * ov.y; acc.z += f * ov.z; acc.w += f * ov.w;
      }
      if (whole) {
        const int row = seg.rt * R + r, node = row / p.G;
        const size_t grow = ((size_t)s * p.T + node) * p.Hq + kvh * p.G + row - node * p.G;
        const float inv = L > 0.f ? p.v_mul / L : 0.f;
        uint2 w2;
        w2.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        w2.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(p.out + grow * 128 + d) = w2;
        if (p.lse && d == 0) p.lse[grow] = kv4_lse(M, L, kPShift);
      } else {
        const size_t at = (size_t)kv4_slot(blockIdx.x, seg.first) * R + r;
        *reinterpret_cast<float4*>(p.o_part + at * 128 + d) = acc;
        if (d == 0) p.ml_part[at] = make_float2(M, L);
      }
    }
    fence_proxy_async();   // the rings were written by ordinary stores: order them before the next copies
    __syncthreads();
  }
}

// One warp per query row of a cut unit: the parts in the order of the CTAs.  What bounds it is
// latency, so the first parts' outputs are on their way before their weights are known.
constexpr int kCombRows = 8, kCombParts = 8;   // rows of a CTA; parts brought at once
__global__ void __launch_bounds__(kCombRows * 32) kv4_combine_kernel(const Kv4AttnParams p, int ctas) {   // CTAs of a sequence
  const int s = blockIdx.x / ctas, at = (int)(blockIdx.x - s * ctas) * kCombRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int node = at / p.Hq, head = at - node * p.Hq;
  const int kvh = head / p.G, r = node * p.G + head - kvh * p.G;
  const int rt = r / p.R, in_tile = r - rt * p.R;
  pdl_wait();
  pdl_trigger();
  if (node >= p.T) return;
  const size_t row = ((size_t)s * p.T + node) * p.Hq + head;
  const int2 range = p.range[(s * p.Hkv + kvh) * p.nrt + rt];
  const int c0 = max(range.x, 0), c1 = min(range.y, p.n_cta - 1);
  const int parts = c1 - c0 + 1;
  if (parts <= 1) return;
  auto slot = [&](int i) { return (size_t)kv4_slot(c0 + i, i == 0) * p.R + in_tile; };
  float4 o[kCombParts];
  auto bring = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kCombParts; ++i)
      o[i] = i0 + i < parts ? reinterpret_cast<const float4*>(p.o_part + slot(i0 + i) * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // lane i holds part i's maximum and sum (parts behind the 32nd in turn)
  float2 v = lane < parts ? p.ml_part[slot(lane)] : make_float2(-INFINITY, 0.f);
  bring(0);
  float M = v.x;
  for (int i = 32 + lane; i < parts; i += 32) M = fmaxf(M, p.ml_part[slot(i)].x);
  M = warp_max(M);
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0;;) {
    const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
    L += warp_sum(f * v.y);
    const int end = min(i0 + 32, parts);
    for (int j = i0;;) {
#pragma unroll
      for (int i = 0; i < kCombParts; ++i) {   // parts behind the last: 0 times 0
        const float fi = __shfl_sync(0xffffffffu, f, (j + i) & 31);
        acc.x += fi * o[i].x; acc.y += fi * o[i].y; acc.z += fi * o[i].z; acc.w += fi * o[i].w;
      }
      if ((j += kCombParts) >= end) break;
      bring(j);
    }
    if ((i0 += 32) >= parts) break;
    v = i0 + lane < parts ? p.ml_part[slot(i0 + lane)] : make_float2(-INFINITY, 0.f);
    bring(i0);
  }
  const float inv = L > 0.f ? p.v_mul / L : 0.f;
  uint2 w2;
  w2.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  w2.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(p.out + row * 128)[lane] = w2;
  if (p.lse && lane == 0) p.lse[row] = kv4_lse(M, L, p.shift);
}

// ------------------------------------------------------------------------------- host
int launch_kv4_attn_few(Kv4AttnParams p, cudaStream_t st) {
  p.shift = kPShift;
  const size_t merge = (size_t)kWarps * p.R * 128 * 4;
  const size_t smem = merge > kRingBytes ? merge : kRingBytes;
  if (p.R == 8) {
    if (ensure_dynamic_smem(kv4_attn_kernel<1>, smem) != cudaSuccess) return DF_ERR_CUDA;
    launch_k(kv4_attn_kernel<1>, dim3(p.n_cta), dim3(kWarps * 32), smem, st, p);
  } else {
    if (ensure_dynamic_smem(kv4_attn_kernel<2>, smem) != cudaSuccess) return DF_ERR_CUDA;
    launch_k(kv4_attn_kernel<2>, dim3(p.n_cta), dim3(kWarps * 32), smem, st, p);
  }
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

namespace {
// Rows, stage and grid of a call, by its rows per kv head.  Over 8 sequences of 16000 slots, 8
// kv heads: 8 rows take 39 us in a tile of 8, 53 us in one of 16, 78 us on tcgen05; 16 rows
// take 56 us in a tile of 16, 80 us on tcgen05; 32 rows take 95 us in two tiles of 16, 81 us on
// tcgen05.  A share of fewer stages than warps would leave warps idle.
void kv4_attn_plan(int T, int G, Kv4AttnParams& p) {
  const long long rows = (long long)T * G;
  p.R = rows <= 8 ? 8 : rows <= 16 ? 16 : 256;
  p.nrt = (int)((rows + p.R - 1) / p.R);
  p.last_single = p.R == 256 && rows - (long long)(p.nrt - 1) * p.R <= 128;
  p.stage_log2 = p.R == 256 ? 7 : 5;
  p.min_stages = p.R == 256 ? 2 : kWarps;
  p.change_step = p.R == 256 ? 1 : 2;
  p.n_cta = num_sms() * (p.R == 256 ? 1 : 2);
}
size_t up16(size_t x) { return (x + 15) & ~(size_t)15; }
}  // namespace

size_t kv4_attn_scratch_bytes(int b, int T, int Hq, int Hkv) {
  Kv4AttnParams p{};
  kv4_attn_plan(T, Hq / Hkv, p);
  const size_t units = (size_t)b * Hkv * p.nrt;
  return up16((size_t)2 * p.n_cta * p.R * (128 * 4 + 8)) + up16(units * sizeof(int2));
}

int launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t st) {
  Kv4AttnParams p{};
  p.p = a.p;
  p.b = a.b; p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.cap = a.cap; p.W = (a.T + 31) / 32;
  p.g_magic = p.G > 1 ? (uint32_t)(((1ull << 32) + p.G - 1) / p.G) : 0u;
  p.q = a.q; p.cache_len = a.cache_len; p.anc = a.anc;
  p.scale2 = ldexpf(a.scale * 1.4426950408889634f, a.k_exp);
  p.v_mul = ldexpf(1.f, a.v_exp);
  p.out = a.out; p.lse = a.lse; p.status = a.status;
  kv4_attn_plan(a.T, p.G, p);
  const size_t slots = (size_t)2 * p.n_cta;
  p.o_part = static_cast<float*>(a.scratch);
  p.ml_part = reinterpret_cast<float2*>(p.o_part + slots * p.R * 128);
  p.range = reinterpret_cast<int2*>(static_cast<unsigned char*>(a.scratch) + up16(slots * p.R * (128 * 4 + 8)));
  {
    DF_TRACE("kv4_attention", st);
    const int rc = p.R == 256 ? launch_kv4_attn_tc(p, st) : launch_kv4_attn_few(p, st);
    if (rc != DF_OK) return rc;
  }
  p.shift = p.R == 256 ? kTcShift : kPShift;
  DF_TRACE("kv4_combine", st);
  const int ctas = (a.T * a.Hq + kCombRows - 1) / kCombRows;
  launch_k(kv4_combine_kernel, dim3((unsigned)(a.b * ctas)), dim3(kCombRows * 32), 0, st, p, ctas);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
