// The attention weight that given query rows lay on every slot of a KV cache held in 4 bits:
//   score_out[j] = decay * score[j] + sum over the rows that see j of exp(scale q k_j - lse).
//
// On the tcgen05 tensor cores as S^T = K Q^T: a block of 128 keys is the operand of 128 rows and
// the query rows are the columns, so that a thread owns a key (its TMEM lane) and sums its weight
// along its own columns: no exchange, no atomics, and the order of every sum is fixed.
//
// What bounds it is the decoding (1000 cycles for a block) beside the exponentials, which share
// the issue slots: 64 rows of each of 8 sequences of 8607 to 16384 slots, 8 kv heads, take 36 us
// (with mma.sync and no tile of decoded keys 47 us); 36 rows over 4105 slots take 7 us, latency.
//
// Warp roles: one warp brings codes (untiled bulk copies), 8 warps decode them into 128-byte-
// swizzled fp16 tiles, one issues the products, two groups of 4 warps take the blocks in turn,
// each with two buffers of 128 TMEM columns.  A unit is one (sequence, kv head); with more than
// 128 rows it is walked again for the next ones, which add to what the first have written.
#include <math.h>

#include "kv4_attn.cuh"
#include "kv4_tc.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {

constexpr int kExpWarps = 8, kDecWarps = 8;
constexpr int kDec0 = kExpWarps, kMmaWarp = kDec0 + kDecWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
constexpr int kKB = 128;                       // keys of a block; launch: stage_log2
constexpr int kRows = 128;                     // query rows of a pass
constexpr int kBufs = 512 / kRows;             // TMEM buffers of a block's products
constexpr uint32_t kTile = 128 * 128 * 2;      // one fp16 tile: two slabs of 64 columns
constexpr uint32_t kQSlab = kRows * 128;       // Q: two slabs of 64 dimensions
constexpr int kTiles = 3, kRaw = 10, kSegs = 4; // rings of decoded tiles, codes, passes
constexpr int kRawScales = kKB * kKv4Codes;    // codes [key][64], then scales [key][8]
constexpr int kRawBytes = kRawScales + kKB * kKv4Scales;

struct Kv4WeightsParams {
  Kv4WeightsArgs a;
  Kv4AttnParams walk;   // its units are (sequence, kv head)
  int G;
  float scale2;         // scale * log2(e) * 2^k_exp
};

struct Pass {           // rows r0 .. of a unit over a CTA's part of its keys
  int s, kvh, key0, count;   // first key, blocks
  int len, base;             // slots seen, slots before the first row's own
  int r0, total;             // first row of the pass, rows of the unit
  int held;                  // kv4_held
};

__global__ void __launch_bounds__(kThreads, 1) kv4_weights_kernel(const __grid_constant__ Kv4WeightsParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* q_smem = smem;
  unsigned char* t_smem = q_smem + 2 * kQSlab;
  unsigned char* raw_smem = t_smem + kTiles * kTile;
  __shared__ __align__(8) uint64_t r_full[kRaw], r_empty[kRaw], t_full[kTiles], t_empty[kTiles], s_full[kBufs], s_empty[kBufs];
  __shared__ __align__(8) uint64_t q_full, unit_done, drain, seg_full[kSegs], seg_empty[kSegs];
  __shared__ Pass passes[kSegs];
  __shared__ __align__(16) float row_s[kRows], row_nl[kRows];   // raw score -> log2 units, -lse in log2 units
  __shared__ uint32_t tmem_slot;

  const Kv4WeightsArgs& a = p.a;
  int* const status = a.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], kDecWarps); }
    for (int i = 0; i < kTiles; ++i) { mbar_init(&t_full[i], kDecWarps); mbar_init(&t_empty[i], 1); }
    for (int i = 0; i < kBufs; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], kExpWarps / 2); }
    for (int i = 0; i < kSegs; ++i) { mbar_init(&seg_full[i], 1); mbar_init(&seg_empty[i], kLoadWarp); }
    mbar_init(&q_full, kExpWarps);
    mbar_init(&unit_done, kExpWarps);
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
  bool ok = true;
  int n_pass = 0;   // passes taken so far
  auto wait = [&](uint64_t* bar, int parity, int id) {
    ok = __all_sync(0xffffffffu, ok && kv4_wait(bar, parity & 1, status, id));
    return ok;
  };
  // Passes from the loading warp to the others; one of 0 blocks ends them.
  auto take = [&]() -> Pass {
    wait(&seg_full[n_pass % kSegs], n_pass / kSegs, 70);
    const Pass x = passes[n_pass % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[n_pass % kSegs]);
    ++n_pass;
    return x;
  };
  auto columns = [](const Pass& x) { return min(kRows, (max(1, x.total - x.r0) + 31) & ~31); };   // of the products

  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- bring codes
    int j = 0;   // tiles so far
    Kv4Walk walk;
    Kv4Seg sg;
    const int held = kv4_held(status);
    bool more = walk.init(p.walk, blockIdx.x, lane);
    while (ok) {
      Pass x{};
      x.r0 = 0;
      x.held = held;
      if (more) more = walk.next(p.walk, sg);
      if (more) {
        x.s = sg.s;
        x.kvh = sg.kvh;
        x.key0 = sg.tile0 * kKB;
        x.count = sg.count;
        const int32_t* src = a.src_slot + (size_t)x.s * a.max_src;
        int mine = a.src_slot && lane < a.max_src ? src[lane] : 0;   // of the list, beside the lengths
        const int n = a.n_rows ? a.n_rows[x.s] : a.T;
        x.len = kv4_len(a.cache_len, x.s, 0, a.cap, status);
        if (x.len < 0) continue;
        x.base = x.len - n;
        // rows that the sequence, the tree and the list have, and nodes that the tree has
        bool fits = n >= 0 && n <= a.T && n <= x.len && (!a.src_slot || n <= a.max_src + 1);
        if (fits && a.src_slot)
          for (int r = lane; r < n - 1 && fits; r += 32) {
            if (r >= 32) mine = src[r];
            fits = (uint32_t)mine - (uint32_t)x.base < (uint32_t)a.T;
          }
        if (!__all_sync(0xffffffffu, fits)) {
          if (lane == 0) set_status(status, DF_ERR_ARG, x.s);
          continue;
        }
        x.total = n * p.G;
      }
      const size_t row = ((size_t)x.s * a.Hkv + x.kvh) * a.cap + x.key0;
      for (; ok; x.r0 += kRows) {
        if (!wait(&seg_empty[n_pass % kSegs], (n_pass / kSegs) ^ 1, 71)) break;
        if (lane == 0) {
          passes[n_pass % kSegs] = x;
          mbar_arrive(&seg_full[n_pass % kSegs]);
        }
        __syncwarp();
        ++n_pass;
        for (int i = 0; i < x.count; ++i, ++j) {
          const int st = j % kRaw;
          if (!wait(&r_empty[st], (j / kRaw) ^ 1, 72)) break;
          if (lane == 0) {
            const int n = min(kKB, a.cap - x.key0 - i * kKB);   // a multiple of 8
            unsigned char* to = raw_smem + st * kRawBytes;
            mbar_arrive_expect_tx(&r_full[st], n * (kKv4Codes + kKv4Scales));
            bulk_load(to, a.p.kc + (row + i * kKB) * kKv4Codes, n * kKv4Codes, &r_full[st]);
            bulk_load(to + kRawScales, a.p.ks + (row + i * kKB) * kKv4Scales, n * kKv4Scales, &r_full[st]);
          }
          __syncwarp();
        }
        if (x.r0 + kRows >= x.total) break;
      }
      if (x.count == 0) break;
    }
    // every copy must have landed before the CTA may exit
    for (int i = max(0, j - kRaw); i < j; ++i) kv4_wait(&r_full[i % kRaw], (i / kRaw) & 1, nullptr, 0);
  } else if (warp >= kDec0 && warp < kMmaWarp) {
    // ---------------------------------------------------------------- decode
    // Half a key per lane: two 16-byte pieces (32 dimensions each), in an order that spreads the
    // lanes of a phase over all banks, both when reading and when writing.
    const int key = (warp - kDec0) * 16 + (lane & 15);
    const int c0 = ((lane >> 4) + (lane >> 1)) & 3, c1 = c0 ^ 2;   // the two pieces
    // swizzled place of a piece's first 8 dimensions; the e-th 8 lie at the place XOR 16 e
    auto place = [&](int c) { return key * 128 + (c >> 1) * (kTile / 2) + ((((c & 1) * 4) ^ (key & 7)) * 16); };
    const int src0 = key * kKv4Codes + c0 * 16, src1 = key * kKv4Codes + c1 * 16;
    const int sc0 = kRawScales + key * kKv4Scales + c0 * 2, sc1 = kRawScales + key * kKv4Scales + c1 * 2;
    const uint32_t dst0 = smem_u32(t_smem) + place(c0), dst1 = smem_u32(t_smem) + place(c1);
    int st = 0, st_phase = 0, buf = 0, buf_phase = 0;
    while (true) {
      const Pass x = take();
      if (!ok || x.count == 0) break;
      for (int i = 0; i < x.count; ++i) {
        if (!wait(&r_full[st], st_phase, 73) || !wait(&t_empty[buf], buf_phase ^ 1, 74)) break;
        const unsigned char* from = raw_smem + st * kRawBytes;
        const uint4 v0 = *reinterpret_cast<const uint4*>(from + src0), v1 = *reinterpret_cast<const uint4*>(from + src1);
        const uint32_t two0 = *reinterpret_cast<const uint16_t*>(from + sc0), two1 = *reinterpret_cast<const uint16_t*>(from + sc1);
        kv4_decode_piece(v0, two0, dst0 + buf * kTile);
        kv4_decode_piece(v1, two1, dst1 + buf * kTile);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&t_full[buf]);
          mbar_arrive(&r_empty[st]);
        }
        if (++st == kRaw) { st = 0; st_phase ^= 1; }
        if (++buf == kTiles) { buf = 0; buf_phase ^= 1; }
      }
      if (!ok) break;
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    // Whatever an MMA's operands depend on is made warp-uniform (a reduction's result is).
    const bool leader = elect_one();
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(q_smem)), k_desc = sdesc_kmajor_sw128(smem_u32(t_smem));
    int buf = 0, phase = 0, j = 0;   // tile ring; blocks so far
    while (true) {
      const Pass x = take();
      const int count = __reduce_max_sync(0xffffffffu, x.count);
      if (!ok || count == 0) break;
      const uint32_t idesc = idesc_f16_f32(128, __reduce_max_sync(0xffffffffu, columns(x)), false);
      if (!wait(&q_full, n_pass - 1, 75)) break;
      for (int i = 0; i < count; ++i, ++j) {
        if (!wait(&t_full[buf], phase, 76) || !wait(&s_empty[j % kBufs], (j / kBufs) ^ 1, 77)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t kd = k_desc + buf * (kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t step = (kk & 3) * (32 >> 4);
            mma_bf16(tm + (j % kBufs) * kRows, kd + (kk >> 2) * (kTile / 2 >> 4) + step, q_desc + (kk >> 2) * (kQSlab >> 4) + step, idesc,
                     kk > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[j % kBufs]);
          mma_commit(&t_empty[buf]);
        }
        __syncwarp();
        if (++buf == kTiles) { buf = 0; phase ^= 1; }
      }
      if (!ok) break;
    }
    // TMEM is freed and the CTA ends only behind the MMAs issued.  They are done where every block
    // was summed, but the weights' warps may have given up when this role had nothing left to issue.
    if (j > 0) {
      if (leader) mma_commit(&drain);
      __syncwarp();
      kv4_wait(&drain, 0, nullptr, 0);
    }
  } else {
    // ---------------------------------------------------------------- weights
    const int w = warp >> 2, my_key = (warp & 3) * 32 + lane;
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int j = 0;   // blocks so far
    while (true) {
      const Pass x = take();
      if (!ok || x.count == 0) break;
      const int cols = columns(x);
      // every product and every read of the rows of the previous pass is done
      if (n_pass > 1 && !wait(&unit_done, n_pass - 2, 78)) break;
      // Q, four lanes a row, into its swizzled places; rows behind the last are zeros
      for (int r = threadIdx.x >> 2; r < cols; r += kExpWarps * 8) {
        const int q4 = lane & 3, rr = x.r0 + r, row = rr / p.G;
        int node = -1;
        if (rr < x.total) node = !a.src_slot ? row : row == 0 ? 0 : a.src_slot[(size_t)x.s * a.max_src + row - 1] - x.base;
        const size_t grow = ((size_t)x.s * a.T + max(node, 0)) * a.Hq + x.kvh * p.G + rr - row * p.G;
        const float lse = node >= 0 ? a.lse[grow] : -INFINITY;
        uint32_t f[8][2];
        float back;
        load_q(a.q + grow * 128, node >= 0, q4, f, back);
        // a NaN belongs to the slots that the row sees: it goes in as the row's numbers, which the mask covers
        if (lse != lse)
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c][0] = f[c][1] = 0x7FFF7FFFu;
        unsigned char* to = q_smem + (q4 >> 1) * kQSlab + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(to + ((((q4 & 1) * 4 + c) ^ (r & 7)) * 16)) =
              make_uint4(f[2 * c][0], f[2 * c][1], f[2 * c + 1][0], f[2 * c + 1][1]);
        if (q4 == 0) {
          row_s[r] = fmaxf(p.scale2 * back, 1.17549435e-38f);   // a masked score times it stays -inf; a real one is as good as 0
          // a row that saw nothing adds 2^(-inf) = 0 everywhere; finite above, for a masked score to stay -inf
          row_nl[r] = lse == -INFINITY ? -INFINITY : fminf(lse * -1.4426950408889634f, 3.402823466e38f);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      if (!wait(&q_full, n_pass - 1, 79)) break;
      // held: give up while the issuer is at work, or has left its role behind the last block
      if (x.held && !(ok = kv4_hold_clear(status, 81, lane))) break;
      const size_t plane = ((size_t)x.s * a.Hkv + x.kvh) * a.cap;
      // what the slot has already, brought a block ahead; a slot of the rows' own starts at 0
      const float* from = x.r0 > 0 ? a.score_out : a.score;
      const float keep = x.r0 > 0 ? 1.f : a.decay;
      const int known = x.r0 > 0 ? x.len : x.base;
      auto bring = [&](int i) {
        const int key = x.key0 + i * kKB + my_key;
        return i < x.count && key < known ? from[plane + key] : 0.f;
      };
      float next = bring((j & 1) ^ w);
      for (int i = 0; i < x.count; ++i, ++j) {
        if ((j & 1) != w) continue;
        const int key = x.key0 + i * kKB + my_key;
        const float old = key < known ? keep * next : 0.f;
        next = bring(i + 2);
        if (!wait(&s_full[j % kBufs], j / kBufs, 80)) break;
        tc_fence_after();
        // Row r (of head r % G of node r / G) sees the slots up to its own: the first column that
        // sees this key.
        const bool edge = x.key0 + (i + 1) * kKB > x.base + 1;
        const int seen = edge ? max(0, min(key - x.base, a.T)) * p.G - x.r0 : 0;
        uint64_t mass[2] = {0, 0};
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          float v[32];
          tmem_ld32(at + (j % kBufs) * kRows + c, v);
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e < seen) v[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(&row_s[c + e]), n4 = *reinterpret_cast<const float4*>(&row_nl[c + e]);
            float y[4];
            unpack2(fma2(pack2(v[e], v[e + 1]), pack2(s4.x, s4.y), pack2(n4.x, n4.y)), y[0], y[1]);
            unpack2(fma2(pack2(v[e + 2], v[e + 3]), pack2(s4.z, s4.w), pack2(n4.z, n4.w)), y[2], y[3]);
            mass[0] = add2(mass[0], pack2(ex2_approx(y[0]), ex2_approx(y[1])));
            mass[1] = add2(mass[1], pack2(ex2_approx(y[2]), ex2_approx(y[3])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[j % kBufs]);
        float m0, m1;
        unpack2(add2(mass[0], mass[1]), m0, m1);
        if (key < x.len) a.score_out[plane + key] = old + (m0 + m1);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_done);
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

int launch_kv4_weights(const Kv4WeightsArgs& a, cudaStream_t st) {
  DF_TRACE("kv4_attention_weights", st);
  Kv4WeightsParams p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.scale2 = ldexpf(a.scale * 1.4426950408889634f, a.k_exp);
  Kv4AttnParams& w = p.walk;
  w.b = a.b; w.Hkv = a.Hkv; w.cap = a.cap; w.cache_len = a.cache_len;
  w.T = 0; w.G = 1; w.R = 1; w.nrt = 1;
  w.stage_log2 = 7;
  w.min_stages = 1;
  w.change_step = 1;
  w.n_cta = num_sms();
  const size_t smem = 1024 + 2 * kQSlab + kTiles * kTile + kRaw * kRawBytes;
  if (ensure_dynamic_smem(kv4_weights_kernel, smem) != cudaSuccess) return DF_ERR_CUDA;
  launch_k(kv4_weights_kernel, dim3(w.n_cta), dim3(kThreads), smem, st, p);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
