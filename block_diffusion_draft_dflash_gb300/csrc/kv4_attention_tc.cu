// Tree attention over a KV cache held in 4 bits on the tcgen05 tensor cores.
//
// Query rows of one (sequence, kv head) lie node-major (a node's heads next to one another)
// in tiles of 128.  A CTA runs two streams side by side, each with its own S, P and O in TMEM
// and its own softmax warpgroup, so that one stream's exponentials run under the other's
// products:
//   pair    the unit has more than 128 rows: the streams are two row tiles, and a stage is one
//           block of 128 keys, decoded once for both;
//   single  it has at most 128: both streams hold the same rows, and a stage is two blocks of
//           128 keys, one for each.  They hold the same rows in the same TMEM lanes, so each
//           reads both outputs and writes half of the merged one's columns.
// Either way a stage is two S = Q K^T, two softmax blocks and two O += P V, which makes equal
// shares of stages (kv4_attn.cuh) equal shares of work.
//
// Per block:  S in fp32 (fp16 operands: the cache's values are fp16 numbers, kv4.cuh, so the
// products are exact), softmax with a running maximum that moves only when a block raises it
// by more than 2^8, P as fp16 over its own S, O += P V.  P is an operand of the tensor cores, so it
// has 16 bits: fp16 keeps 11 significant ones where bf16 would keep 8, more than the output has, and
// sums of P are taken before the rounding.  One thread owns one row of a stream and
// holds its 128 scores in registers (given to it by the decoding warps): S is read once, and
// no exchange between threads is needed.
//
// What bounds it is a stream's way round: for a stage of two row tiles the row maxima take 600
// cycles, the exponentials 1400 (both streams share the special function units and the issue
// slots with the decoding warps), 300 until the issuer has seen P, 1500 for PV and the next S
// beside the other stream's, 250 until S is seen: 4200, of which the tensor cores work 2050.
// Trees of 257 nodes over 2 sequences of 7192 and 8192 slots, 32 heads on 8: 92 us (65 GFLOP).
//
// Warp roles: 4 softmax / epilogue warps and an MMA issuer for each stream, 8 decoding warps and
// one warp that brings the codes.  Codes arrive by untiled bulk copies (a block's rows are
// contiguous); the decoding warps write K and V alike as [key][dim] in 128-byte-swizzled rows,
// which S = Q K^T reads as a K-major operand and O += P V as an MN-major one.
//
// A stream's issue order is fixed: S(0), then PV(i), S(i+1).  One thread's MMAs run in order, so
// S(i+1) may take the place of P(i), and its completion implies that of PV(i): O may be
// rescaled then.
// setmaxnreg and calls do not go together: ptxas cannot allocate registers for both
#define KV4_COLD DF_DEV
#include "kv4_attn.cuh"
#include "kv4_tc.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {

constexpr int kDecWarps = 8;
constexpr int kDec0 = 8;                       // first decoding warp, behind 4 softmax warps of each stream
constexpr int kMmaWarp = kDec0 + kDecWarps, kLoadWarp = kMmaWarp + 2;   // an MMA warp for each stream
constexpr int kThreads = (kLoadWarp + 2) * 32;   // the last warp only fills its warpgroup
constexpr int kKB = 128;                       // keys of a block
constexpr uint32_t kSCol = 0, kOCol = 256;     // S (then P) of stream w at 128 w, O at 256 + 128 w
constexpr uint32_t kTile = 128 * 128 * 2;      // one fp16 tile: two slabs of 64 columns
constexpr int kTiles = 3;                      // ring of decoded tiles
constexpr int kRaw = 6;                        // ring of codes, one tile each
constexpr int kSegs = 4;                       // ring of units
constexpr int kRawScales = kKB * kKv4Codes;    // codes [key][64], then scales [key][8]
constexpr int kRawBytes = kRawScales + kKB * kKv4Scales;

// Shared-memory matrix descriptor, MN-major operand, 128-byte swizzle: rows of 64 fp16 along
// MN; the next 64 follow a slab (half a tile) later, the next 8 rows (along K) 1024 bytes later.
DF_DEV uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)((kTile / 2) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// The 32 query rows from `first` on of a (sequence, kv head): node-major, a node's heads next
// to one another.  One division for the first, a multiplication for each other.
struct Rows {
  int node0, rem0;
  long long base;   // index in q, out and lse of the sequence's first row of the kv head
  DF_DEV Rows(const Kv4AttnParams& p, int s, int kvh, int first) {
    node0 = first / p.G;
    rem0 = first - node0 * p.G;
    base = (long long)s * p.T * p.Hq + kvh * p.G;
  }
  DF_DEV int step(const Kv4AttnParams& p, int x) const { return p.g_magic ? __umulhi(x, p.g_magic) : x; }
  DF_DEV int node(const Kv4AttnParams& p, int k) const { return node0 + step(p, rem0 + k); }
  DF_DEV int at(const Kv4AttnParams& p, int k) const {   // behind `base`; -1: behind the last row
    const int q = step(p, rem0 + k), n = node0 + q;
    return n < p.T ? n * p.Hq + (rem0 + k - q * p.G) : -1;
  }
};

// 32 bits of visibility (keys j0 .. j0+31) of the lane's row, `first` being the warp's first row.
// Out of line, like what it calls: a block at the mask's edge is rare.
DF_DEV uint32_t row_bits(const Kv4AttnParams& p, const Kv4Seg& sg, int first, int lane, int j0) {
  const int node = Rows(p, sg.s, sg.kvh, first).node(p, lane);
  if (node >= p.T) return 0u;
  return kv4_see_bits(p.anc ? p.anc + ((size_t)sg.s * p.T + node) * p.W : nullptr, p.W, sg.N, j0, node, sg.len);
}

// Registers move to the softmax warps.  What a block has is what it was launched with (checked
// at the launch): kWarps x 32 x kLaunchRegs.  A warpgroup changes its share as a whole.
constexpr int kWarps = kThreads / 32, kLaunchRegs = 96, kSoftRegs = 168, kDecRegs = 40, kRestRegs = 64;
static_assert(kWarps == 20 && 8 * kSoftRegs + 8 * kDecRegs + 4 * kRestRegs <= kWarps * kLaunchRegs, "registers");
template <int N> DF_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> DF_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// O of the warp's rows times alpha, 8 columns at a time: few registers are free then.
DF_DEV void scale_rows(uint32_t oaddr, float alpha) {
#pragma unroll 1
  for (int c = 0; c < 128; c += 8) {
    float o[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
                 : "r"(oaddr + c));
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= alpha;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(oaddr + c), "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7])
                 : "memory");
  }
}

// Cycles that stream 1 waits before its first product.  Chains gain as trees do once a unit has
// several stages: 2 x 257 nodes over 8000 slots 89.9 us (90.2 without), 16 x 16 nodes 80.6 (81.1),
// 4 x 32 nodes 31.5 (32.0); a unit of one stage only waits: 16 nodes over 200 slots 13.0 us (12.3).
constexpr int kStagger = 1500;
DF_DEV void pause(int cycles) {
  const long long t0 = clock64();
  while (clock64() - t0 < cycles) {}
}

__global__ void __launch_bounds__(kThreads, 1) kv4_attn_tc_kernel(const __grid_constant__ Kv4AttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* q_smem = smem;                       // one tile per stream
  unsigned char* t_smem = q_smem + 2 * kTile;         // kTiles decoded tiles
  unsigned char* raw_smem = t_smem + kTiles * kTile;  // kRaw tiles of codes
  __shared__ __align__(8) uint64_t r_full[kRaw], r_empty[kRaw], t_full[kTiles], t_empty[kTiles];
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drain[2], ml_full[2], merged;
  __shared__ __align__(8) uint64_t seg_full[kSegs], seg_empty[kSegs];
  __shared__ Kv4Seg segs[kSegs];
  __shared__ float2 pair_ml[2][128];   // single: maximum and sum of a stream's rows
  __shared__ uint32_t tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], kDecWarps); }
    for (int i = 0; i < kTiles; ++i) { mbar_init(&t_full[i], kDecWarps); mbar_init(&t_empty[i], 2); }
    for (int i = 0; i < 2; ++i) { mbar_init(&q_full[i], 4); mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4); mbar_init(&o_full[i], 1); mbar_init(&ml_full[i], 4); }
    mbar_init(&merged, 8);
    for (int i = 0; i < kSegs; ++i) { mbar_init(&seg_full[i], 1); mbar_init(&seg_empty[i], kLoadWarp); }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) { tmem_alloc(&tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_slot;
  // Units of this CTA's share, from the loading warp to the others; a unit of 0 stages ends them.
  bool ok = true;
  int n_seg = 0;   // units taken so far
  auto take = [&]() -> const Kv4Seg& {
    ok = __all_sync(0xffffffffu, kv4_wait(&seg_full[n_seg % kSegs], (n_seg / kSegs) & 1, p.status, 59));
    return segs[n_seg++ % kSegs];
  };
  auto give_back = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[(n_seg - 1) % kSegs]);
  };

  if (warp >= kMmaWarp) regs_down<kRestRegs>();
  if (warp > kLoadWarp) {
    // nothing to do
  } else if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- bring codes
    int j = 0;          // tiles so far
    int st = 0, phase = 0;
    Kv4Walk walk;
    Kv4Seg sg;
    sg.held = kv4_held(p.status);
    bool more = walk.init(p, blockIdx.x, lane);
    while (ok) {
      sg.count = 0;
      if (more) more = walk.next(p, sg);
      ok = __all_sync(0xffffffffu, kv4_wait(&seg_empty[n_seg % kSegs], ((n_seg / kSegs) & 1) ^ 1, p.status, 58));
      if (!ok) break;
      if (lane == 0) {
        segs[n_seg % kSegs] = sg;
        mbar_arrive(&seg_full[n_seg % kSegs]);
      }
      __syncwarp();
      ++n_seg;
      if (sg.count == 0) break;
      const size_t plane = ((size_t)sg.s * p.Hkv + sg.kvh) * p.cap;
      const bool single = sg.single;
      const int tiles = sg.count * (single ? 4 : 2), block0 = sg.tile0 * (single ? 2 : 1);
      for (int x = 0; x < tiles; ++x) {
        ok = __all_sync(0xffffffffu, kv4_wait(&r_empty[st], phase ^ 1, p.status, 60));
        if (!ok) break;
        if (lane == 0) {   // two copies a tile: what a bulk copy costs hardly depends on its size
          // tiles of a pair's block: K, V; of a single's two blocks: Ka, Kb, Va, Vb
          const bool is_v = single ? (x >> 1) & 1 : x & 1;
          const int key0 = (block0 + (single ? (x >> 2) * 2 + (x & 1) : x >> 1)) * kKB;
          const int n = max(0, min(kKB, p.cap - key0));   // a multiple of 8; 0: a single's block behind the cache
          unsigned char* to = raw_smem + st * kRawBytes;
          const size_t row = plane + key0;
          mbar_arrive_expect_tx(&r_full[st], n * (kKv4Codes + kKv4Scales));
          if (n > 0) {
            bulk_load(to, (is_v ? p.p.vc : p.p.kc) + row * kKv4Codes, n * kKv4Codes, &r_full[st]);
            bulk_load(to + kRawScales, (is_v ? p.p.vs : p.p.ks) + row * kKv4Scales, n * kKv4Scales, &r_full[st]);
          }
        }
        __syncwarp();
        ++j;
        if (++st == kRaw) { st = 0; phase ^= 1; }
      }
    }
    // every copy must have landed before the CTA may exit
    for (int i = max(0, j - kRaw); i < j; ++i) kv4_wait(&r_full[i % kRaw], (i / kRaw) & 1, nullptr, 0);
  } else if (warp >= kDec0 && warp < kMmaWarp) {
    // ---------------------------------------------------------------- decode
    regs_down<kDecRegs>();
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
      const Kv4Seg& sg = take();
      const int tiles = sg.count * (sg.single ? 4 : 2);
      give_back();
      if (!ok || tiles == 0) break;
      for (int x = 0; x < tiles; ++x) {
        ok = kv4_wait(&r_full[st], st_phase, p.status, 61) && kv4_wait(&t_empty[buf], buf_phase ^ 1, p.status, 62);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
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
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ---------------------------------------------------------------- MMA issuers
    // Warp w issues the products of stream w: while one waits on a barrier the other's MMAs run.
    // A warp runs in lockstep and one elected lane issues.  Whatever an MMA's operands depend on
    // is made warp-uniform (a reduction's result is): operands in ordinary registers cost some
    // 100 cycles an MMA.
    constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false), idesc_pv = idesc_f16_f32(128, 128, true);
    const int w = __reduce_max_sync(0xffffffffu, warp - kMmaWarp);
    const bool leader = elect_one();
    bool issued = false;
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const uint32_t tm_s = tm + kSCol + w * 128, tm_o = tm + kOCol + w * 128;
    const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(q_smem + w * kTile)), k_desc = sdesc_kmajor_sw128(smem_u32(t_smem)),
                   v_desc = sdesc_mnmajor_sw128(smem_u32(t_smem));
    int slot = 0, phase = 0;   // ring place and phase of the segment's next stage's first tile
    int n_p = 0;               // P blocks seen so far
    // K-major: 16-byte units between the operands of two 16-wide steps
    constexpr uint32_t kStep = 32 >> 4, kSlab = (kTile / 2) >> 4;
    // the d-th tile from the stage's first: ring place, phase
    auto at = [&](int d, int& sl, int& ph) {
      sl = slot + d;
      ph = phase;
      while (sl >= kTiles) { sl -= kTiles; ph ^= 1; }
    };
    auto wait = [&](uint64_t* bar, int parity, int id) {
      ok = __all_sync(0xffffffffu, ok && kv4_wait(bar, parity & 1, p.status, id));
      return ok;
    };
    // a tile is free again when both streams have read it; one that a single stream reads is
    // released twice by it
    auto release = [&](int sl, int single) {
      mma_commit(&t_empty[sl]);
      if (single) mma_commit(&t_empty[sl]);
    };
    auto issue_s = [&](int sl, int single) {
      if (leader) {
        const uint64_t kd = k_desc + sl * (kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kSlab + (kk & 3) * kStep;
          mma_bf16(tm_s, q_desc + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[w]);
        release(sl, single);
      }
      __syncwarp();
      issued = true;
    };
    auto issue_pv = [&](int sl, int single, bool first, bool last) {
      if (leader) {
        const uint64_t vd = v_desc + sl * (kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // keys 16 kk ..: 16 rows of 128 bytes further
          mma_bf16_ts(tm_o, tm_s + kk * 8, vd + kk * (2048 >> 4), idesc_pv, (!first || kk > 0) ? 1u : 0u);
        }
        if (last) mma_commit(&o_full[w]);
        release(sl, single);
      }
      __syncwarp();
    };
    while (true) {
      // tiles of a stage: pair K, V; single Ka, Kb, Va, Vb
      const Kv4Seg& sg = take();
      const int single = __reduce_max_sync(0xffffffffu, sg.single), count = __reduce_max_sync(0xffffffffu, sg.count);
      give_back();
      if (!ok || count == 0) break;
      const int per = single ? 4 : 2, k_at = single ? w : 0, v_at = single ? 2 + w : 1;
      int sl, ph;
      // Q is there, and with it the epilogue has read the previous unit's O
      at(k_at, sl, ph);
      if (wait(&t_full[sl], ph, 63) && wait(&q_full[w], n_seg - 1, 63)) {
        tc_fence_after();
        // stream 1 starts half a block behind stream 0, and stays there: each has the
        // exponentials to itself while the other has the tensor core
        if (w == 1) pause(kStagger);
        issue_s(sl, single);
      }
      for (int i = 0; i < count && ok; ++i) {
        const bool more = i + 1 < count;
        int vs, vp;
        at(v_at, vs, vp);
        at(per, sl, ph);
        slot = sl;
        phase = ph;
        at(k_at, sl, ph);
        if (!wait(&t_full[vs], vp, 64) || !wait(&p_full[w], n_p++, 65)) break;
        tc_fence_after();
        // K is mostly there by now: then S follows without another wait
        const bool ready = __any_sync(0xffffffffu, mbar_test_wait(&t_full[sl], ph));
        issue_pv(vs, single, i == 0, !more);
        if (!more) break;
        if (!ready && !wait(&t_full[sl], ph, 66)) break;
        tc_fence_after();
        issue_s(sl, single);
      }
      if (!ok) break;
    }
    // TMEM is freed and the CTA ends only behind the MMAs issued.  They are done where every unit
    // was finished, but the softmax warps may have given up when this role had nothing left to issue.
    if (issued) {
      if (leader) mma_commit(&drain[w]);
      __syncwarp();
      kv4_wait(&drain[w], 0, nullptr, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax, epilogue
    // Stream w; the warp's rows are 32 (warp % 4) .. + 31 of it, a thread owns the row of its
    // TMEM lane.
    regs_up<kSoftRegs>();
    const int w = warp >> 2, r0 = (warp & 3) * 32;
    const uint32_t sp = tmem + ((uint32_t)r0 << 16) + kSCol + w * 128, oaddr = sp - kSCol + kOCol;
    int n_s = 0, n_single = 0;   // S blocks, single units so far
    while (true) {
      const Kv4Seg& sg = take();   // given back behind the epilogue
      if (!ok || sg.count == 0) break;
      const int row0 = sg.rt * p.R + (sg.single ? 0 : w * 128);   // the stream's first row
      const bool live = row0 + r0 < p.T * p.G;                    // the warp has a row
      if (sg.len == 0 && threadIdx.x == 0) set_status(p.status, DF_ERR_CAPACITY, sg.s);
      // Q into its swizzled places as bf16 (16 lanes a row), then every lane brings its own row to
      // fp16 by a power of two; every S of the previous unit is complete (o_full).  Everything
      // is unrolled: one warp's latency is what the first product waits for.
      float qs;
      {
        const Rows rows(p, sg.s, sg.kvh, row0 + r0);
        const int row_at = rows.at(p, lane);   // the lane's row behind rows.base, -1: none
        const uint32_t box = smem_u32(q_smem + w * kTile + r0 * 128);
        const int c = lane & 15;
        const df_bf16* q = p.q + rows.base * 128 + c * 8;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int lr = i * 2 + (lane >> 4);
          const int at = __shfl_sync(0xffffffffu, row_at, lr);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"   // no bytes: zeros
                       ::"r"(box + (c >> 3) * (kTile / 2) + lr * 128 + (((c & 7) ^ (lr & 7)) * 16)),
                         "l"(q + (size_t)max(at, 0) * 128), "r"(at < 0 ? 0 : 16) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        unsigned char* mine = q_smem + w * kTile + (r0 + lane) * 128;
        auto place = [&](int i) { return reinterpret_cast<uint4*>(mine + (i >> 3) * (kTile / 2) + (((i & 7) ^ (lane & 7)) * 16)); };
        uint4 v[16];
        float amax = 0.f, back;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = *place(i);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = max3(amax, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u)));
        }
        const float f = f16_row_factor(amax, back);
        qs = fmaxf(p.scale2 * back, 1.17549435e-38f);   // a masked score times it stays -inf; a real one is as good as 0
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = pack_f16x2(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xFFFF0000u) * f);
          *place(i) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[w]);
      }
      // no row of the stream has its mask before this key
      const int edge_key = sg.len == 0 ? 0 : p.anc ? sg.N : sg.N + min(p.T - 1, row0 / p.G) + 1;
      float m_run = -INFINITY, l = 0.f;   // the maximum in raw scores, the sum
      const int count = sg.count, stride = sg.single ? 2 * kKB : kKB;
      int key0 = (sg.tile0 * (sg.single ? 2 : 1) + (sg.single ? w : 0)) * kKB;
      for (int i = 0; i < count; ++i, ++n_s, key0 += stride) {
        ok = __all_sync(0xffffffffu, kv4_wait(&s_full[w], n_s & 1, p.status, 67));
        if (!ok) break;
        tc_fence_after();
        if (live) {
          // the mask first: its code is out of line, and the scores fill the registers
          const bool edge = key0 + kKB > edge_key;
          uint32_t adm[4] = {0u, 0u, 0u, 0u};
          if (edge) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {   // one copy of the code
              const uint32_t x = row_bits(p, sg, row0 + r0, lane, key0 + 32 * c);
              adm[0] = c == 0 ? x : adm[0]; adm[1] = c == 1 ? x : adm[1];
              adm[2] = c == 2 ? x : adm[2]; adm[3] = c == 3 ? x : adm[3];
            }
          }
          float sv[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(sp + c * 32, reinterpret_cast<float(&)[32]>(sv[c * 32]));
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (!((adm[e >> 5] >> (e & 31)) & 1u)) sv[e] = -INFINITY;
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 2) m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], sv[e], sv[e + 1]);
          const float mx = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          float alpha = 1.f;
          if ((mx - m_run) * qs > 8.f) {           // also on the first key a row sees
            alpha = ex2_approx((m_run - mx) * qs);
            m_run = mx;
            l *= alpha;
          }
          if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) scale_rows(oaddr, alpha);
          const float mb = m_run == -INFINITY ? kTcShift : kTcShift - m_run * qs;
          const uint64_t qs2 = pack2(qs, qs), mb2 = pack2(mb, mb);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float pf[16];   // 32 probabilities as fp16, over the scores' own place
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float y0, y1;
              unpack2(fma2(pack2(sv[c * 32 + e], sv[c * 32 + e + 1]), qs2, mb2), y0, y1);
              y0 = ex2_approx(y0);
              y1 = ex2_approx(y1);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(y0, y1));
              pf[e >> 1] = __uint_as_float(pack_f16x2(y0, y1));
            }
            tmem_st16(sp + c * 16, pf);
          }
          float y0, y1;
          unpack2(add2(sum[0], sum[1]), y0, y1);
          l += y0 + y1;
        } else {
          float pf[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pf[e] = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) tmem_st16(sp + c * 16, pf);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      // held: give up while the issuers finish the unit, or have left their role behind the last one
      if (sg.held) ok = kv4_hold_clear(p.status, 55, lane);
      ok = __all_sync(0xffffffffu, ok && kv4_wait(&o_full[w], (n_seg - 1) & 1, p.status, 69));
      if (!ok) break;
      tc_fence_after();
      float m2 = m_run == -INFINITY ? -INFINITY : m_run * qs, mine = 1.f, other = 0.f;
      const bool single = sg.single, whole = sg.first && sg.last;
      if (single) {
        pair_ml[w][r0 + lane] = make_float2(m2, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ml_full[w]);
        ok = __all_sync(0xffffffffu, kv4_wait(&ml_full[w ^ 1], n_single & 1, p.status, 56) &&
                                         kv4_wait(&o_full[w ^ 1], (n_seg - 1) & 1, p.status, 56));
        if (!ok) break;
        tc_fence_after();
        const float2 y = pair_ml[w ^ 1][r0 + lane];
        const float M = fmaxf(m2, y.x);
        mine = m2 == -INFINITY ? 0.f : ex2_approx(m2 - M);
        other = y.x == -INFINITY ? 0.f : ex2_approx(y.x - M);
        l = mine * l + other * y.y;
        m2 = M;
      }
      const float inv = m2 == -INFINITY ? 0.f : p.v_mul / l;
      const size_t at = (size_t)kv4_slot(blockIdx.x, sg.first) * p.R + (single ? 0 : w * 128) + r0;   // the warp's first row in the parts
      // O goes out by way of the warp's own rows of Q, which no product reads any more: 32 rows x
      // 128 bytes, swizzled, then 8 lanes write a row's 128 bytes
      if (live) {
        const Rows rows(p, sg.s, sg.kvh, row0 + r0);
        const int row_at = rows.at(p, lane);
        unsigned char* box = q_smem + w * kTile + r0 * 128;
        const int sw = lane & 7;
#pragma unroll 1
        for (int c = single ? 2 * w : 0; c < (single ? 2 * w + 2 : 4); ++c) {
          float o[32];
          tmem_ld32(oaddr + c * 32, o);
          if (single) {
            float y[32];
            tmem_ld32((oaddr ^ 128) + c * 32, y);   // the other stream's
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = mine * o[e] + other * y[e];
          } else {
            tmem_ld_wait();
          }
          if (whole) {   // bf16: two of the four make one row of 128 bytes
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t x[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) x[y] = pack_bf16x2(o[8 * e + 2 * y] * inv, o[8 * e + 2 * y + 1] * inv);
              *reinterpret_cast<uint4*>(box + lane * 128 + ((((c & 1) * 4 + e) ^ sw) * 16)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
            if ((c & 1) == 0) continue;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(box + lane * 128 + ((e ^ sw) * 16)) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
          const int d = lane & 7;   // a row's 16 bytes of these 128
          unsigned char* to = whole ? reinterpret_cast<unsigned char*>(p.out + rows.base * 128) + (c >> 1) * 128 + d * 16
                                    : reinterpret_cast<unsigned char*>(p.o_part + at * 128) + c * 128 + d * 16;
          const int bytes = whole ? 256 : 512;   // of a row
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int lr = i * 4 + (lane >> 3), row = __shfl_sync(0xffffffffu, row_at, lr);
            const uint4 v = *reinterpret_cast<const uint4*>(box + lr * 128 + ((d ^ (lr & 7)) * 16));
            if (row >= 0) *reinterpret_cast<uint4*>(to + (size_t)(whole ? row : lr) * bytes) = v;
          }
          __syncwarp();
        }
        if (row_at >= 0 && !(single && w == 1)) {
          if (!whole) p.ml_part[at + lane] = make_float2(m2, l);
          else if (p.lse) p.lse[rows.base + row_at] = kv4_lse(m2, l, kTcShift);   // m2 = -inf gives -inf
        }
      }
      if (threadIdx.x == 0) {
        if (sg.first) p.range[sg.unit].x = blockIdx.x;
        if (sg.last) p.range[sg.unit].y = blockIdx.x;
      }
      tc_fence_before();
      if (single) {   // neither goes on before the other has read its output
        __syncwarp();
        if (lane == 0) mbar_arrive(&merged);
        ok = __all_sync(0xffffffffu, kv4_wait(&merged, n_single++ & 1, p.status, 57));
        if (!ok) break;
      }
      give_back();
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
  const size_t smem = 1024 + (2 + kTiles) * kTile + kRaw * kRawBytes;
  if (ensure_dynamic_smem(kv4_attn_tc_kernel, smem) != cudaSuccess) return DF_ERR_CUDA;
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kv4_attn_tc_kernel) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < kLaunchRegs) return DF_ERR_CUDA;   // setmaxnreg would wait for registers that are not there
  launch_k(kv4_attn_tc_kernel, dim3(p.n_cta), dim3(kThreads), smem, st, p);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace df
