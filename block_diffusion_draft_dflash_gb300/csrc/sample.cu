// Draws under top-k, top-p and min-p from rows of logits, and rows' largest logits.
//
// A row's tokens stand in order of (logit descending, id ascending), as numbers comp = key << 32
// | ~id that are all different (key: the logit as an order-preserving integer).  Every filter
// keeps a prefix of that order, so a draw needs borders in it: the token at which a count or a
// mass is reached.
//
// A list of the first tokens.  One pass keeps the largest logit of each of 2048 groups (the
// elements that one thread reads).  The k-th largest of these is a lower bound of the k-th largest
// logit, and only the few groups that reach it are read again (from L2): hardly more than k
// candidates, which one CTA sorts.  That is all for a top-k up to 1024, for the largest logits and
// for min-p alone (whose bound is known).  For up to 64 tokens and for mass, every CTA of a row
// bounds and lists its own part, which saves two of the cluster's barriers.
// Mass alone (top-p, or nothing cut).  The first pass also sums exp((l - max) / T) in fp32, which
// gives the mass of the tokens that are not listed within 2^-15 of it, and half a unit of masses for
// each of them (a mass is a whole number of units).  If both ends of that
// interval put the borders on the same tokens of the list, they are right; a sure row's are.
// Otherwise a pass counts tokens in 2048 bins of 1/64 of a power of two of probability, from which
// follows where a border should lie; one more pass sums all masses, and those before the bins of
// the two borders, exactly, and lists these bins' tokens (up to 1024 for each border).  A border
// that is not among them is looked for bin by bin between exact masses.  Where a bin has too many
// tokens, its range of keys is cut by 2048 again until one key is left, whose tokens stand in order
// of their ids.
//
// Bounds.  The least that a row can do is to be read once.  What is measured (rows of 151936, one
// GB300, whole calls):
//   1 row, fp32                   11 us: the cluster's start and barriers, and one warp's end of the row
//   16 rows, 20 largest, fp32     12 us: the same
//   257 rows, top-k 20, fp32      46 us for 156 MB; a kernel that only reads them takes 26, a row's end 8
//   256 rows, top-p 0.9, bf16     137 to 210 us, by the inputs: 73 of the rows are searched, which reads each
//                                 twice more with some 25 instructions for a token's exact mass
//   2064 rows, mixed, bf16        325 us for 627 MB: first pass 191 (3.9 TB/s: four CTAs an SM, and each
//                                 ends its row without reading), 114 rows searched 135
//   2048 rows, 256 largest, bf16  243 us for 622 MB, and 288 MB of groups read again
#include <algorithm>

#include "rows.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {
namespace {

constexpr int kListCap = 2048;     // tokens that one CTA sorts
constexpr int kHalf = kListCap / 2;
constexpr int kMaxTop = 1024;      // top-k and K that the list of the first tokens is used for
constexpr int kFewTop = 64;        // up to this many, every CTA finds its own part's first ones
constexpr int kLikely = 64;        // tokens listed (about) where mass alone decides
constexpr int kBuckets = 512;      // of threshold() and sort_list()
constexpr int kBins = 2048;
constexpr int kBinBits = 11;
constexpr uint32_t kCountMask = (1u << 19) - 1;   // a bin's tokens; above it the sum of their places in the bin
constexpr int kSub = 8;            // groups of a thread
constexpr uint32_t kNone = 1u << 20, kAbove = 1u << 21;   // no bin of a level: below it, above it
constexpr uint32_t kAround = 512;  // tokens listed on either side of the bin where a border should be

constexpr uint32_t kMaskedKey = 0x0EB60D35u;   // of -1e30: masks by a type's lowest number lie below it
__device__ const Pow2Table kPow2;

struct Bins {          // running sums over bins: tokens, and about their mass
  uint32_t count[kBins];
  float mass[kBins];
};
struct Shared {
  union {
    uint32_t group_key[kSub * kRowThreads];  // of the whole row, in the first CTA (from several CTAs: of larger groups)
    uint64_t list[kListCap];                 // the first CTA's is the row's
  };
  union {
    Bins bins;
    uint64_t each_mass[kListCap];            // of the list's tokens
  };
  union {
    uint32_t hist[kBins];
    uint16_t chosen[kSub * kRowThreads];     // groups that one CTA reads again
  };
  float2 table[1024];
  // written by the first CTA in every CTA
  uint32_t word[8];
  // collected in the first CTA
  uint64_t mass, mass_in, mass_2;
  uint32_t n_list, n_list2, key_min, key_max, equal[8], at_id, live;
  float tail[8], sums[8];                    // of each CTA's part
  uint32_t part_max[8], part_least[8];
  // one CTA's own
  uint64_t tmp64[kRowWarps];
  uint32_t tmp32[kRowWarps];
  float tmpf[kRowWarps];
  uint64_t found_comp, found_mass;
  uint32_t found_n, found, n_chosen[kRowWarps], window[6];
  uint32_t n_rows;
  int rows[kRowThreads];
};

DF_DEV uint32_t logit_key(float l) { return float_key(l + 0.f); }   // -0 as +0
DF_DEV uint64_t comp_of(uint32_t key, int id) { return ((uint64_t)key << 32) | (uint32_t)~id; }
DF_DEV uint32_t key_of(uint64_t comp) { return (uint32_t)(comp >> 32); }
DF_DEV int id_of(uint64_t comp) { return (int)~(uint32_t)comp; }

struct GlobalTable {
  DF_DEV float2 operator[](uint32_t j) const { return make_float2(kPow2.hi[j], kPow2.lo[j]); }
};
template <class Table>
DF_DEV uint64_t mass_of(const MassScale& c, const Table& table, float l) {
  MassSum m;
  add_mass(m, c, table, l);
  m.n = 1;
  m.fold();
  return m.sum;
}
DF_DEV uint64_t mass_of(const MassScale& c, float l) { return mass_of(c, GlobalTable{}, l); }

// A border in the order: its token, the tokens up to it and their mass.
struct Border {
  uint64_t comp, mass;
  uint32_t n;
};

// f * m for f = 0 .. 1, rounded down; *more: it was not a whole number.
DF_DEV uint64_t part_of(float f, uint64_t m, bool* more) {
  const uint32_t b = __float_as_uint(f) & 0x7FFFFFFFu, e = b >> 23;
  const uint64_t mant = e ? (b & 0x7FFFFFu) | 0x800000u : b;
  const int shift = 150 - (int)max(e, 1u);                     // f = mant / 2^shift
  const uint64_t lo = m * mant, hi = __umul64hi(m, mant);      // hi < 2^24
  if (shift >= 64) {
    const int s = shift - 64;
    *more = lo != 0 || (s < 64 && (hi & ((1ull << s) - 1)) != 0) || (s >= 64 && hi != 0);
    return s < 64 ? hi >> s : 0;
  }
  *more = (lo & ((1ull << shift) - 1)) != 0;
  return (hi << (64 - shift)) | (lo >> shift);
}
// First mass above u * m, and first mass that reaches p * m.
DF_DEV uint64_t mass_above(float u, uint64_t m) {
  bool more;
  return part_of(u, m, &more) + 1;
}
DF_DEV uint64_t mass_share(float p, uint64_t m) {
  bool more;
  const uint64_t x = part_of(p, m, &more);
  return x + more ? x + more : 1;
}

template <class E>
struct RowWork {
  Shared& s;
  const RowPart<E> part;
  const int rank, ctas, tid;
  MassScale scale;
  static constexpr int VE = RowPart<E>::VE;

  DF_DEV RowWork(Shared& s_, const RowPart<E>& p, int rank_, int ctas_)
      : s(s_), part(p), rank(rank_), ctas(ctas_), tid(threadIdx.x) {}

  // The first CTA tells every CTA words 0 .. n - 1.
  DF_DEV void tell(const uint32_t* w, int n) {
    if (tid < ctas)
      for (int i = 0; i < n; ++i) st_remote(at_rank(&s.word[i], tid), w[i]);
  }

  // -------------------------------------------------------------------------- the first tokens
  // What a thread keeps of its groups (kSub of them, an eighth of its pieces each).  In registers: not
  // part of RowWork, whose address functions that are not inlined take.
  struct Tops {
    float top[kSub];     // their largest logits
    float sum[kSub];     // with SUMS: their sums of 2^(l c - ref)
    float ref;           // an exponent at most 8 below that of the thread's largest logit; inf: that of `far`
    float far;
  };

  // Reads the row.  SUMS: also the groups' sums, and with `count` the number of logits above -inf.
  template <bool SUMS>
  DF_DEV void read_tops(Tops& my, float c, bool count, uint32_t* live) {
    float m[kSub];
    uint32_t n_live = 0;
    my.ref = -INFINITY, my.far = 0.f;
#pragma unroll
    for (int j = 0; j < kSub; ++j) m[j] = -INFINITY, my.sum[j] = 0.f;
    // four groups' pieces, largest logit `big`
    auto add = [&](const uint4* v, int n, float big, float* to) {
      const float y = big * c;
      if (y > my.ref + 8.f) {              // also the first time
        const float f = my.ref > -INFINITY ? ex2_approx(my.ref - y) : 0.f;
#pragma unroll
        for (int j = 0; j < kSub; ++j) my.sum[j] = f > 0.f ? my.sum[j] * f : 0.f;     // a sum may be infinite, see sum_far
        my.ref = y;
      }
      if (!(my.ref > -INFINITY)) {         // nothing, or l c overflows
        if (count && big > -INFINITY)
#pragma unroll
          for (int j = 0; j < n; ++j) {
            float x[VE];
            RowOf<E>::unpack(v[j], x);
#pragma unroll
            for (int e = 0; e < VE; ++e) n_live += x[e] > -INFINITY;
          }
        return;
      }
#pragma unroll
      for (int j = 0; j < n; ++j) {
        float x[VE];
        RowOf<E>::unpack(v[j], x);
        if (count)
#pragma unroll
          for (int e = 0; e < VE; ++e) n_live += x[e] > -INFINITY;
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = ex2_approx(fmaf(x[e], c, -my.ref));
#pragma unroll
        for (int w = VE / 2; w > 0; w >>= 1)
#pragma unroll
          for (int e = 0; e < w; ++e) x[e] += x[e + w];
        to[j] += x[0];
      }
    };
    constexpr int U = SUMS ? 4 : 8;
    for (int i0 = part.lo + tid; i0 < part.hi; i0 += kSub * kRowThreads) {
#pragma unroll
      for (int h = 0; h < kSub; h += U) {
        uint4 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = part.whole_or_nothing(i0 + (h + j) * kRowThreads);
        float big = -INFINITY;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const float l = RowOf<E>::largest(v[j]);
          m[h + j] = max_nan(m[h + j], l);
          if (SUMS) big = fmaxf(big, l);
        }
        if (SUMS) add(v, U, big, my.sum + h);
      }
    }
    const int edge = part.my_edge();       // goes with the thread's first group
    if (edge >= 0) {
      const uint4 v = part.edge(edge);
      const float l = RowOf<E>::largest(v);
      m[0] = max_nan(m[0], l);
      if (SUMS) add(&v, 1, l, my.sum);
    }
#pragma unroll
    for (int j = 0; j < kSub; ++j) my.top[j] = m[j];
    if (SUMS) *live = n_live;
    if (SUMS && !(fabsf(my.ref) < 0x1p24f)) {     // also a thread without logits
      float big = -INFINITY;
#pragma unroll
      for (int j = 0; j < kSub; ++j) big = fmaxf(big, m[j]);
      my.ref = -INFINITY;
      if (big > -INFINITY) {
        my.ref = INFINITY;
        my.far = big;
        const Sums far = sum_far(c, big);
#pragma unroll
        for (int j = 0; j < kSub; ++j) my.sum[j] = far.of[j];
      }
    }
  }
  // The sums of a thread for which l c is too large a number: as a float it is off by so much that
  // 2^(l c - ref) may overflow, or it overflows itself.  Relative to the thread's largest logit m.
  struct Sums {
    float of[kSub];
  };
  __device__ __noinline__ Sums sum_far(float c, float m) const {
    Sums sum;
    auto add = [&](const uint4& v, float* to) {
      float x[VE];
      RowOf<E>::unpack(v, x);
#pragma unroll
      for (int e = 0; e < VE; ++e) *to += ex2_approx((x[e] - m) * c);
    };
#pragma unroll 1
    for (int g = 0; g < kSub; ++g) {
      sum.of[g] = 0.f;
#pragma unroll 1
      for (int i = part.lo + tid + g * kRowThreads; i < part.hi; i += kSub * kRowThreads) add(part.pieces[i], &sum.of[g]);
    }
    const int edge = part.my_edge();
    if (edge >= 0) add(part.edge(edge), &sum.of[0]);
    return sum;
  }
  static DF_DEV uint32_t top_key(float l) { return l == l ? logit_key(l) : 0xFFFFFFFFu; }

  // The groups' keys to the first CTA, those of several CTAs as the largest of `ctas` groups each.
  DF_DEV void post_groups(const Tops& my) {
    float m[kSub];
#pragma unroll
    for (int j = 0; j < kSub; ++j) m[j] = my.top[j];
    const int sub = kSub / ctas;
#pragma unroll
    for (int n = kSub / 2; n > 0; n >>= 1)
      if (sub <= n)
#pragma unroll
        for (int j = 0; j < n; ++j) m[j] = max_nan(m[2 * j], m[2 * j + 1]);
#pragma unroll
    for (int g = 0; g < kSub; ++g)
      if (g < sub) st_remote(at_rank(&s.group_key[(rank * sub + g) * kRowThreads + tid], 0), top_key(m[g]));
  }

  // This CTA's largest key (*largest), and a key that at least k of its threads reach, or all that
  // have a token: the upper 16 bits of the k-th largest of the threads' keys.  Every warp finds it.
  DF_DEV uint32_t part_threshold(const Tops& my, int k, uint32_t* largest) {
    float m = my.top[0];
#pragma unroll
    for (int j = 1; j < kSub; ++j) m = max_nan(m, my.top[j]);
    s.hist[tid] = top_key(m);
    __syncthreads();
    uint32_t key[kRowWarps], big = 0, n = 0;
#pragma unroll
    for (int j = 0; j < kRowWarps; ++j) {
      key[j] = s.hist[(tid & 31) + 32 * j];
      big = max(big, key[j]);
      n += key[j] > kNegInfKey;
    }
    *largest = __reduce_max_sync(0xffffffffu, big);
    uint32_t least = 0;
    if ((int)__reduce_add_sync(0xffffffffu, n) >= k)
#pragma unroll 1
      for (uint32_t bit = 1u << 31; bit > 1u << 15; bit >>= 1) {
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < kRowWarps; ++j) c += key[j] >= (least | bit);
        if ((int)__reduce_add_sync(0xffffffffu, c) >= k) least |= bit;
      }
    return max(least, kNegInfKey + 1);
  }
  // Lists what of this CTA's part reaches the key that k of its threads reach; the part's largest
  // key.  In the first CTA:
  // part_max and part_least; with SUMS tail, relative to the part's largest logit.
  template <bool SUMS>
  DF_DEV uint32_t list_part(const Tops& my, int k, float c) {
    uint32_t big;
    const uint32_t least = part_threshold(my, k, &big);
    if (tid == 0) {
      st_remote(at_rank(&s.part_max[rank], 0), big);
      st_remote(at_rank(&s.part_least[rank], 0), least);
    }
    list_tops<SUMS>(my, least, key_float(big), c);
    return big;
  }

  // First CTA, behind a row_sync: the largest key, and for k > 1 a key above -inf's that at least k
  // groups reach, or all that have a token.  Groups are counted in bins between the largest
  // and the smallest, and the smallest key of the bins that hold the first k is taken.
  DF_DEV uint32_t threshold(int k, uint32_t* largest) {
    uint32_t key[kSub];
    uint32_t big = 0, small = 0xFFFFFFFFu;
    if (k > 1)
      for (int b = tid; b < kBuckets; b += kRowThreads) s.hist[b] = 0;
    if (tid == 0) s.key_max = 0, s.key_min = 0xFFFFFFFFu, s.found = kBuckets;
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      key[j] = s.group_key[j * kRowThreads + tid];
      big = max(big, key[j]);
      if (key[j] > kMaskedKey) small = min(small, key[j]);
    }
    __syncthreads();
    big = __reduce_max_sync(0xffffffffu, big);
    small = __reduce_min_sync(0xffffffffu, small);
    if ((tid & 31) == 0) {
      atomicMax(&s.key_max, big);
      atomicMin(&s.key_min, small);
    }
    __syncthreads();
    big = s.key_max;
    *largest = big;
    if (k <= 1 || big <= kNegInfKey || big >= kPosInfKey) return big;
    const float bigf = key_float(big), scale_to = (float)kBuckets / (bigf - key_float(s.key_min));
    auto bin = [&](uint32_t kk) { return min((int)((bigf - key_float(kk)) * scale_to), kBuckets - 1); };   // NaN: 0
#pragma unroll
    for (int j = 0; j < kSub; ++j)
      if (key[j] > kNegInfKey) atomicAdd(&s.hist[bin(key[j])], 1u);
    __syncthreads();
    constexpr int PER = kBuckets / kRowThreads;
    uint32_t c[PER], mine = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += c[j] = s.hist[tid * PER + j];
    uint32_t run = block_scan(mine, s.tmp32, &all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (run < (uint32_t)k && run + c[j] >= (uint32_t)k) s.found = tid * PER + j;
      run += c[j];
    }
    if (tid == 0) s.key_max = 0xFFFFFFFFu;
    __syncthreads();
    const int last = (int)s.found;
    small = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kSub; ++j)
      if (key[j] > kNegInfKey && bin(key[j]) <= last) small = min(small, key[j]);
    small = __reduce_min_sync(0xffffffffu, small);
    if ((tid & 31) == 0) atomicMin(&s.key_max, small);
    __syncthreads();
    return (int)all < k ? kNegInfKey + 1 : s.key_max;
  }

  // Puts the elements that reach `least` on the row's list: the groups that reach it are read
  // again, by all threads.  Every CTA lists its own and hands them to the first one.  SUMS: the sum
  // of the others, relative to the largest logit, goes to the first CTA's tail: of the groups not
  // read again from the first pass, of those that are from this one, so that no large term that is
  // on the list has left its rounding there.  (A group's pieces are lo + who, lo + who + kSub *
  // kRowThreads, ..., who = the thread + its group * kRowThreads.)
  template <bool SUMS>
  DF_DEV void list_tops(const Tops& my, uint32_t least, float largest, float c) {
    const int lane = tid & 31, warp = tid / 32;
    float tail = 0.f;
    uint32_t who[kSub], at = 0;
#pragma unroll
    for (int g = 0; g < kSub; ++g) {
      const bool yes = logit_key(my.top[g]) >= least;
      if (SUMS && !yes) tail += my.sum[g];
      who[g] = __ballot_sync(0xffffffffu, yes);
      at += __popc(who[g]);
    }
    // in a fixed order, on which the rounding of the threads' sums depends
    if (lane == 0) s.n_chosen[warp] = at;
    if (SUMS) tail *= over_largest(my, largest, c);
    __syncthreads();
    uint32_t n_chosen = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      if (w == warp) at = n_chosen;
      n_chosen += s.n_chosen[w];
    }
#pragma unroll
    for (int g = 0; g < kSub; ++g) {
      if (who[g] >> lane & 1u) s.chosen[at + __popc(who[g] & ((1u << lane) - 1))] = (uint16_t)(g * kRowThreads + tid);
      at += __popc(who[g]);
    }
    __syncthreads();
    auto look = [&](const uint4& v, int piece) {
      const bool any = logit_key(RowOf<E>::largest(v)) >= least;
      if (!SUMS && !any) return;
      float x[VE];
      RowOf<E>::unpack(v, x);
      float t = 0.f;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        bool listed = false;
        if (any) {
          const uint32_t key = logit_key(x[e]);
          listed = key >= least;
          if (listed) put(&s.n_list, s.list, kListCap, key, part.id(piece, e));
        }
        if (SUMS && !listed) t += ex2_approx((x[e] - largest) * c);
      }
      if (SUMS) tail += t;
    };
    const int each = (part.hi - part.lo + kSub * kRowThreads - 1) / (kSub * kRowThreads);   // pieces of a group
    const int n = (int)n_chosen * each;
    for (int q0 = tid; q0 < n; q0 += 4 * kRowThreads) {
      uint4 v[4];
      int piece[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = q0 + j * kRowThreads, c = q / each, k = q - c * each;
        piece[j] = part.hi;
        if (q < n) {
          const int who = s.chosen[c];
          piece[j] = part.lo + who + k * kSub * kRowThreads;
        }
        v[j] = part.whole_or_nothing(piece[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) look(v[j], piece[j]);
    }
    const int edge = part.my_edge();
    if (edge >= 0 && logit_key(my.top[0]) >= least) look(part.edge(edge), edge);
    if (SUMS) {
      tail = block_add(tail, s.tmpf);
      if (tid == 0) st_remote(at_rank(&s.tail[rank], 0), tail);
    }
    hand_over(&s.n_list, s.list, kListCap);
  }
  // 2^(my.ref - largest c): ref is a float, l c - ref in the sums is rounded once, and so is this.
  static DF_DEV float over_largest(const Tops& my, float largest, float c) {
    if (my.ref == INFINITY) return ex2_approx((my.far - largest) * c);
    return my.ref > -INFINITY ? ex2_approx(fmaf(-largest, c, my.ref)) : 0.f;
  }
  // The part's sum relative to its largest logit, in the first CTA: sums.
  DF_DEV void give_sum(const Tops& my, float largest, float c) {
    float all = 0.f;
#pragma unroll
    for (int g = 0; g < kSub; ++g) all += my.sum[g];
    all = block_add(all * over_largest(my, largest, c), s.tmpf);
    if (tid == 0) st_remote(at_rank(&s.sums[rank], 0), all);
  }
  // What this CTA has put on its own list goes to the first CTA's (which has put its own there).
  DF_DEV void hand_over(uint32_t* counter, uint64_t* list, uint32_t room) {
    if (rank == 0) return;
    __syncthreads();
    const uint32_t mine = *counter;
    if (tid == 0) s.found_n = mine ? add_remote(at_rank(counter, 0), mine) : 0;
    __syncthreads();
    const uint32_t at = s.found_n;
    for (uint32_t i = tid; i < mine && at + i < room; i += kRowThreads) st_remote(at_rank(&list[at + i], 0), list[i]);
    __syncthreads();
  }
  // A token for this CTA's list (hand_over() follows).
  DF_DEV void put(uint32_t* counter, uint64_t* list, uint32_t room, uint32_t key, int id) {
    const uint32_t n = atomicAdd(counter, 1u);
    if (n < room) list[n] = comp_of(key, id);
  }

  // One CTA: n entries (at most kListCap) in order.  Few: an entry's place is the number of entries
  // before it.  Else they are dealt into buckets between the largest and the smallest logit first,
  // and counted in their bucket alone.
  __device__ __noinline__ void sort_list(uint64_t* list, int n) {
    if (n <= kRowThreads / 2) {
      const uint64_t e = tid < n ? list[tid] : 0;
      int at = 0;
      if (tid < n)
#pragma unroll 4
        for (int i = 0; i < n; ++i) at += list[i] > e;
      __syncthreads();
      if (tid < n) list[at] = e;
      __syncthreads();
      return;
    }
    if (n <= 2 * kRowThreads)
      deal<2>(list, n);
    else
      deal<kListCap / kRowThreads>(list, n);
  }
  template <int OWN>     // entries of a thread
  DF_DEV void deal(uint64_t* list, int n) {
    if (tid == 0) s.key_max = 0, s.key_min = 0xFFFFFFFFu;
    for (int b = tid; b < kBuckets; b += kRowThreads) s.hist[b] = 0;
    __syncthreads();
    uint32_t big = 0, small = 0xFFFFFFFFu;
#pragma unroll 1
    for (int i = tid; i < n; i += kRowThreads) {
      const uint32_t key = key_of(list[i]);
      big = max(big, key);
      small = min(small, key);
    }
    big = __reduce_max_sync(0xffffffffu, big);
    small = __reduce_min_sync(0xffffffffu, small);
    if ((tid & 31) == 0) {
      atomicMax(&s.key_max, big);
      atomicMin(&s.key_min, small);
    }
    __syncthreads();
    const float bigf = key_float(s.key_max), to = (float)kBuckets / (bigf - key_float(s.key_min));
    // A list of bf16 logits may have few different ones: these share the buckets, and the tokens of
    // one are dealt by their ids (2064 mixed rows 325 us, by the logit alone 346; 256 nucleus rows of four
    // inputs 165, 176, 143, 137 against 182, 198, 157, 163).
    const uint32_t levels = ((s.key_max - s.key_min) >> 16) + 1, each = VE == 8 ? kBuckets / levels : 0;
    const float by_id = (float)each / (float)part.V;
    uint64_t e[OWN];
    uint32_t place[OWN];
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      const int i = tid + j * kRowThreads;
      if (i >= n) break;
      e[j] = list[i];
      int b;
      if (each > 1)
        b = ((s.key_max - key_of(e[j])) >> 16) * each + min((uint32_t)((float)id_of(e[j]) * by_id), each - 1);
      else
        b = min((int)((bigf - key_float(key_of(e[j]))) * to), kBuckets - 1);   // NaN: 0
      place[j] = ((uint32_t)b << 16) | atomicAdd(&s.hist[b], 1u);
    }
    __syncthreads();
    constexpr int PER = kBuckets / kRowThreads;
    uint32_t c[PER], mine = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += c[j] = s.hist[tid * PER + j];
    uint32_t run = block_scan(mine, s.tmp32, &all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      s.hist[tid * PER + j] = run;
      run += c[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      if (tid + j * kRowThreads >= n) break;
      list[s.hist[place[j] >> 16] + (place[j] & 0xFFFFu)] = e[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      if (tid + j * kRowThreads >= n) break;
      const uint32_t b = place[j] >> 16, from = s.hist[b], upto = b + 1 < kBuckets ? s.hist[b + 1] : (uint32_t)n;
      uint32_t at = from;
      for (uint32_t i = from; i < upto; ++i) at += list[i] > e[j];
      place[j] = at;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      if (tid + j * kRowThreads >= n) break;
      list[place[j]] = e[j];
    }
    __syncthreads();
  }

  // One CTA, sorted list of n entries behind n_before tokens of mass_before: the border where the
  // tokens reach want_n or the mass reaches `want`.  False: it is not here; *mass_after: behind the list.
  __device__ __noinline__ bool border_in_list(const uint64_t* list, int n, uint32_t n_before, uint64_t mass_before, bool by_count,
                             uint32_t want_n, uint64_t want, uint64_t* mass_after, Border* found) {
    const int per = (n + kRowThreads - 1) / kRowThreads, from = tid * per, upto = min(from + per, n);
    uint64_t mine = 0, all;
#pragma unroll 1
    for (int i = from; i < upto; ++i) mine += mass_of(scale, s.table, key_float(key_of(list[i])));
    if (tid == 0) s.found = 0;
    uint64_t run = mass_before + block_scan(mine, s.tmp64, &all);
#pragma unroll 1
    for (int i = from; i < upto; ++i) {
      const uint64_t before = run;
      run += mass_of(scale, s.table, key_float(key_of(list[i])));
      if (by_count ? n_before + i + 1 == want_n : before < want && run >= want) {
        s.found_comp = list[i];
        s.found_mass = run;
        s.found_n = n_before + i + 1;
        s.found = 1;
      }
    }
    __syncthreads();
    const bool yes = s.found != 0;
    if (yes) *found = Border{s.found_comp, s.found_mass, s.found_n};
    *mass_after = mass_before + all;
    __syncthreads();
    return yes;
  }

  // -------------------------------------------------------------------------- all tokens
  DF_DEV void load_table() {
    for (int i = tid; i < 1024; i += kRowThreads) s.table[i] = make_float2(kPow2.hi[i], kPow2.lo[i]);
  }
  DF_DEV void give_mass(MassSum& m, uint64_t* to) {   // to the first CTA's
    m.fold();
    const uint64_t sum = block_add(m.sum, s.tmp64);
    if (tid == 0 && sum) add_remote(at_rank(to, 0), sum);
  }

  // All CTAs, behind a row_sync: running sums of the cluster's histograms in the first one's bins.
  // weight(b, n, places): about the mass of a bin's n tokens.
  template <class W>
  DF_DEV void run_bins(W&& weight) {
    const int share = kBins / ctas;
    for (int i = tid; i < share; i += kRowThreads) {
      const int b = rank * share + i;
      uint32_t h[8], n = 0, places = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) h[r] = r >= ctas ? 0 : ctas == 1 ? s.hist[b] : ld_remote(at_rank(&s.hist[b], r));
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        n += h[r] & kCountMask;
        places += h[r] >> 19;
        if ((h[r] & kCountMask) > 1170) places = 1u << 30;      // their sum does not fit
      }
      st_remote(at_rank(&s.bins.count[b], 0), n);
      st_remote(at_rank(&s.bins.mass[b], 0), n ? weight(b, n, places) : 0.f);
    }
    row_sync(ctas);
    if (rank != 0) return;
    constexpr int PER = kBins / kRowThreads / 4;
    uint4* const counts = reinterpret_cast<uint4*>(s.bins.count) + tid * PER;
    float4* const masses = reinterpret_cast<float4*>(s.bins.mass) + tid * PER;
    uint32_t n = 0, all_n;
    float m = 0.f, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint4 c = counts[j];
      const float4 e = masses[j];
      n += (c.x + c.y) + (c.z + c.w);
      m += (e.x + e.y) + (e.z + e.w);
    }
    n = block_scan(n, s.tmp32, &all_n);
    m = block_scan(m, s.tmpf, &all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      uint4 c = counts[j];
      float4 e = masses[j];
      n = c.w = (c.z = (c.y = (c.x += n) + c.y) + c.z) + c.w;
      m = e.w = (e.z = (e.y = (e.x += m) + e.y) + e.z) + e.w;
      counts[j] = c;
      masses[j] = e;
    }
    __syncthreads();
  }
  // Tokens' bins by probability: 1/64 of a power of two, the last one all below 2^-32; what is added
  // for one (its place in the bin in eighths goes above the count).  Of 1/32 (no last one) flat rows
  // have more tokens in a bin than a list takes: 2064 mixed rows 338 to 438 us against 346 to 356.
  static DF_DEV uint32_t bin_of(uint32_t below_top) { return min(below_top >> 4, kBins - 1u); }
  static DF_DEV uint32_t entry_of(uint32_t below_top) { return 1u + ((below_top & 14u) << 18); }
  static DF_DEV float bin_mass(int b, uint32_t n, uint32_t places) {
    const float at = places < 1u << 30 ? ((float)places / (float)n + 0.5f) * 0.125f : 0.5f;
    return (float)n * exp2f(b < kBins - 1 ? -((float)b + at) * (1.f / 64.f) : -40.f);
  }
  bool by_probability;     // the bins are these (else of a range of keys)

  // Counts tokens in bins by probability; SUMS: and sums all masses (first CTA's s.mass).
  template <bool SUMS>
  DF_DEV void count_pass() {
    for (int b = tid; b < kBins; b += kRowThreads) s.hist[b] = 0;
    if (SUMS) load_table();
    __syncthreads();
    MassSum m;
    const MassScale c = scale;
    const RowPart<E> p = part;
    uint32_t* const hist = s.hist;
    const float2* const table = s.table;
    for_pieces<4>(p, [&](const float* x, int, bool) {
      if (SUMS) m.room(VE);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint32_t d = c.top - (SUMS ? add_mass(m, c, table, x[e]) : c.bits(x[e]));
        if (x[e] > -INFINITY) atomicAdd(&hist[bin_of(d)], entry_of(d));
      }
      m.n += VE;
    });
    if (SUMS) give_mass(m, &s.mass);
    by_probability = true;
  }
  // First CTA: *total, *live = tokens above -inf.  Ends with a barrier, like locate(): what follows may
  // set the sums that every thread has just read back to 0.
  __device__ __noinline__ void count_all(uint64_t* total, uint32_t* live) {
    if (tid == 0) s.mass = 0;
    row_sync(ctas);
    count_pass<true>();
    row_sync(ctas);
    run_bins(bin_mass);
    if (rank == 0) {
      *total = s.mass;
      *live = s.bins.count[kBins - 1];
    }
    row_sync(ctas);
  }

  // The part of a search that a level's bins are left with (first CTA): the border lies in bins
  // first .. last; before them n0 + count[first - 1] tokens and mass m0, with them mass m1.
  struct Window {
    uint32_t first, last, n0;
    uint64_t m0, m1;
  };
  // The number of bins whose running sum is below `upto`.
  template <class V>
  static DF_DEV uint32_t bins_below(const V* sum, V upto) {
    uint32_t n = 0;
#pragma unroll 1
    for (uint32_t step = kBins; step; step >>= 1)
      if (n + step <= kBins && sum[n + step - 1] < upto) n += step;
    return n;
  }
  // A thread of the first CTA: the bin where the border should be (exactly, for a count), with some
  // around it as far as their tokens fit in `room`.  w: first and last bin, their tokens.
  DF_DEV void choose(const Window& v, int tries, bool by_count, uint32_t want_n, uint64_t want, uint32_t* w,
                     uint32_t room = kListCap, uint32_t around = kAround) {
    const uint32_t* const count = s.bins.count;
    uint32_t at;
    if (by_count) {
      at = bins_below(count, want_n - v.n0);
    } else {
      const float e0 = v.first ? s.bins.mass[v.first - 1] : 0.f, e1 = s.bins.mass[v.last];
      at = bins_below((const float*)s.bins.mass, e0 + (float)(want - v.m0) / (float)(v.m1 - v.m0) * (e1 - e0));
      if (tries >= 3) at = v.first + (v.last - v.first) / 2;   // the masses mislead
    }
    at = min(max(at, v.first), v.last);
    const uint32_t upto = count[at], before = at ? count[at - 1] : 0;
    uint32_t lo = at, hi = at;
    if (!by_count && upto - before < room) {
      around = min(around, (room - (upto - before)) / 2);
      // bins from which at most `around` tokens lie before `at`, and up to which behind it
      lo = before > around ? bins_below(count, before - around) + 1 : 0;
      hi = bins_below(count, upto + around + 1);
      lo = min(max(lo, v.first), at);
      hi = max(min(hi, kBins) - (hi > 0), at);
      hi = min(hi, v.last);
    }
    w[0] = lo;
    w[1] = hi;
    w[2] = count[hi] - (lo ? count[lo - 1] : 0);
  }
  // All CTAs: mass before the window (s.mass); its tokens on the list if they fit, else their mass
  // (s.mass_in) and range of keys.  bin(l, key): a logit's bin of this level, above kBins: none,
  // not smaller for a smaller logit but above the level.
  template <class B>
  DF_DEV void read_window(B&& bin) {
    const uint32_t b1 = s.word[0], b2 = s.word[1];
    const bool few = s.word[2] <= kListCap;
    const MassScale c = scale;
    const RowPart<E> p = part;
    const float2* const table = s.table;
    MassSum m, in;
    uint32_t kmin = 0xFFFFFFFFu, kmax = 0;
    for_pieces<4>(p, [&](const float* x, int piece, bool) {
      float big = x[0];
#pragma unroll
      for (int e = 1; e < VE; ++e) big = fmaxf(big, x[e]);
      const uint32_t first = bin(big, logit_key(big));
      if (first > b2 && first < kAbove) return;    // all of the piece lies behind the window
      m.room(VE);
      in.room(VE);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint32_t key = logit_key(x[e]), b = bin(x[e], key);
        if (b > b2) continue;
        if (b < b1) {
          add_mass(m, c, table, x[e]);
          ++m.n;
        } else if (few) {
          put(&s.n_list, s.list, kListCap, key, p.id(piece, e));
        } else {
          add_mass(in, c, table, x[e]);
          ++in.n;
          kmin = min(kmin, key);
          kmax = max(kmax, key);
        }
      }
    });
    give_mass(m, &s.mass);
    if (few) {
      hand_over(&s.n_list, s.list, kListCap);
      return;
    }
    give_mass(in, &s.mass_in);
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if ((tid & 31) == 0) {
      min_remote(at_rank(&s.key_min, 0), kmin);
      max_remote(at_rank(&s.key_max, 0), kmax);
    }
  }
  // Words 3 .. 6 of a search: what comes next, and the next level's range of keys.
  enum { kAgain = 0, kFound = 1, kDeeper = 2 };

  // Looks for the border among one level's bins.  `lv`: the level's tokens and masses; on kDeeper
  // those of the bin that holds it (first CTA).
  template <class B>
  DF_DEV uint32_t search(Window* lv, bool by_count, uint32_t want_n, uint64_t want, Border* found, B&& bin) {
    const uint64_t base = lv->m0;      // mass before the level's bins
    for (int tries = 0; tries < 16; ++tries) {
      uint32_t w[3];
      if (rank == 0) {
        if (tid == 0) choose(*lv, tries, by_count, want_n, want, s.window);
        __syncthreads();
        for (int i = 0; i < 3; ++i) w[i] = s.window[i];
        tell(w, 3);
      }
      if (tid == 0) s.mass = s.mass_in = 0, s.n_list = 0, s.key_min = 0xFFFFFFFFu, s.key_max = 0;
      row_sync(ctas);
      read_window(bin);
      row_sync(ctas);
      if (rank == 0) {
        const uint32_t n_before = lv->n0 + (w[0] ? s.bins.count[w[0] - 1] : 0);
        const uint64_t before = base + s.mass;
        uint64_t after = before + s.mass_in;
        uint32_t next = kAgain;
        if (w[2] <= kListCap) {
          const int n = (int)min(s.n_list, (uint32_t)kListCap);
          sort_list(s.list, n);
          if (border_in_list(s.list, n, n_before, before, by_count, want_n, want, &after, found)) next = kFound;
        } else if (by_count || (before < want && after >= want)) {
          next = kDeeper;
          *lv = Window{0, kBins - 1, n_before, before, after};
        }
        uint32_t word[4] = {next, 0, s.key_max, s.key_min};
        if (next == kAgain) {
          if (want <= before) {
            lv->last = w[0] ? w[0] - 1 : 0;
            lv->m1 = before;
          } else {
            lv->first = min(w[1] + 1, (uint32_t)kBins - 1);
            lv->m0 = after;
          }
        } else if (next == kDeeper) {
          word[1] = (uint32_t)max(0, 32 - __clz(word[2] - word[3]) - kBinBits);
        }
        if (tid < ctas)
          for (int i = 0; i < 4; ++i) st_remote(at_rank(&s.word[3 + i], tid), word[i]);
      }
      row_sync(ctas);
      if (s.word[3] != kAgain) break;
    }
    return s.word[3];
  }

  // The border where the tokens reach want_n or their mass reaches `want` (arguments and result
  // of the first CTA; every CTA calls it), after count_all.
  __device__ __noinline__ Border locate(bool by_count, uint32_t want_n, uint64_t want, uint64_t total) {
    Border found{0, 0, 0};
    Window lv{0, kBins - 1, 0, 0, total};
    const MassScale c = scale;
    const RowPart<E> p = part;
    if (!by_probability) {         // the last search left a level's bins
      row_sync(ctas);
      count_pass<false>();
      row_sync(ctas);
      run_bins(bin_mass);
    }
    uint32_t next = search(&lv, by_count, want_n, want, &found, [&](float l, uint32_t) {
      return l > -INFINITY ? bin_of(c.top - c.bits(l)) : kNone;
    });
    // Too many tokens in one bin: cut its keys into bins again, until they fit or one key is left.
    for (int level = 0; level < 4 && next == kDeeper; ++level) {
      const uint32_t shift = s.word[4], hi = s.word[5], lo = s.word[6];
      if (hi == lo) break;
      by_probability = false;
      for (int b = tid; b < kBins; b += kRowThreads) s.hist[b] = 0;
      row_sync(ctas);
      for_pieces<4>(p, [&](const float* x, int, bool) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const uint32_t key = logit_key(x[e]);
          if (key >= lo && key <= hi) atomicAdd(&s.hist[(hi - key) >> shift], 1u);
        }
      });
      row_sync(ctas);
      run_bins([&](int b, uint32_t n, uint32_t) {
        const uint32_t mid = ((uint32_t)b << shift) + (shift ? 1u << (shift - 1) : 0);
        return (float)n * (float)mass_of(scale, key_float(hi - min(mid, hi - lo)));
      });
      next = search(&lv, by_count, want_n, want, &found, [&](float, uint32_t key) {
        return key > hi ? kAbove : key >= lo ? (hi - key) >> shift : kNone;
      });
    }
    if (next == kDeeper) one_key(s.word[5], lv, by_count, want_n, want, &found);
    row_sync(ctas);
    return found;
  }

  // All CTAs: all masses (s.mass) and those before two windows of bins, words 0 and 1 (s.mass_in),
  // words 3 and 4 (s.mass_2); the windows' tokens on the list's halves.
  __device__ __noinline__ void sum_and_list() {
    const MassScale c = scale;
    const RowPart<E> p = part;
    // bins are not cut off at the last one here; a window that ends there has no end
    auto end = [](uint32_t b) { return b < kBins - 1 ? b : ~0u; };
    const uint32_t a1 = s.word[0], a2 = end(s.word[1]), d1 = s.word[3], d2 = end(s.word[4]), last = max(a2, d2);
    const float2* const table = s.table;
    MassSum m, ma, md;
    for_pieces<2>(p, [&](const float* x, int piece, bool) {
      float big = x[0];
#pragma unroll
      for (int e = 1; e < VE; ++e) big = fmaxf(big, x[e]);
      m.room(VE);
      m.n += VE;
      if ((c.top - c.bits(big)) >> 4 > last) {      // the piece lies behind both windows
#pragma unroll
        for (int e = 0; e < VE; ++e) add_mass(m, c, table, x[e]);
        return;
      }
      ma.room(VE);
      md.room(VE);
      uint32_t in = 0;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        uint32_t ta, tb;
        const uint32_t bin = (c.top - mass_terms(c, table, x[e], &ta, &tb)) >> 4;
        m.a += ta;
        m.b += tb;
        if (bin < a1) ma.a += ta, ma.b += tb, ++ma.n;
        else if (bin <= a2) in |= 1u << e;
        if (bin < d1) md.a += ta, md.b += tb, ++md.n;
        else if (bin <= d2) in |= 256u << e;
      }
      if (in)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if ((in >> e & 257u) && x[e] > -INFINITY) {
            const uint32_t key = logit_key(x[e]);
            const int id = p.id(piece, e);
            if (in >> e & 1u) put(&s.n_list, s.list, kHalf, key, id);
            if (in >> e & 256u) put(&s.n_list2, s.list + kHalf, kHalf, key, id);
          }
    });
    give_mass(m, &s.mass);
    give_mass(ma, &s.mass_in);
    give_mass(md, &s.mass_2);
    hand_over(&s.n_list, s.list, kHalf);
    hand_over(&s.n_list2, s.list + kHalf, kHalf);
  }
  // The borders of top-p (p < 1) and of the draw, in one pass over all masses; m_about: about the
  // row's.  Bit 0: *kept is right, bit 1: *drawn too (first CTA); for what is not, the row's exact
  // mass is in *total and bins are counted, for locate().
  __device__ __noinline__ uint32_t two_borders(float p, float u, uint64_t m_about, uint64_t* total, uint32_t* live, Border* kept,
                                           Border* drawn) {
    if (tid == 0) s.mass = s.mass_in = s.mass_2 = 0;
    load_table();
    count_pass<false>();
    row_sync(ctas);
    run_bins(bin_mass);
    uint32_t w[6];
    if (rank == 0) {
      const Window all{0, kBins - 1, 0, 0, m_about};
      const uint64_t keep = p < 1.f ? mass_share(p, m_about) : m_about;
      if (tid < 2) choose(all, 0, false, 0, tid == 0 ? keep : mass_above(u, keep), s.window + 3 * tid, kHalf, kHalf);
      __syncthreads();
      for (int i = 0; i < 6; ++i) w[i] = s.window[i];
#pragma unroll
      for (int i = 0; i < 6; i += 3)
        if (w[i + 2] > kHalf || (i == 0 && p >= 1.f)) w[i] = 1, w[i + 1] = 0;     // not listed
      tell(w, 6);
    }
    if (tid == 0) s.n_list = s.n_list2 = 0;
    row_sync(ctas);
    sum_and_list();
    row_sync(ctas);
    uint32_t ok = 0;
    if (rank == 0) {
      const uint64_t m = s.mass, before_a = s.mass_in, before_d = s.mass_2;
      *total = m;
      *live = s.bins.count[kBins - 1];
      *kept = Border{0, m, *live};
      uint64_t after;
      bool yes = true;
      if (p < 1.f) {
        const int n = (int)min(s.n_list, (uint32_t)kHalf);
        yes = w[0] <= w[1];
        if (yes) {
          sort_list(s.list, n);
          yes = border_in_list(s.list, n, w[0] ? s.bins.count[w[0] - 1] : 0, before_a, false, 0, mass_share(p, m), &after, kept);
        }
      }
      ok = yes;
      if (yes && w[3] <= w[4]) {
        const int n = (int)min(s.n_list2, (uint32_t)kHalf);
        sort_list(s.list + kHalf, n);
        if (border_in_list(s.list + kHalf, n, w[3] ? s.bins.count[w[3] - 1] : 0, before_d, false, 0,
                           mass_above(u, kept->mass), &after, drawn))
          ok = 3;
      }
      if (tid < ctas) st_remote(at_rank(&s.word[7], tid), ok);
    }
    row_sync(ctas);
    return s.word[7];
  }

  // All tokens of the bin have one key: in order of their ids.
  DF_DEV void one_key(uint32_t key, const Window& lv, bool by_count, uint32_t want_n, uint64_t want, Border* found) {
    uint32_t mine = 0;
    for_pieces<4>(part, [&](const float* x, int, bool) {
#pragma unroll
      for (int e = 0; e < VE; ++e) mine += logit_key(x[e]) == key;
    });
    mine = block_add(mine, s.tmp32);
    if (tid == 0) st_remote(at_rank(&s.equal[rank], 0), mine);
    row_sync(ctas);
    if (rank == 0) {
      const uint64_t w = mass_of(scale, key_float(key));
      uint64_t r = by_count ? want_n - lv.n0 : w ? (want - lv.m0 + w - 1) / w : 1;
      uint32_t all = 0;
      for (int i = 0; i < ctas; ++i) all += s.equal[i];
      r = r < 1 ? 1 : r > all ? all : r;
      found->n = lv.n0 + (uint32_t)r;
      found->mass = lv.m0 + r * w;
      uint32_t left = (uint32_t)r, who = 0;
      while (who + 1 < (uint32_t)ctas && left > s.equal[who]) left -= s.equal[who++];
      const uint32_t word[2] = {who, left};
      tell(word, 2);
    }
    row_sync(ctas);
    if ((uint32_t)rank == s.word[0]) {
      uint32_t left = s.word[1];
      for (int i0 = part.begin; i0 < part.end; i0 += kRowThreads) {
        const int i = i0 + tid;
        float x[VE];
        RowOf<E>::unpack(i < part.end ? part.load(i) : part.whole_or_nothing(part.hi), x);
        uint32_t c = 0, all;
#pragma unroll
        for (int e = 0; e < VE; ++e) c += logit_key(x[e]) == key;
        uint32_t before = block_scan(c, s.tmp32, &all);
        if (before < left && left <= before + c) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (logit_key(x[e]) == key && ++before == left) st_remote(at_rank(&s.at_id, 0), (uint32_t)part.id(i, e));
        }
        if (left <= all) break;
        left -= all;
      }
    }
    row_sync(ctas);
    if (rank == 0) found->comp = comp_of(key, (int)s.at_id);
  }
};

// The smallest logit that min-p keeps; one thread's work for the block (64-bit arithmetic is slow).
DF_DEV float least_logit(float largest, float T, float min_p, float* tmp) {
  __syncthreads();
  if (threadIdx.x == 0) {
    const double d = (double)largest + (double)T * log((double)min_p);
    float f = (float)d;
    if ((double)f < d) f = key_float(float_key(f) + 1);
    *tmp = f;
  }
  __syncthreads();
  return *tmp;
}
DF_DEV float log_share(const MassScale& c, float l, uint64_t w, uint64_t m) {
  if (w >= m) return 0.f;
  if (2 * w >= m) return log1pf(-((float)(m - w) / (float)m));
  const float x = c.arg(l), t = fmaf(x, c.c_hi, c.shift), g = t - c.shift;
  float r = fmaf(x, c.c_hi, -g);
  r = fmaf(x, c.c_lo, r);
  // y = l c - ref = (t - 12288) + r
  const float y = (t - 12288.f) + r;
  return 0.693147180559945f * (y - log2f((float)m * kMassUnit));
}

// How far the mass of tokens that are not listed may be from the sum of their probabilities, in units:
// that sum's own error, and each token's rounding to a whole number.
DF_DEV uint64_t tail_error(uint64_t tail, int V) { return (tail >> 15) + (uint64_t)V / 2 + 1; }

// The first CTA's end of a row whose first n tokens are on the list, in order.  whole: the kept
// tokens are among them, all that top-k or min-p left; else the others have about the mass `tail`
// (within tail_error) and the row has `live` tokens.  True: done; *about: about the row's mass.
template <class E, class Give>
DF_DEV bool finish(RowWork<E>& w, int n, bool whole, uint64_t tail, uint32_t live, float p, uint32_t key_low, float u,
                   bool log, uint64_t* about, Give&& give) {
  Shared& s = w.s;
  const int per = (n + kRowThreads - 1) / kRowThreads, from = w.tid * per, upto = min(from + per, n);
  uint64_t mine = 0, total;
#pragma unroll 1
  for (int i = from; i < upto; ++i) mine += s.each_mass[i] = mass_of(w.scale, key_float(key_of(s.list[i])));
  const uint64_t start = block_scan(mine, s.tmp64, &total);
  uint64_t m_lo = total, m_hi = total, m_mid = total;
  if (!whole) {
    const uint64_t e = tail_error(tail, w.part.V);
    m_lo += tail - min(tail, e);
    m_hi += tail + e;
    *about = m_mid = total + tail;
  }
  uint32_t n_kept = whole ? n : live;
  int room = n;                      // listed tokens that may be drawn
  if (p < 1.f || key_low) {
    const uint64_t share_lo = p < 1.f ? mass_share(p, m_lo) : ~0ull, share_hi = p < 1.f ? mass_share(p, m_hi) : ~0ull;
    uint32_t c = 0;                  // tokens kept at either end of the interval
    uint64_t before = start;
    mine = 0;
#pragma unroll 1
    for (int i = from; i < upto; ++i) {
      if (key_of(s.list[i]) >= key_low) {
        c += (before < share_lo) + ((before < share_hi) << 16);
        if (before < share_lo) mine += s.each_mass[i];
      }
      before += s.each_mass[i];
    }
    c = block_add(c, s.tmp32);
    n_kept = room = c & 0xFFFF;
    if (!whole && (room != (int)(c >> 16) || room == n)) return false;
    m_lo = m_hi = m_mid = block_add(mine, s.tmp64);
  }
  const uint64_t want_lo = mass_above(u, m_lo), want_hi = mass_above(u, m_hi);
  if (w.tid == 0) s.found = 0;
  __syncthreads();
  uint64_t at = start;
#pragma unroll 1
  for (int i = from; i < min(upto, room); ++i) {
    const uint64_t before = at, m = s.each_mass[i];
    at += m;
    if (before < want_lo && at >= want_hi) {
      const uint64_t comp = s.list[i];
      give(id_of(comp), log ? log_share(w.scale, key_float(key_of(comp)), m, m_mid) : 0.f, (int32_t)n_kept);
      s.found = 1;
    }
  }
  __syncthreads();
  return s.found != 0;
}

// The same for at most 64 tokens, by the first warp alone.
template <class E, class Give>
DF_DEV bool finish_few(RowWork<E>& w, int n, bool whole, uint64_t tail, uint32_t live, float p, uint32_t key_low, float u,
                       bool log, uint64_t* about, Give&& give) {
  Shared& s = w.s;
  const int lane = w.tid & 31;
  const uint64_t e0 = 2 * lane < n ? s.list[2 * lane] : 0, e1 = 2 * lane + 1 < n ? s.list[2 * lane + 1] : 0;
  const uint64_t m0 = 2 * lane < n ? mass_of(w.scale, key_float(key_of(e0))) : 0;
  const uint64_t m1 = 2 * lane + 1 < n ? mass_of(w.scale, key_float(key_of(e1))) : 0;
  uint64_t incl = m0 + m1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const uint64_t start = incl - m0 - m1, total = __shfl_sync(0xffffffffu, incl, 31);
  uint64_t m_lo = total, m_hi = total, m_mid = total;
  if (!whole) {
    const uint64_t e = tail_error(tail, w.part.V);
    m_lo += tail - min(tail, e);
    m_hi += tail + e;
    *about = m_mid = total + tail;
  }
  uint32_t n_kept = whole ? n : live;
  int room = n;
  if (p < 1.f || key_low) {
    const uint64_t share_lo = p < 1.f ? mass_share(p, m_lo) : ~0ull, share_hi = p < 1.f ? mass_share(p, m_hi) : ~0ull;
    const bool k0 = 2 * lane < n && key_of(e0) >= key_low, k1 = 2 * lane + 1 < n && key_of(e1) >= key_low;
    const bool y0 = k0 && start < share_lo, y1 = k1 && start + m0 < share_lo;
    const uint32_t c = (uint32_t)y0 + y1 + (((uint32_t)(k0 && start < share_hi) + (k1 && start + m0 < share_hi)) << 16);
    const uint32_t both = __reduce_add_sync(0xffffffffu, c);
    n_kept = room = both & 0xFFFF;
    if (!whole && (room != (int)(both >> 16) || room == n)) return false;
    m_lo = m_hi = m_mid = warp_add((y0 ? m0 : 0) + (y1 ? m1 : 0));
  }
  const uint64_t want_lo = mass_above(u, m_lo), want_hi = mass_above(u, m_hi);
  const bool at0 = 2 * lane < room && start < want_lo && start + m0 >= want_hi;
  const bool at1 = 2 * lane + 1 < room && start + m0 < want_lo && incl >= want_hi;
  if (at0 || at1) {
    const uint64_t comp = at0 ? e0 : e1;
    give(id_of(comp), log ? log_share(w.scale, key_float(key_of(comp)), at0 ? m0 : m1, m_mid) : 0.f,
         (int32_t)n_kept);
  }
  return __any_sync(0xffffffffu, at0 || at1);
}

// A row's settings.
struct Settings {
  float T, p, low, u;
  int k;
  bool ok, by_k, by_min, by_mass;
  bool as_unset;       // nothing is cut, and the draw is keyed: the token of a draw without settings

  DF_DEV Settings(const SampleArgs& a, int r) {
    const int g = (a.row0 + r) / a.group;
    T = a.temperature ? a.temperature[g] : 1.f;
    k = a.top_k ? a.top_k[g] : 0;
    p = a.top_p ? a.top_p[g] : 1.f;
    low = a.min_p ? a.min_p[g] : 0.f;
    u = a.u ? a.u[r] : draw_uniform(a.draw_key[r], 0);
    ok = T >= 0.f && T <= 0x1p100f && p > 0.f && p <= 1.f && low >= 0.f && low <= 1.f && u >= 0.f && u < 1.f;
    if (T < 0x1p-126f) {   // the first token
      T = 1.f;
      k = 1;
    }
    // what the list of the first tokens is for: top-k, min-p alone, or mass (which may need more)
    by_k = k > 0 && k <= kMaxTop;
    by_min = k <= 0 && p >= 1.f && low > 0.f;
    by_mass = k <= 0 && !by_min;
    as_unset = !a.u && by_mass && p >= 1.f && low == 0.f;
  }
};

DF_DEV void give_row(const SampleArgs& a, int r, int32_t token, float lp, int32_t n) {
  a.token[r] = token;
  if (a.logprob) a.logprob[r] = lp;
  if (a.n_kept) a.n_kept[r] = n;
}

// A row whose kept tokens the list does not hold, or whose borders the sums do not decide.  w.scale
// is set; about: about the row's mass, 0: not known.
template <class E>
__device__ __noinline__ void search_row(RowWork<E>& w, const SampleArgs& a, int r, const Settings& st, uint32_t key_low,
                                        uint64_t about) {
  Shared& s = w.s;
  uint64_t total = 0;
  uint32_t live = 0;
  Border kept{0, 0, 0}, drawn{0, 0, 0};
  uint32_t done = 0;
  if (about && st.by_mass && st.low == 0.f)
    done = w.two_borders(st.p, st.u, about, &total, &live, &kept, &drawn);
  else
    w.count_all(&total, &live);
  if (done == 0) {
    kept = Border{0, total, live};
    if (st.k > 0) {
      const Border b = w.locate(true, min((uint32_t)st.k, live), 0, total);
      if (w.rank == 0) kept = b;
    }
    if (st.p < 1.f) {
      const Border b = w.locate(false, 0, mass_share(st.p, kept.mass), total);
      if (w.rank == 0 && b.n < kept.n) kept = b;
    }
    if (st.low > 0.f) {
      const float from = key_float(key_low);
      if (w.tid == 0) s.mass = 0, s.n_list = 0;
      row_sync(w.ctas);
      MassSum m;
      uint32_t n = 0;
      const MassScale sc = w.scale;
      const float2* const table = s.table;
      for_pieces<4>(w.part, [&](const float* x, int, bool) {
        m.room(RowPart<E>::VE);
#pragma unroll
        for (int e = 0; e < RowPart<E>::VE; ++e)
          if (x[e] >= from) {
            add_mass(m, sc, table, x[e]);
            ++m.n;
            ++n;
          }
      });
      w.give_mass(m, &s.mass);
      n = block_add(n, s.tmp32);
      if (w.tid == 0) add_remote(at_rank(&s.n_list, 0), n);
      row_sync(w.ctas);
      if (w.rank == 0 && s.n_list < kept.n) kept = Border{0, s.mass, s.n_list};
    }
  }
  if (done < 3) drawn = w.locate(false, 0, mass_above(st.u, kept.mass), total);
  if (w.rank == 0 && w.tid == 0) {
    const float l = key_float(key_of(drawn.comp));
    give_row(a, r, id_of(drawn.comp), log_share(w.scale, l, mass_of(w.scale, l), kept.mass), (int32_t)kept.n);
  }
}

// A keyed draw that no setting cuts: the token that the LM head's own temperature draw gives (the argmax over
// logit / T + draw_noise(), in the same operations), so that settings which cut nothing change no text.
template <class E>
__device__ __noinline__ void draw_uncut(Shared& s, const E* row, int V, uint32_t draw, float T, int32_t* token, int* status, int r,
                                        int rank, int ctas) {     // values: the kernel's arguments stay where they are
  if (ctas > 1) cluster_arrive();
  const RowPart<E> part(row, 0, 0, V, rank, ctas);
  const float inv_temp = 1.f / T;
  const int tid = threadIdx.x;
  uint64_t best = 0;       // 0: no token; all bits: a NaN or +inf
  for_pieces<2>(part, [&](const float* x, int piece, bool) {
#pragma unroll
    for (int e = 0; e < RowPart<E>::VE; ++e) {
      if (x[e] == -INFINITY) continue;
      const int id = part.id(piece, e);
      const float v = __fadd_rn(__fmul_rn(x[e], inv_temp), draw_noise(draw, id));
      best = max(best, x[e] < INFINITY ? comp_of(float_key(v), id) : ~(uint64_t)0);
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if ((tid & 31) == 0) s.tmp64[tid >> 5] = best;
  __syncthreads();
  if (ctas > 1) cluster_wait();     // every CTA of the cluster runs before its memory is written
  if (tid == 0) {
    for (int w = 1; w < kRowWarps; ++w) best = max(best, s.tmp64[w]);
    st_remote(at_rank(&s.list[rank], 0), best);
  }
  row_sync(ctas);
  if (rank == 0 && tid == 0) {
    for (int i = 0; i < ctas; ++i) best = max(best, s.list[i]);
    if (best == ~(uint64_t)0) set_status(status, DF_ERR_NAN, r);
    *token = best == 0 || best == ~(uint64_t)0 ? -1 : id_of(best);
  }
}

// grid: rows x CTAs of a row.  SEARCH: rows that need it are searched here, else left to
// search_kernel (a.left).
template <class E, bool SEARCH>
__global__ void __launch_bounds__(kRowThreads, SEARCH ? 2 : 4) sample_kernel(SampleArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int r = blockIdx.x / ctas;
  const Settings st(a, r);
  auto leave = [&](uint64_t about, uint32_t largest, uint32_t on) {
    if (!SEARCH) a.left[r] = SampleLeft{about, largest, on};
  };
  if (!st.ok) {          // the same in every CTA, so all of them leave together
    if (rank == 0 && tid == 0) {
      set_status(a.status, DF_ERR_ARG, r);
      give_row(a, r, -1, -INFINITY, 0);
      leave(0, 0, 0);
    }
    return;
  }
  if (st.as_unset) {
    draw_uncut(s, static_cast<const E*>(a.x.data) + r * a.x.ld, a.x.V, a.draw_key[r], st.T, a.token + r, a.status, r, rank, ctas);
    if (rank == 0 && tid == 0) leave(0, 0, 0);
    return;
  }
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  RowWork<E> w(s, part, rank, ctas);
  typename RowWork<E>::Tops my;
  const bool count = st.by_mass && st.p >= 1.f && a.n_kept;
  // Every CTA finds the first tokens of its own part, if they are few; else the row's are found together.
  const bool parts = st.by_mass || (st.by_k && st.k <= kFewTop);
  if (tid == 0) s.n_list = s.live = 0;
  if (ctas > 1) cluster_arrive();
  const float c = 1.44269504f / st.T;
  uint32_t big = 0, key_low = 0;
  if (st.by_mass) {
    uint32_t live;
    w.template read_tops<true>(my, c, count, &live);
    if (ctas > 1) cluster_wait();   // every CTA of the cluster runs before its memory is written
    w.template list_part<true>(my, kLikely / ctas + 8, c);
    if (count) {
      live = block_add(live, s.tmp32);
      if (tid == 0) add_remote(at_rank(&s.live, 0), live);
    }
  } else {
    w.template read_tops<false>(my, 0.f, false, nullptr);
    if (ctas > 1) cluster_wait();
    if (parts) {
      w.template list_part<false>(my, st.k, 0.f);
    } else {
      w.post_groups(my);
      row_sync(ctas);
      if (rank == 0) {
        const uint32_t least = w.threshold(st.by_k ? st.k : 1, &big);
        const uint32_t word[2] = {big, least};
        w.tell(word, 2);
      }
      row_sync(ctas);
      big = s.word[0];
      uint32_t least = s.word[1];
      if (big > kNegInfKey && big < kPosInfKey && st.k <= kMaxTop) {
        if (st.low > 0.f) key_low = logit_key(least_logit(key_float(big), st.T, st.low, s.tmpf));
        if (st.p >= 1.f) least = st.by_min ? key_low : max(least, key_low);
        w.template list_tops<false>(my, least, 0.f, 0.f);
      }
    }
  }
  row_sync(ctas);
  uint64_t about = 0;
  bool done = false;
  if (rank == 0) {
    uint32_t cut = 0;              // above it the list is complete
    if (parts)
      for (int i = 0; i < ctas; ++i) {
        big = max(big, s.part_max[i]);
        cut = max(cut, s.part_least[i]);
      }
    if (big <= kNegInfKey || big >= kPosInfKey) {   // nothing to draw from; a NaN or +inf
      if (tid == 0) {
        if (big >= kPosInfKey) set_status(a.status, DF_ERR_NAN, r);
        give_row(a, r, -1, -INFINITY, 0);
      }
      done = true;
    } else if (st.k <= kMaxTop && s.n_list <= kListCap) {
      const float largest = key_float(big);
      w.scale.set(st.T, largest);
      if (st.low > 0.f && !key_low) key_low = logit_key(least_logit(largest, st.T, st.low, s.tmpf));
      int n = (int)s.n_list;
      w.sort_list(s.list, n);
      uint64_t tail = 0;
      if (st.by_mass) {
        float t = 0.f;
        int above = 0;
        for (int i = tid; i < n; i += kRowThreads) {
          const uint32_t key = key_of(s.list[i]);
          if (key >= cut) ++above;
          else t += ex2_approx((key_float(key) - largest) * c);
        }
        n = block_add(above, (int*)s.tmp32);
        t = block_add(t, s.tmpf);
        for (int i = 0; i < ctas; ++i)
          if (s.part_max[i] > kNegInfKey) t += s.tail[i] * ex2_approx((key_float(s.part_max[i]) - largest) * c);
        tail = (uint64_t)(t * (float)mass_of(w.scale, largest));
      }
      if (st.by_k) n = min(st.k, n);
      auto give = [&](int32_t token, float lp, int32_t kept) { give_row(a, r, token, lp, kept); };
      if (n > 64)
        done = finish(w, n, !st.by_mass, tail, s.live, st.p, key_low, st.u, a.logprob != nullptr, &about, give);
      else if (tid < 32)
        done = finish_few(w, n, !st.by_mass, tail, s.live, st.p, key_low, st.u, a.logprob != nullptr, &about, give);
    }
  }
  if (!SEARCH) {
    if (rank == 0 && tid == 0) leave(about, big, !done);
    return;
  }
  if (rank == 0 && tid < ctas) {     // of the first warp
    st_remote(at_rank(&s.word[4], tid), big);
    st_remote(at_rank(&s.word[5], tid), (uint32_t)(about != 0));
    st_remote(at_rank(&s.word[6], tid), (uint32_t)done);
  }
  if (rank == 0 && tid == 0) s.mass_2 = about;
  row_sync(ctas);
  if (s.word[6]) return;
  const float largest = key_float(s.word[4]);
  about = rank == 0 ? s.mass_2 : s.word[5];
  __syncthreads();
  w.scale.set(st.T, largest);
  if (st.low > 0.f) key_low = logit_key(least_logit(largest, st.T, st.low, s.tmpf));
  search_row(w, a, r, st, key_low, about);
}

// grid: clusters that take the rows left by sample_kernel in turn.
template <class E>
__global__ void __launch_bounds__(kRowThreads, 2) search_kernel(SampleArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int me = blockIdx.x / ctas, all = gridDim.x / ctas;
  uint32_t mine = 0, n;
#pragma unroll 4
  for (int r = tid; r < a.x.rows; r += kRowThreads) mine += a.left[r].on;
  const uint32_t before = block_scan(mine, s.tmp32, &n);
  bool first = true;
  // this cluster's rows: of all that are left, in the threads' order, me, me + all, ...
  for (uint32_t from = 0; from < n; from += (uint32_t)all * kRowThreads) {
    __syncthreads();
    if (tid == 0) s.n_rows = 0;
    __syncthreads();
    if (mine) {
      uint32_t at = before;
      for (int r = tid; r < a.x.rows; r += kRowThreads) {
        if (!a.left[r].on) continue;
        const uint32_t q = at++ - from;       // wraps around below `from`
        if (q < (uint32_t)all * kRowThreads && q % all == (uint32_t)me) {
          s.rows[q / all] = r;
          atomicAdd(&s.n_rows, 1u);
        }
      }
    }
    __syncthreads();
    const int k = (int)s.n_rows;
    for (int i = 0; i < k; ++i) {
      row_sync(ctas);     // the last row's memory; every CTA of the cluster runs
      first = false;
      const int r = s.rows[i];
      const SampleLeft left = a.left[r];
      const Settings st(a, r);
      const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
      RowWork<E> w(s, part, rank, ctas);
      const float largest = key_float(left.largest);
      w.scale.set(st.T, largest);
      const uint32_t key_low = st.low > 0.f ? logit_key(least_logit(largest, st.T, st.low, s.tmpf)) : 0;
      search_row(w, a, r, st, key_low, left.about);
      __syncthreads();
    }
  }
  // no CTA leaves while another of its cluster may read its memory
  if (!first && ctas > 1) row_sync(ctas);
}

template <class E>
__global__ void __launch_bounds__(kRowThreads, 4) top_logits_kernel(TopArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int r = blockIdx.x / ctas, K = a.K;
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  RowWork<E> w(s, part, rank, ctas);
  typename RowWork<E>::Tops my;
  int32_t* id = a.id + (size_t)r * K;
  float* val = a.val + (size_t)r * K;
  auto fill = [&](int from) {
    for (int i = from + tid; i < K; i += kRowThreads) {
      id[i] = -1;
      val[i] = -INFINITY;
    }
  };
  if (tid == 0) s.n_list = 0;
  if (ctas > 1) cluster_arrive();
  uint32_t live, big = 0;
  const float c = 1.44269504f / a.temperature;
  const bool parts = K <= kFewTop;
  w.template read_tops<true>(my, c, false, &live);
  if (ctas > 1) cluster_wait();     // every CTA of the cluster runs before its memory is written
  if (parts) {
    w.give_sum(my, key_float(w.template list_part<false>(my, K, 0.f)), c);
  } else {
    w.post_groups(my);
    row_sync(ctas);
    if (rank == 0) {
      const uint32_t least = w.threshold(K, &big);
      const uint32_t word[2] = {big, least};
      w.tell(word, 2);
      if (tid < ctas) s.part_max[tid] = big;
    }
    row_sync(ctas);
    big = s.word[0];
    if (big > kNegInfKey && big < kPosInfKey) {
      w.template list_tops<false>(my, s.word[1], 0.f, 0.f);
      w.give_sum(my, key_float(big), c);
    }
  }
  row_sync(ctas);
  bool many = false;
  float largest = 0.f;
  if (rank == 0) {
    for (int i = 0; i < ctas; ++i) big = max(big, s.part_max[i]);
    largest = key_float(big);
    const int n_list = (int)s.n_list;
    if (big <= kNegInfKey || big >= kPosInfKey) {
      fill(0);
      if (tid == 0) {
        if (big >= kPosInfKey) set_status(a.status, DF_ERR_NAN, r);
        if (a.lse) a.lse[r] = big >= kPosInfKey ? NAN : -INFINITY;
      }
    } else {
      many = n_list > kListCap;
      if (!many) {
        w.sort_list(s.list, n_list);
        const int n = min(K, n_list);
        for (int i = tid; i < n; i += kRowThreads) {
          const uint64_t comp = s.list[i];
          id[i] = id_of(comp);
          val[i] = key_float(key_of(comp));
        }
        fill(n);
      }
      if (tid == 0 && a.lse) {
        float sum = 0.f;
        for (int i = 0; i < ctas; ++i)
          if (s.part_max[i] > kNegInfKey) sum += s.sums[i] * ex2_approx((key_float(s.part_max[i]) - largest) * c);
        a.lse[r] = largest / a.temperature + logf(sum);
      }
    }
    if (tid < ctas) {
      st_remote(at_rank(&s.word[6], tid), (uint32_t)many);
      st_remote(at_rank(&s.word[4], tid), big);
    }
  }
  row_sync(ctas);
  if (!s.word[6]) return;
  // many equal logits: the K-th token's place decides
  largest = key_float(s.word[4]);
  w.scale.set(1.f, largest);
  uint64_t total = 0;
  w.count_all(&total, &live);
  const Border b = w.locate(true, min((uint32_t)K, live), 0, total);
  if (rank == 0) {
    const uint32_t word[2] = {(uint32_t)(b.comp >> 32), (uint32_t)b.comp};
    w.tell(word, 2);
  }
  if (tid == 0) s.n_list = 0;
  row_sync(ctas);
  const uint64_t last = ((uint64_t)s.word[0] << 32) | s.word[1];
  for_pieces<4>(part, [&](const float* x, int piece, bool) {
#pragma unroll
    for (int e = 0; e < RowPart<E>::VE; ++e) {
      const uint32_t key = logit_key(x[e]);
      if (comp_of(key, part.id(piece, e)) >= last) w.put(&s.n_list, s.list, kListCap, key, part.id(piece, e));
    }
  });
  w.hand_over(&s.n_list, s.list, kListCap);
  row_sync(ctas);
  if (rank == 0) {
    const int n = min(K, (int)min(s.n_list, (uint32_t)kListCap));
    w.sort_list(s.list, n);
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t comp = s.list[i];
      id[i] = id_of(comp);
      val[i] = key_float(key_of(comp));
    }
    fill(n);
  }
}

template <class A, void (*KERNEL)(A, int)>
int launch_rows(const A& a, int clusters, int ctas, const char* tag, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  if (prepare_kernel(reinterpret_cast<const void*>(KERNEL), sizeof(Shared), done) != cudaSuccess) return DF_ERR_CUDA;
  DF_TRACE(tag, st);
  if (launch_cluster(KERNEL, (unsigned)clusters * ctas, ctas, sizeof(Shared), st, a, ctas) != cudaSuccess) return DF_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

template <class E>
int launch_draws(const SampleArgs& a, cudaStream_t st) {
  const int rows = a.x.rows, sms = num_sms(), ctas = row_ctas(rows, a.x.V, 2 * sms), most = row_ctas(1, a.x.V, 2 * sms);
  // Few rows have all the CTAs that a search wants from the start; among many, rows to be searched
  // get them from a second launch (also of small rows: with the search in it a kernel has two CTAs an
  // SM, without four; 4096 rows of 1000, 193 us against 117).
  if (ctas == most && (long long)rows * ctas <= 2 * sms)
    return launch_rows<SampleArgs, sample_kernel<E, true>>(a, rows, ctas, "sample", st);
  const int rc = launch_rows<SampleArgs, sample_kernel<E, false>>(a, rows, ctas, "sample", st);
  if (rc != DF_OK) return rc;
  // Clusters of 4, as many as are resident at two CTAs to an SM (of 8 and at four CTAs, the last
  // clusters began when others were through: 73 rows of 151936, 190 us against 173); of 2 where so
  // many rows may be left that clusters of 4 would take them in turns (by mass alone, 1024 rows of
  // 100000: 335 us against 496, 2064 mixed rows of 151936: 354 against 385; but 256 rows: 299 against 224).
  const int search = std::max(ctas, std::min(most, rows > 4 * sms ? 2 : 4));
  return launch_rows<SampleArgs, search_kernel<E>>(a, std::min(rows, 2 * sms / search), search, "sample_search", st);
}

}  // namespace

int launch_sample(const SampleArgs& a, cudaStream_t st) {
  return a.x.dtype == DF_F32 ? launch_draws<float>(a, st) : launch_draws<uint16_t>(a, st);
}
int launch_top_logits(const TopArgs& a, cudaStream_t st) {
  const int ctas = row_ctas(a.x.rows, a.x.V, 2 * num_sms());
  return a.x.dtype == DF_F32 ? launch_rows<TopArgs, top_logits_kernel<float>>(a, a.x.rows, ctas, "top_logits", st)
                             : launch_rows<TopArgs, top_logits_kernel<uint16_t>>(a, a.x.rows, ctas, "top_logits", st);
}

int row_ctas(int rows, int V, int most) {
  int c = 1;
  while (c < 8 && (long long)rows * c * 2 <= most && V >= 4096 * c) c *= 2;
  while (c < 8 && V > (1 << 18) * c) c *= 2;   // a thread's sums and a CTA's bitmap are made for 2^18 elements
  return c;
}

}  // namespace df
