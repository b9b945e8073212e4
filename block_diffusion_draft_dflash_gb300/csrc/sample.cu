// Draws under top-k, top-p and min-p from rows of logits, and rows' largest logits.
//
// A row's tokens stand in order of (logit descending, id ascending), as numbers comp = key << 32
// | ~id that are all different (key: the logit as an order-preserving integer).  Every filter
// keeps a prefix of that order, so a draw needs borders in it: the comp at which a count or a
// mass is reached.
//
// Few tokens (top-k up to 1024, the largest logits): one pass keeps the largest logit of each of
// up to 4096 groups (the elements that one thread reads).  The k-th largest of these is a lower
// bound of the k-th largest logit, and only the few groups that reach it are read again (from
// L2): hardly more than k candidates, which one CTA sorts.
// Any number of tokens: a second pass sums the masses and counts tokens in 1024 bins of 1/16 of
// a power of two of probability.  The counts say in which bin a border should lie; a third pass
// sums the mass before that bin and its neighbours exactly and lists their tokens, and if the
// border is not among them the next bin is chosen between exact masses.  Where a bin has too many
// tokens, its range of keys is cut by 1024 again until one key is left, whose tokens stand in
// order of their ids.
#include "rows.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {
namespace {

constexpr int kListCap = 2048;     // candidates that one CTA sorts
constexpr int kMaxTop = 1024;      // tokens that the first way can find
constexpr int kBins = 1024;
constexpr int kMaxGroups = 4096;
constexpr uint32_t kAround = 512;  // tokens listed on either side of the bin where a border should be

__device__ const Pow2Table kPow2;

struct Bins {          // running sums over bins: tokens, and about their mass
  uint32_t count[kBins];
  float mass[kBins];
};
struct Shared {
  union {
    uint32_t group_key[kMaxGroups];          // of the whole row, in the first CTA
    uint64_t list[kListCap];                 // candidates, in the first CTA
  };
  Bins bins, fine;
  uint32_t hist[kBins];
  float t_hi[1024], t_lo[1024];
  // written by the first CTA in every CTA
  uint32_t word[8];
  // collected in the first CTA
  uint64_t mass, mass_in;
  uint32_t n_list, key_min, key_max, equal[8], at_id;
  // one CTA's own
  uint64_t tmp64[kRowWarps];
  uint32_t tmp32[kRowWarps];
  float tmpf[kRowWarps];
  uint64_t found_comp, found_mass;
  uint32_t found_n, found;
};

DF_DEV uint32_t logit_key(float l) { return float_key(l + 0.f); }   // -0 as +0
DF_DEV uint64_t comp_of(uint32_t key, int id) { return ((uint64_t)key << 32) | (uint32_t)~id; }
DF_DEV uint32_t key_of(uint64_t comp) { return (uint32_t)(comp >> 32); }
DF_DEV int id_of(uint64_t comp) { return (int)~(uint32_t)comp; }

// A border in the order: its token, the tokens up to it and their mass.
struct Border {
  uint64_t comp, mass;
  uint32_t n;
};

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

  // -------------------------------------------------------------------------- largest logits
  int sub;             // groups of a thread: 4 / ctas, at least 1
  float top[4];        // their largest logits (the first `sub`)

  // Reads the row; SUMS: also a running log-sum (max, sum of 2^((l - max) c)) of the thread.
  template <bool SUMS>
  DF_DEV void read_tops(float c, float* run_max, float* run_sum) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    float rm = -INFINITY, rs = 0.f;
    for (int i = part.lo + tid; i < part.hi; i += 4 * kRowThreads) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = i + j * kRowThreads < part.hi ? part.load(i + j * kRowThreads) : RowPart<E>::nothing();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float big = RowOf<E>::largest(v[j]);
        m[j] = max_nan(m[j], big);
        if (SUMS && big > -INFINITY) {
          if (big > rm) {
            rs *= ex2_approx((rm - big) * c);
            rm = big;
          }
          float x[VE];
          RowOf<E>::unpack(v[j], x);
#pragma unroll
          for (int e = 0; e < VE; ++e) rs += ex2_approx((x[e] - rm) * c);
        }
      }
    }
    sub = ctas == 1 ? 4 : ctas == 2 ? 2 : 1;
    if (sub == 4) {
      top[0] = m[0]; top[1] = m[1]; top[2] = m[2]; top[3] = m[3];
    } else {
      top[0] = max_nan(m[0], m[1]);
      top[1] = max_nan(m[2], m[3]);
      if (sub == 1) top[0] = max_nan(top[0], top[1]);
    }
    if (SUMS) { *run_max = rm; *run_sum = rs; }
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (g < sub)
        st_remote(at_rank(&s.group_key[(rank * sub + g) * kRowThreads + tid], 0),
                  top[g] == top[g] ? logit_key(top[g]) : 0xFFFFFFFFu);
  }

  // First CTA, behind a row_sync: the largest key, and for k > 0 a key that at least k of the
  // groups reach (at least 1 above -inf's).
  DF_DEV uint32_t threshold(int k, uint32_t* largest) {
    uint32_t key[8];
    uint32_t big = 0;
    const int n = ctas * sub;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      key[j] = j < n ? s.group_key[j * kRowThreads + tid] : 0;
      big = max(big, key[j]);
    }
    big = __reduce_max_sync(0xffffffffu, big);
    __syncthreads();
    if ((tid & 31) == 0) s.tmp32[tid >> 5] = big;
    __syncthreads();
    big = __reduce_max_sync(0xffffffffu, s.tmp32[tid & (kRowWarps - 1)]);
    *largest = big;
    if (k <= 1 || big <= kNegInfKey || big >= kPosInfKey) return big;
    // lo: reached by k groups or the smallest finite key; hi: reached by fewer
    uint32_t lo = kNegInfKey + 1, hi = big;
    const int enough = k + (k >> 3) + 4;
    for (int step = 0; step < 32 && hi - lo > 1; ++step) {
      const uint32_t mid = lo + ((hi - lo) >> 1);
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) c += key[j] >= mid;
      c = block_add(c, s.tmp32);
      if ((int)c >= k) {
        lo = mid;
        if ((int)c <= enough) break;
      } else {
        hi = mid;
      }
    }
    return lo;
  }

  // Every warp puts the elements that reach `least` of its threads' groups on the first CTA's list.
  DF_DEV void list_tops(uint32_t least) {
    const int lane = tid & 31, per = 4 / sub;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g >= sub) break;
      uint32_t who = __ballot_sync(0xffffffffu, logit_key(top[g]) >= least);
      while (who) {
        const int t0 = (tid & ~31) + __ffs(who) - 1;
        who &= who - 1;
        for (int q = lane;; q += 32) {
          const int i = part.lo + t0 + (g * per + q % per) * kRowThreads + (q / per) * 4 * kRowThreads;
          if (part.lo + t0 + (q / per) * 4 * kRowThreads >= part.hi) break;
          if (i >= part.hi) continue;
          float x[VE];
          RowOf<E>::unpack(part.load(i), x);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const uint32_t key = logit_key(x[e]);
            if (key >= least) put(key, part.id(i, e));
          }
        }
      }
    }
  }
  DF_DEV void put(uint32_t key, int id) {
    const uint32_t n = add_remote(at_rank(&s.n_list, 0), 1u);
    if (n < kListCap) st_remote(at_rank(&s.list[n], 0), comp_of(key, id));
  }

  // One CTA: the list's first n entries in order.
  DF_DEV void sort_list(int n) {
    if (n <= kRowThreads) {
      // an entry's place is the number of entries before it; several threads count for one
      int share = 1;
      while (share < 32 && n * share * 2 <= kRowThreads) share *= 2;
      const int e = tid / share, part_of = tid % share;
      uint64_t mine = 0;
      uint32_t place = 0;
      if (e < n) {
        mine = s.list[e];
        for (int i = part_of; i < n; i += share) place += s.list[i] > mine;
      }
      for (int o = share / 2; o > 0; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
      __syncthreads();
      if (e < n && part_of == 0) s.list[place] = mine;
      __syncthreads();
      return;
    }
    for (int i = n + tid; i < kListCap; i += kRowThreads) s.list[i] = 0;
    const int size = n <= 1024 ? 1024 : kListCap;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = tid; i < size / 2; i += kRowThreads) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const uint64_t x = s.list[a], y = s.list[b];
          if ((x < y) == ((a & k) == 0)) {
            s.list[a] = y;
            s.list[b] = x;
          }
        }
        __syncthreads();
      }
  }

  // One CTA, sorted list of n entries behind n_before tokens of mass_before: the border where the
  // tokens reach want_n or the mass reaches `want`.  False: it is not here; *mass_after: behind the list.
  DF_DEV bool border_in_list(int n, uint32_t n_before, uint64_t mass_before, bool by_count, uint32_t want_n,
                             uint64_t want, uint64_t* mass_after, Border* found) {
    constexpr int PER = kListCap / kRowThreads;
    uint64_t w[PER], mine = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j;
      w[j] = i < n ? mass_of(scale, kPow2.hi, kPow2.lo, key_float(key_of(s.list[i]))) : 0;
      mine += w[j];
    }
    if (tid == 0) s.found = 0;
    uint64_t run = mass_before + block_scan(mine, s.tmp64, &all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint64_t before = run;
      run += w[j];
      const int i = tid * PER + j;
      if (i < n && (by_count ? n_before + i + 1 == want_n : before < want && run >= want)) {
        s.found_comp = s.list[i];
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
    for (int i = tid; i < 1024; i += kRowThreads) {
      s.t_hi[i] = kPow2.hi[i];
      s.t_lo[i] = kPow2.lo[i];
    }
  }
  DF_DEV void add(MassSum& m, float l) {
    add_mass(m, scale, s.t_hi, s.t_lo, l);
    if (m.n == 512) m.fold();
  }
  DF_DEV void give_mass(MassSum& m, uint64_t* to) {   // to the first CTA's
    m.fold();
    const uint64_t sum = block_add(m.sum, s.tmp64);
    if (tid == 0 && sum) add_remote(at_rank(to, 0), sum);
  }
  DF_DEV uint32_t bin_of(float l) const { return min((scale.top - scale.bits(l)) >> 6, (uint32_t)kBins - 1); }

  // First CTA: running sums of the cluster's histograms; weight(b): about a token's mass in bin b.
  template <class W>
  DF_DEV void run_bins(Bins& to, W&& weight) {
    constexpr int PER = kBins / kRowThreads;
    uint32_t c[PER] = {}, n = 0, all_n;
    float w[PER], mine = 0.f, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int b = tid * PER + j;
      for (int r = 0; r < ctas; ++r) c[j] += ld_remote(at_rank(&s.hist[b], r));
      w[j] = c[j] ? (float)c[j] * weight(b) : 0.f;
      n += c[j];
      mine += w[j];
    }
    uint32_t rn = block_scan(n, s.tmp32, &all_n);
    float rw = block_scan(mine, s.tmpf, &all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int b = tid * PER + j;
      rn += c[j]; rw += w[j];
      to.count[b] = rn;
      to.mass[b] = rw;
    }
    __syncthreads();
  }

  // Sums all masses and counts tokens in bins.  First CTA: *total, *live = tokens above -inf.
  __device__ __noinline__ void count_all(uint64_t* total, uint32_t* live) {
    for (int b = tid; b < kBins; b += kRowThreads) s.hist[b] = 0;
    if (tid == 0) s.mass = 0;
    load_table();
    row_sync(ctas);
    MassSum m;
    for_pieces<4>(part, [&](const float* x, int) {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (x[e] > -INFINITY) {
          add(m, x[e]);
          atomicAdd(&s.hist[bin_of(x[e])], 1u);
        }
    });
    give_mass(m, &s.mass);
    row_sync(ctas);
    if (rank == 0) {
      run_bins(s.bins, [](int b) { return exp2f(-((float)b + 0.5f) * (1.f / 16.f)); });
      *total = s.mass;
      *live = s.bins.count[kBins - 1];
    }
  }

  // The part of a search that a level's bins are left with (first CTA): the border lies in bins
  // first .. last; before them n0 + count[first - 1] tokens and mass m0, with them mass m1.
  struct Window {
    uint32_t first, last, n0;
    uint64_t m0, m1;
  };
  // First CTA: the bin where the border should be (exactly, for a count), with some around it as
  // far as their tokens fit in the list.  Words 0, 1: first and last bin, 2: their tokens.
  DF_DEV void choose(const Bins& of, const Window& v, int tries, bool by_count, uint32_t want_n, uint64_t want,
                     uint32_t* w) {
    constexpr int PER = kBins / kRowThreads;
    const float e0 = v.first ? of.mass[v.first - 1] : 0.f, e1 = of.mass[v.last];
    const float e = e0 + (float)(want - v.m0) / (float)(v.m1 - v.m0) * (e1 - e0);
    uint32_t at = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int b = tid * PER + j;
      at += by_count ? v.n0 + of.count[b] < want_n : of.mass[b] < e;
    }
    at = min(max(block_add(at, s.tmp32), v.first), v.last);
    if (!by_count && tries >= 3) at = v.first + (v.last - v.first) / 2;   // the masses mislead
    const uint32_t upto = of.count[at], before = at ? of.count[at - 1] : 0;
    uint32_t less = 0, more = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t b = tid * PER + j, c0 = b ? of.count[b - 1] : 0;
      less += b >= v.first && b < at && before - c0 <= kAround;
      more += b > at && b <= v.last && of.count[b] - upto <= kAround;
    }
    less = block_add(less, s.tmp32);
    more = block_add(more, s.tmp32);
    if (by_count || upto - before > kListCap - 2 * kAround) less = more = 0;
    w[0] = at - less;
    w[1] = at + more;
    w[2] = of.count[w[1]] - (w[0] ? of.count[w[0] - 1] : 0);
  }
  // All CTAs: mass before the window (s.mass); its tokens on the list if they fit, else their mass
  // (s.mass_in) and range of keys.  bin(l, key): a logit's bin of this level, above kBins: none.
  template <class B>
  DF_DEV void read_window(B&& bin) {
    const uint32_t b1 = s.word[0], b2 = s.word[1];
    const bool few = s.word[2] <= kListCap;
    MassSum m, in;
    uint32_t kmin = 0xFFFFFFFFu, kmax = 0;
    for_pieces<4>(part, [&](const float* x, int piece) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint32_t key = logit_key(x[e]), b = bin(x[e], key);
        if (b > b2) continue;
        if (b < b1) {
          add(m, x[e]);
        } else if (few) {
          put(key, part.id(piece, e));
        } else {
          add(in, x[e]);
          kmin = min(kmin, key);
          kmax = max(kmax, key);
        }
      }
    });
    give_mass(m, &s.mass);
    if (few) return;
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
  DF_DEV uint32_t search(const Bins& of, Window* lv, bool by_count, uint32_t want_n, uint64_t want, Border* found, B&& bin) {
    const uint64_t base = lv->m0;      // mass before the level's bins
    for (int tries = 0; tries < 16; ++tries) {
      uint32_t w[3];
      if (rank == 0) {
        choose(of, *lv, tries, by_count, want_n, want, w);
        tell(w, 3);
        if (tid == 0) { s.mass = s.mass_in = 0; s.n_list = 0; s.key_min = 0xFFFFFFFFu; s.key_max = 0; }
      }
      row_sync(ctas);
      read_window(bin);
      row_sync(ctas);
      if (rank == 0) {
        const uint32_t n_before = lv->n0 + (w[0] ? of.count[w[0] - 1] : 0);
        const uint64_t before = base + s.mass;
        uint64_t after = before + s.mass_in;
        uint32_t next = kAgain;
        if (w[2] <= kListCap) {
          const int n = (int)min(s.n_list, (uint32_t)kListCap);
          sort_list(n);
          if (border_in_list(n, n_before, before, by_count, want_n, want, &after, found)) next = kFound;
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
          word[1] = (uint32_t)max(0, 32 - __clz(word[2] - word[3]) - 10);
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
    uint32_t next = search(s.bins, &lv, by_count, want_n, want, &found, [&](float l, uint32_t) {
      return l > -INFINITY ? bin_of(l) : 0xFFFFFFFFu;
    });
    // Too many tokens in one bin: cut its keys into 1024 bins again, until they fit or one key is left.
    for (int level = 0; level < 4 && next == kDeeper; ++level) {
      const uint32_t shift = s.word[4], hi = s.word[5], lo = s.word[6];
      if (hi == lo) break;
      for (int b = tid; b < kBins; b += kRowThreads) s.hist[b] = 0;
      row_sync(ctas);
      for_pieces<4>(part, [&](const float* x, int) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const uint32_t key = logit_key(x[e]);
          if (key >= lo && key <= hi) atomicAdd(&s.hist[(hi - key) >> shift], 1u);
        }
      });
      row_sync(ctas);
      if (rank == 0)
        run_bins(s.fine, [&](int b) {
          const uint32_t mid = ((uint32_t)b << shift) + (shift ? 1u << (shift - 1) : 0);
          return (float)mass_of(scale, kPow2.hi, kPow2.lo, key_float(hi - min(mid, hi - lo)));
        });
      next = search(s.fine, &lv, by_count, want_n, want, &found, [&](float, uint32_t key) {
        return key >= lo && key <= hi ? (hi - key) >> shift : 0xFFFFFFFFu;
      });
    }
    if (next == kDeeper) one_key(s.word[5], lv, by_count, want_n, want, &found);
    row_sync(ctas);
    return found;
  }

  // All tokens of the bin have one key: in order of their ids.
  DF_DEV void one_key(uint32_t key, const Window& lv, bool by_count, uint32_t want_n, uint64_t want, Border* found) {
    uint32_t mine = 0;
    for_pieces<4>(part, [&](const float* x, int) {
#pragma unroll
      for (int e = 0; e < VE; ++e) mine += logit_key(x[e]) == key;
    });
    mine = block_add(mine, s.tmp32);
    if (tid == 0) st_remote(at_rank(&s.equal[rank], 0), mine);
    row_sync(ctas);
    if (rank == 0) {
      const uint64_t w = mass_of(scale, kPow2.hi, kPow2.lo, key_float(key));
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
      for (int i0 = part.lo; i0 < part.hi; i0 += kRowThreads) {
        const int i = i0 + tid;
        float x[VE];
        RowOf<E>::unpack(i < part.hi ? part.load(i) : RowPart<E>::nothing(), x);
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
DF_DEV float log_share(const MassScale& c, float l, uint64_t w, uint64_t m) {
  if (2 * w >= m) return log1pf(-((float)(m - w) / (float)m));
  const float x = c.arg(l), t = fmaf(x, c.c_hi, c.shift), g = t - c.shift;
  float r = fmaf(x, c.c_hi, -g);
  r = fmaf(x, c.c_lo, r);
  // y = l c - ref = (t - 12288) + r
  const float y = (t - 12288.f) + r;
  return 0.693147180559945f * (y - log2f((float)m * kMassUnit));
}

// grid: rows x CTAs of a row.  Bound by the row's bytes where the few-token way decides.
template <class E>
__global__ void __launch_bounds__(kRowThreads) sample_kernel(SampleArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int r = blockIdx.x / ctas;
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  RowWork<E> w(s, part, rank, ctas);
  const int g = r / a.group;
  float T = a.temperature ? a.temperature[g] : 1.f;
  int k = a.top_k ? a.top_k[g] : 0;
  const float p = a.top_p ? a.top_p[g] : 1.f, low = a.min_p ? a.min_p[g] : 0.f, u = a.u[r];
  auto give = [&](int32_t token, float lp, int32_t n) {
    a.token[r] = token;
    if (a.logprob) a.logprob[r] = lp;
    if (a.n_kept) a.n_kept[r] = n;
  };
  // the row's settings: the same in every CTA, so all of them leave together
  if (!(T >= 0.f && T <= 0x1p100f) || !(p > 0.f && p <= 1.f) || !(low >= 0.f && low <= 1.f) || !(u >= 0.f && u < 1.f)) {
    if (rank == 0 && tid == 0) {
      set_status(a.status, DF_ERR_ARG, r);
      give(-1, -INFINITY, 0);
    }
    return;
  }
  if (T < 0x1p-126f) {   // the first token
    T = 1.f;
    k = 1;
  }
  const bool few = k > 0 && k <= kMaxTop;
  if (tid == 0) s.n_list = 0;
  if (ctas > 1) row_sync(ctas);   // every CTA of the cluster runs before its memory is written
  w.template read_tops<false>(0.f, nullptr, nullptr);
  row_sync(ctas);
  if (rank == 0) {
    uint32_t big;
    const uint32_t least = w.threshold(few ? k : 1, &big);
    const uint32_t word[2] = {big, least};
    w.tell(word, 2);
  }
  row_sync(ctas);
  const uint32_t big = s.word[0], least = s.word[1];
  if (big <= kNegInfKey || big >= kPosInfKey) {   // nothing to draw from; a NaN or +inf
    if (rank == 0 && tid == 0) {
      if (big >= kPosInfKey) set_status(a.status, DF_ERR_NAN, r);
      give(-1, -INFINITY, 0);
    }
    return;
  }
  const float largest = key_float(big);
  w.scale.set(T, largest);
  if (few) {
    w.list_tops(least);
    row_sync(ctas);
    const uint32_t n_list = ctas == 1 ? s.n_list : ld_remote(at_rank(&s.n_list, 0));
    if (ctas > 1) cluster_arrive();
    if (n_list <= kListCap) {
      if (rank == 0) {
        w.sort_list((int)n_list);
        const int n_k = min(k, (int)n_list);
        constexpr int PER = kMaxTop / kRowThreads;
        uint64_t m[PER], mine = 0, total;
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int i = tid * PER + j;
          key[j] = i < n_k ? key_of(s.list[i]) : 0;
          m[j] = i < n_k ? mass_of(w.scale, kPow2.hi, kPow2.lo, key_float(key[j])) : 0;
          mine += m[j];
        }
        const uint64_t run = block_scan(mine, s.tmp64, &total);
        uint32_t n = (uint32_t)n_k;
        if (p < 1.f || low > 0.f) {
          const uint64_t share = p < 1.f ? mass_share(p, total) : total;
          const uint32_t key_low = low > 0.f ? logit_key(least_logit(largest, T, low, s.tmpf)) : 0;
          uint32_t c = 0;
          uint64_t before = run;
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            c += tid * PER + j < n_k && (before < share || p >= 1.f) && key[j] >= key_low;
            before += m[j];
          }
          n = block_add(c, s.tmp32);
        }
        mine = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (tid * PER + j >= (int)n) m[j] = 0;
          else mine += m[j];
        total = block_add(mine, s.tmp64);
        const uint64_t want = mass_above(u, total);
        uint64_t at = run;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const uint64_t before = at;
          at += m[j];
          if (before < want && at >= want) {
            const uint64_t comp = s.list[tid * PER + j];
            give(id_of(comp), a.logprob ? log_share(w.scale, key_float(key[j]), m[j], total) : 0.f, (int32_t)n);
          }
        }
      }
      if (ctas > 1) cluster_wait();
      return;
    }
    if (ctas > 1) cluster_wait();
  }
  // any number of tokens
  uint64_t total = 0;
  uint32_t live = 0;
  w.count_all(&total, &live);
  Border top{0, total, live};
  if (k > 0) {
    const Border b = w.locate(true, min((uint32_t)k, live), 0, total);
    if (rank == 0) top = b;
  }
  Border kept = top;
  if (p < 1.f) {
    const Border b = w.locate(false, 0, mass_share(p, top.mass), total);
    if (rank == 0 && b.n < kept.n) kept = b;
  }
  if (low > 0.f) {
    const float from = least_logit(largest, T, low, s.tmpf);
    if (tid == 0) { s.mass = 0; s.n_list = 0; }
    row_sync(ctas);
    MassSum m;
    uint32_t n = 0;
    for_pieces<4>(part, [&](const float* x, int) {
#pragma unroll
      for (int e = 0; e < RowPart<E>::VE; ++e)
        if (x[e] >= from) {
          w.add(m, x[e]);
          ++n;
        }
    });
    w.give_mass(m, &s.mass);
    n = block_add(n, s.tmp32);
    if (tid == 0) add_remote(at_rank(&s.n_list, 0), n);
    row_sync(ctas);
    if (rank == 0 && s.n_list < kept.n) kept = Border{0, s.mass, s.n_list};
  }
  const Border b = w.locate(false, 0, mass_above(u, kept.mass), total);
  if (rank == 0 && tid == 0) {
    const float l = key_float(key_of(b.comp));
    give(id_of(b.comp), log_share(w.scale, l, mass_of(w.scale, kPow2.hi, kPow2.lo, l), kept.mass), (int32_t)kept.n);
  }
}

template <class E>
__global__ void __launch_bounds__(kRowThreads) top_logits_kernel(TopArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int r = blockIdx.x / ctas, K = a.K;
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  RowWork<E> w(s, part, rank, ctas);
  int32_t* id = a.id + (size_t)r * K;
  float* val = a.val + (size_t)r * K;
  auto fill = [&](int from) {
    for (int i = from + tid; i < K; i += kRowThreads) {
      id[i] = -1;
      val[i] = -INFINITY;
    }
  };
  if (tid == 0) s.n_list = 0;
  if (ctas > 1) row_sync(ctas);
  float rm, rs;
  const float c = 1.44269504f / a.temperature;
  w.template read_tops<true>(c, &rm, &rs);
  row_sync(ctas);
  if (rank == 0) {
    uint32_t big;
    const uint32_t least = w.threshold(K, &big);
    const uint32_t word[2] = {big, least};
    w.tell(word, 2);
  }
  row_sync(ctas);
  const uint32_t big = s.word[0], least = s.word[1];
  if (big <= kNegInfKey || big >= kPosInfKey) {
    if (rank == 0) {
      fill(0);
      if (tid == 0) {
        if (big >= kPosInfKey) set_status(a.status, DF_ERR_NAN, r);
        if (a.lse) a.lse[r] = big >= kPosInfKey ? NAN : -INFINITY;
      }
    }
    return;
  }
  const float largest = key_float(big);
  // the CTA's share of the log-sum, to the first CTA
  {
    const float sum = block_add(rm > -INFINITY ? rs * ex2_approx((rm - largest) * c) : 0.f, s.tmpf);
    if (tid == 0) st_remote(at_rank(&s.hist[rank], 0), sum);
  }
  w.list_tops(least);
  row_sync(ctas);
  if (rank == 0 && tid == 0 && a.lse) {
    float sum = 0.f;
    for (int i = 0; i < ctas; ++i) sum += __uint_as_float(s.hist[i]);
    a.lse[r] = largest / a.temperature + logf(sum);
  }
  const uint32_t n_list = ctas == 1 ? s.n_list : ld_remote(at_rank(&s.n_list, 0));
  int n_have = (int)min(n_list, (uint32_t)kListCap);
  if (n_list > kListCap) {   // many equal logits: the K-th token's place decides
    row_sync(ctas);
    w.scale.set(1.f, largest);
    uint64_t total = 0;
    uint32_t live = 0;
    w.count_all(&total, &live);
    const Border b = w.locate(true, min((uint32_t)K, live), 0, total);
    if (rank == 0) {
      const uint32_t word[2] = {(uint32_t)(b.comp >> 32), (uint32_t)b.comp};
      w.tell(word, 2);
      if (tid == 0) s.n_list = 0;
    }
    row_sync(ctas);
    const uint64_t last = ((uint64_t)s.word[0] << 32) | s.word[1];
    for_pieces<4>(part, [&](const float* x, int piece) {
#pragma unroll
      for (int e = 0; e < RowPart<E>::VE; ++e) {
        const uint32_t key = logit_key(x[e]);
        if (comp_of(key, part.id(piece, e)) >= last) w.put(key, part.id(piece, e));
      }
    });
    row_sync(ctas);
    n_have = (int)min(s.n_list, (uint32_t)kListCap);   // of the first CTA
  } else if (ctas > 1) {
    cluster_arrive();
  }
  if (rank == 0) {
    w.sort_list(n_have);
    const int n = min(K, n_have);
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t comp = s.list[i];
      id[i] = id_of(comp);
      val[i] = key_float(key_of(comp));
    }
    fill(n);
  }
  if (n_list <= kListCap && ctas > 1) cluster_wait();
}

template <class A, class F>
int launch_rows(F f32, F b16, const A& a, const df_rows& x, const char* tag, cudaStream_t st) {
  const int ctas = row_ctas(x.rows, x.V);
  F f = x.dtype == DF_F32 ? f32 : b16;
  if (ensure_dynamic_smem(f, sizeof(Shared)) != cudaSuccess) return DF_ERR_CUDA;
  DF_TRACE(tag, st);
  if (launch_cluster(f, (unsigned)x.rows * ctas, ctas, sizeof(Shared), st, a, ctas) != cudaSuccess) return DF_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

}  // namespace

int launch_sample(const SampleArgs& a, cudaStream_t st) {
  return launch_rows(sample_kernel<float>, sample_kernel<uint16_t>, a, a.x, "sample", st);
}
int launch_top_logits(const TopArgs& a, cudaStream_t st) {
  return launch_rows(top_logits_kernel<float>, top_logits_kernel<uint16_t>, a, a.x, "top_logits", st);
}

int row_ctas(int rows, int V) {
  int c = 1;
  while (c < 8 && (long long)rows * c < 2LL * num_sms() && V >= 4096 * c) c *= 2;
  while (c < 8 && V > (1 << 18) * c) c *= 2;   // a thread's sums and a CTA's bitmap are made for 2^18 elements
  return c;
}

}  // namespace df
