// Distillation from a teacher's top logits: loss of student rows and its gradient.
//
// With e_j = exp((z_j - m) / T), m the row's largest logit, S = sum of e_j over all tokens and R
// over those outside the teacher's list (t_i, rho):
//   loss / weight = sum_i t_i (ln t_i - (z_i - m) / T) + sum t ln S + rho (ln rho - ln(R / S))
//   gradient = weight / T (e_j / S - t_j) in the list, weight / T e_j / R (R / S - rho) outside,
//   where sum t + rho = 1 (else e_j / S and R / S are times that)
// R is summed over the tokens outside (a bit for each token marks the list), not taken as S minus
// the list's part: where the student is sure of the list, that difference has no digits left.  It is
// summed relative to the largest logit outside, m', and e_j / R is made from z_j - m' or, from kept
// statistics, from the difference of exponents: relative to m all of it falls to 0 where m' lies 87 T
// below m.  ln R is kept in two floats where it is below -64 (in one its rounding is that of the shares
// e_j / R), and from 2^30 on, where two have no digits for them either, the others count as masked.
// Both passes are bound by the row's bytes: loss reads a row once; with the gradient a row is read
// again from L2 by the CTAs that just read it, and written.  512 threads a CTA: a list's 1024 entries
// are two a thread, and a row's CTAs are few.  Measured with rows of 151936 on one GB300, whole calls:
// 240 rows fp32, loss alone 35 us (4.2 TB/s); 960 rows bf16 with the gradient 131 us (4.5 TB/s of what
// has to move); 960 rows fp32, gradient from kept statistics, 174 us (6.7 TB/s, the copy rate);
// 15 rows fp32 with the gradient 13 us, of which 11 in a graph.
#define DF_ROW_THREADS 512
#include "rows.cuh"
#include "runtime.h"
#include "trace.h"

namespace df {
namespace {

constexpr int kMaxList = 1024;
constexpr int kPer = kMaxList / kRowThreads;   // entries of a thread

// What a CTA tells the others of its part of a row, as floats: the largest logit, the largest outside
// the list, the sum of exp((z - that) / T) outside the list, that of exp((z - largest) / T) in it, the sums of
// t_i (ln t_i - (z_i - largest) / T) and of t_i, and flags (1: NaN or +inf, 2: a bad list).
enum { kLargest, kLargestRest, kRest, kListed, kCross, kT, kFlags, kPosts };
struct Shared {
  float post[8][kPosts];   // of every CTA of the row
  float tmp[kRowWarps], tmp2[kRowWarps];
  uint32_t flags;
};
constexpr float kFar = -64.f;         // below it ln R is kept in two floats
constexpr float kMasked = -0x1p30f;   // (m' - m) / T below which the tokens outside count as masked

// Largest number of the warp, in one instruction (NaN only where all are).
DF_DEV float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / T in two floats, and log2(e) / T.
struct Temper {
  float hi, lo, c;
  DF_DEV explicit Temper(float T) {
    hi = 1.f / T;
    lo = fmaf(-hi, T, 1.f) / T;
    c = 1.44269504f * hi;
  }
  // x / T, and x / T - minus (finite); infinite where x hi is, whatever x lo, which may be infinite as well, says
  DF_DEV float over(float x) const {
    const float p = x * hi;
    return fabsf(p) < INFINITY ? fmaf(x, hi, x * lo) : p;
  }
  DF_DEV float over(float x, float minus) const {
    const float p = x * hi;
    return fabsf(p) < INFINITY ? fmaf(x, hi, -minus) + x * lo : p;
  }
};

// A thread's entries of a teacher's list: entry tid + 512 j.
struct Entries {
  int id[kPer];
  float ln_t[kPer], t[kPer];
  float sum;             // of all t of the list
  float rho, all;        // what is left for the others, and sum + rho: 1 where lse is the list's
  uint32_t bad;          // of this thread's entries

  DF_DEV void load(const DistillArgs& a, const Temper& T, int list, float* tmp) {
    const int V = a.x.V;
    float lse = 0.f;
    bad = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = (int)threadIdx.x + j * kRowThreads;
      id[j] = -1;
      ln_t[j] = -INFINITY;
      if (i < a.K) {
        id[j] = a.id[(size_t)list * a.K + i];
        ln_t[j] = a.val[(size_t)list * a.K + i];
      }
    }
    if (a.lse) lse = a.lse[list];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (id[j] < -1 || id[j] >= V) {
        bad |= 2;
        id[j] = -1;
      }
      if (id[j] < 0)
        ln_t[j] = -INFINITY;
      else if (!(ln_t[j] < INFINITY))
        bad |= 1;
    }
    if (a.lse) {
      if (!(fabsf(lse) < INFINITY)) bad |= 1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) ln_t[j] = ln_t[j] > -INFINITY ? T.over(ln_t[j], lse) : -INFINITY;
    } else {
      // softmax over the list
      float m = ln_t[0];
#pragma unroll
      for (int j = 1; j < kPer; ++j) m = max_nan(m, ln_t[j]);
      m = warp_max(m);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = m;
      __syncthreads();
      m = warp_max(tmp[threadIdx.x & (kRowWarps - 1)]);
      if (!(m > -INFINITY)) bad |= 1;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        ln_t[j] = ln_t[j] > -INFINITY ? T.over(ln_t[j] - m) : -INFINITY;
        s += expf(ln_t[j]);
      }
      const float ln_s = logf(block_add(s, tmp));
#pragma unroll
      for (int j = 0; j < kPer; ++j) ln_t[j] -= ln_s;
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      t[j] = expf(ln_t[j]);
      s += t[j];
    }
    sum = block_add(s, tmp);
    if (!(sum < INFINITY)) bad |= 1;
    rho = a.lse ? fmaxf(1.f - sum, 0.f) : 0.f;
    all = a.lse && sum > 1.f + 0x1p-20f + 0x1p-23f * fabsf(lse) ? sum : 1.f;    // not what the rounding of lse makes
  }
};

// The list of row r; -1: it does not learn, -2: outside the lists.
DF_DEV int list_of(const DistillArgs& a, int r) {
  if (a.weight && a.weight[r] == 0.f) return -1;
  const int list = a.teacher_row ? a.teacher_row[r] : r;
  return list < -1 || list >= a.n_teacher ? -2 : list;
}

// Replaces x (VE values, the student's logits with READ) by f(x) in this CTA's pieces of the
// gradient's row, U loads ahead.
template <int U, bool READ, class E, class F>
DF_DEV void write_pieces(const RowPart<E>& p, E* grad, F&& f) {
  constexpr int VE = RowPart<E>::VE;
  // the gradient's pieces start at 16-byte addresses like the student's
  const bool aligned = (reinterpret_cast<uintptr_t>(grad - p.head) & 15) == 0;
  uint4* out = reinterpret_cast<uint4*>(grad - p.head);
  float x[VE];
  auto set = [&](int piece) {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int k = p.id(piece, e);
      if ((unsigned)k < (unsigned)p.V) RowOf<E>::set(grad, k, x[e]);
    }
  };
  for (int i = p.lo + (int)threadIdx.x; i < p.hi; i += U * kRowThreads) {
    uint4 v[U];
    if (READ)
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = p.whole_or_nothing(i + j * kRowThreads);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int piece = i + j * kRowThreads;
      if (READ) RowOf<E>::unpack(v[j], x);
      f(x);
      if (piece >= p.hi) continue;
      if (aligned)
        out[piece] = RowOf<E>::pack(x);
      else
        set(piece);
    }
  }
  const int edge = p.my_edge();
  if (edge >= 0) {
    if (READ) RowOf<E>::unpack(p.edge(edge), x);
    f(x);
    set(edge);
  }
}
template <class E>
DF_DEV void write_zeros(const RowPart<E>& p, E* grad) {
  write_pieces<4, false>(p, grad, [](float* x) {
#pragma unroll
    for (int e = 0; e < RowPart<E>::VE; ++e) x[e] = 0.f;
  });
}

// The list's own gradient, over what the formula of the tokens outside has left there.  z: the student's
// logits at the thread's entries, where they lie in the part.
template <class E>
DF_DEV void write_listed(E* grad, const Entries& en, const float* z, const bool* mine, float m, float c, float scale, float inv_s) {
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (mine[j]) RowOf<E>::set(grad, en.id[j], scale * (ex2_approx((z[j] - m) * c) * inv_s * en.all - en.t[j]));
}

// grid: rows x CTAs of a row.
template <class E>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(DistillArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));   // one for each element of the part
  constexpr int VE = RowPart<E>::VE;
  pdl_wait();
  pdl_trigger();
  const int rank = ctas == 1 ? 0 : (int)cluster_rank(), tid = threadIdx.x;
  const int r = blockIdx.x / ctas;
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  E* grad = a.grad ? static_cast<E*>(a.grad) + r * a.ld_grad : nullptr;
  const int list = list_of(a, r);
  auto give = [&](float v) {
    a.loss[r] = v;
    reinterpret_cast<float4*>(a.stats)[r] = make_float4(v, v, v, v);
  };
  if (list < 0) {
    if (grad) write_zeros(part, grad);
    if (rank == 0 && tid == 0) {
      if (list == -1) {
        give(0.f);
      } else {
        set_status(a.status, DF_ERR_ARG, r);
        give(NAN);
      }
    }
    return;
  }
  const Temper T(a.temperature);
  const int n_words = ((part.end - part.begin) * VE + 31) / 32;
  for (int i = tid; i < n_words; i += kRowThreads) bits[i] = 0;
  if (tid == 0) s.flags = 0;
  if (ctas > 1) {
    cluster_arrive();
    // few rows: theirs are on the way while the list is read
    for (int i = part.lo + tid * 8; i < part.hi; i += 8 * kRowThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(part.pieces + i));
  }
  Entries en;
  en.load(a, T, list, s.tmp);       // with barriers behind the zeros
  float z[kPer];
  bool mine[kPer];
  const int bit0 = part.begin * VE - part.head;   // element of bit 0
  uint32_t bad = en.bad;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = en.id[j] - bit0;
    mine[j] = en.id[j] >= 0 && b >= 0 && b < (part.end - part.begin) * VE;
    z[j] = mine[j] ? RowOf<E>::value(part.row, en.id[j]) : -INFINITY;
    if (mine[j] && (atomicOr(&bits[b >> 5], 1u << (b & 31)) >> (b & 31) & 1)) bad |= 2;
  }
  if (bad) atomicOr(&s.flags, bad);
  __syncthreads();
  // largest logit and the sum outside the list, a thread's own.  With the lowest number to begin with, what is
  // masked adds 0 without a question; the sum is 0 where nothing is left.
  float mr = -0x1.fffffep127f, rest = 0.f, check = -INFINITY;
  const uint8_t* marks = reinterpret_cast<const uint8_t*>(bits);
  for_pieces<4>(part, [&](float* x, int piece, bool on) {
    float big = x[0];
#pragma unroll
    for (int e = 1; e < VE; ++e) big = max_nan(big, x[e]);
    check = max_nan(check, big);
    uint32_t listed = 0;
    if (on) {
      const int q = piece - part.begin;
      listed = VE == 8 ? marks[q] : (marks[q >> 1] >> ((q & 1) * 4)) & 15u;
    }
    if (listed) {          // few pieces; one way through the sums for all (960 rows of 151936: with two 141 us, not 131)
      big = -INFINITY;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (listed >> e & 1) x[e] = -INFINITY;
        big = fmaxf(big, x[e]);
      }
    }
    if (big > mr) {
      rest *= ex2_approx((mr - big) * T.c);
      mr = big;
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) rest += ex2_approx((x[e] - mr) * T.c);
  });
  if (rest == 0.f) mr = -INFINITY;
  // the CTA's part
  float zmax = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) zmax = fmaxf(zmax, z[j]);
  float big = redux_max(zmax), big_rest = redux_max(mr);
  __syncthreads();
  if ((tid & 31) == 0) {
    s.tmp[tid >> 5] = big;
    s.tmp2[tid >> 5] = big_rest;
  }
  if (!(check < INFINITY)) atomicOr(&s.flags, 1u);
  __syncthreads();
  big_rest = redux_max(s.tmp2[tid & (kRowWarps - 1)]);
  big = fmaxf(redux_max(s.tmp[tid & (kRowWarps - 1)]), big_rest);
  rest = block_add(mr > -INFINITY ? rest * ex2_approx((mr - big_rest) * T.c) : 0.f, s.tmp);
  float in = 0.f, cross = 0.f, tsum = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (mine[j]) {
      if (z[j] > -INFINITY) in += ex2_approx((z[j] - big) * T.c);
      if (en.t[j] > 0.f) {
        tsum += en.t[j];
        cross += z[j] > -INFINITY ? en.t[j] * (en.ln_t[j] - T.over(z[j] - big)) : INFINITY;
      }
    }
  in = block_add(in, s.tmp);
  cross = block_add(cross, s.tmp);
  tsum = block_add(tsum, s.tmp);
  if (ctas > 1) cluster_wait();     // every CTA of the cluster runs before its memory is written
  if (tid < ctas) {
    const float w[kPosts] = {big, big_rest, rest, in, cross, tsum, __uint_as_float(s.flags)};
    for (int i = 0; i < kPosts; ++i) st_remote(at_rank(&s.post[rank][i], tid), w[i]);
  }
  row_sync(ctas);
  float m = -INFINITY;
  mr = -INFINITY;
  bad = 0;
  for (int i = 0; i < ctas; ++i) {
    m = fmaxf(m, s.post[i][kLargest]);
    mr = fmaxf(mr, s.post[i][kLargestRest]);
    bad |= __float_as_uint(s.post[i][kFlags]);
  }
  if (!(m > -INFINITY)) bad |= 1;
  if (bad) {
    if (grad) write_zeros(part, grad);
    if (rank == 0 && tid == 0) {
      set_status(a.status, bad & 2 ? DF_ERR_ARG : DF_ERR_NAN, r);
      give(NAN);
    }
    return;
  }
  float R = 0.f, S = 0.f;              // R relative to m'
  cross = 0.f;
  for (int i = 0; i < ctas; ++i) {
    const float mi = s.post[i][kLargest], mri = s.post[i][kLargestRest];
    if (mri > -INFINITY) R += s.post[i][kRest] * ex2_approx((mri - mr) * T.c);
    cross += s.post[i][kCross];
    if (mi > -INFINITY) {
      S += s.post[i][kListed] * ex2_approx((mi - m) * T.c);
      if (s.post[i][kT] > 0.f) cross += T.over(m - mi) * s.post[i][kT];     // (m - mi) / T may be infinite
    }
  }
  const float below = T.over(mr - m);
  const bool others = below >= kMasked;     // not: there are none, or they count as masked
  if (!others) {
    R = 0.f;
    mr = m;
  }
  const float to_m = ex2_approx((mr - m) * T.c);     // e_j = exp((z_j - m') / T) times this
  S += R * to_m;
  const float rho = en.rho;
  const float weight = a.weight ? a.weight[r] : 1.f;
  if (rank == 0 && tid == 0) {
    const float ln_s = logf(S);
    float ln_r = others ? below + logf(R) : -INFINITY, left = 0.f;
    if (others && ln_r < kFar) {
      const double exact = ((double)mr - (double)m) / (double)a.temperature + (double)logf(R);
      ln_r = (float)exact;
      left = (float)(exact - (double)ln_r);
    }
    const float kl = cross + en.sum * ln_s + (rho > 0.f ? rho * (logf(rho) - (ln_r - ln_s)) : 0.f);
    a.loss[r] = weight * kl;
    reinterpret_cast<float4*>(a.stats)[r] = make_float4(m, ln_s, ln_r, left);
  }
  if (grad) {
    const float scale = T.over(weight), inv_s = 1.f / S;
    const float out = scale * (to_m * inv_s * en.all - (others ? rho / R : 0.f));
    write_pieces<4, true>(part, grad, [&](float* x) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = ex2_approx((x[e] - mr) * T.c) * out;
    });
    write_listed(grad, en, z, mine, m, T.c, scale, inv_s);
  }
}

// The gradient of the tokens outside the list where ln R, in the two floats ln_r + left, lies so far below 0
// that exponents need more digits than a float has; few rows do.
template <class E>
__device__ __noinline__ void write_far(const E* row, int V, int rank, int ctas, E* grad, float T, float m, float ln_r, float left,
                                       float out) {
  const RowPart<E> p(row, 0, 0, V, rank, ctas);
  const double c = 1.4426950408889634 / (double)T, to = ((double)ln_r + (double)left) * 1.4426950408889634;
  write_pieces<1, true>(p, grad, [&](float* x) {
#pragma unroll
    for (int e = 0; e < RowPart<E>::VE; ++e) x[e] = ex2_approx((float)(((double)x[e] - (double)m) * c - to)) * out;
  });
}

// grid: rows x CTAs of a row; they do not depend on each other.
template <class E>
__global__ void __launch_bounds__(kRowThreads) distill_backward_kernel(DistillArgs a, int ctas) {
  __shared__ float tmp[kRowWarps];
  constexpr int VE = RowPart<E>::VE;
  pdl_wait();
  pdl_trigger();
  const int rank = blockIdx.x % ctas, r = blockIdx.x / ctas;
  const RowPart<E> part(static_cast<const E*>(a.x.data), a.x.ld, r, a.x.V, rank, ctas);
  E* grad = static_cast<E*>(a.grad) + r * a.ld_grad;
  const float4 st = reinterpret_cast<const float4*>(a.stats)[r];
  const int list = list_of(a, r);
  if (list == -2 && rank == 0 && threadIdx.x == 0) set_status(a.status, DF_ERR_ARG, r);
  if (list < 0 || st.x != st.x) {
    write_zeros(part, grad);
    return;
  }
  const Temper T(a.temperature);
  Entries en;
  en.load(a, T, list, tmp);
  float z[kPer];
  bool mine[kPer];
  const int bit0 = part.begin * VE - part.head;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = en.id[j] - bit0;
    mine[j] = en.id[j] >= 0 && b >= 0 && b < (part.end - part.begin) * VE;
    z[j] = mine[j] ? RowOf<E>::value(part.row, en.id[j]) : 0.f;
  }
  __syncthreads();     // an entry's logit is read before it may be written over
  const float rho = en.rho;
  const float scale = T.over((a.weight ? a.weight[r] : 1.f) * (a.grad_loss ? a.grad_loss[r] : 1.f));
  const bool others = st.z > -INFINITY;
  // e_j / R (without others e_j), times R / S - rho (1 / S)
  const float ln_r = others ? st.z : 0.f, out = scale * (expf(ln_r - st.y) * en.all - (others ? rho : 0.f));
  const float m = st.x, to = ln_r * 1.44269504f;
  if (ln_r < kFar)
    write_far(part.row, a.x.V, rank, ctas, grad, a.temperature, m, ln_r, st.w, out);
  else
    write_pieces<4, true>(part, grad, [&](float* x) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = ex2_approx(fmaf(x[e] - m, T.c, -to)) * out;
    });
  write_listed(grad, en, z, mine, m, T.c, scale, expf(-st.y));
}

__global__ void __launch_bounds__(256) path_rows_kernel(int b, int D, int n_tree, const int32_t* __restrict__ n_new,
                                                        const int32_t* __restrict__ src_slot, int max_src,
                                                        const int32_t* __restrict__ cache_len, int32_t* __restrict__ row) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)b * D) return;
  const int s = (int)(i / D), d = (int)(i % D);
  int node = -1;
  if (d < n_new[s]) node = d == 0 ? 0 : src_slot[(size_t)s * max_src + d - 1] - (cache_len[s] - n_new[s]);
  if (node >= n_tree || node < (d > 0)) node = -1;
  row[i] = node < 0 ? -1 : s * n_tree + node;
}

int done(cudaError_t e) { return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA; }

}  // namespace

template <void (*KERNEL)(DistillArgs, int)>
static int launch_loss(const DistillArgs& a, int ctas, cudaStream_t st) {
  static std::atomic<unsigned long long> done_{0};
  // one bit for each element of a CTA's part; a part is at most 2^18 elements and a piece or two
  const size_t smem = sizeof(Shared) + ((size_t)(a.x.V + 16) / ctas + 64) / 8 + 16;
  if (prepare_kernel(reinterpret_cast<const void*>(KERNEL), sizeof(Shared) + (1 << 15) + 64, done_) != cudaSuccess)
    return DF_ERR_CUDA;
  DF_TRACE("distill", st);
  return done(launch_cluster(KERNEL, (unsigned)a.x.rows * ctas, ctas, smem, st, a, ctas));
}
// CTAs of all rows that are one wave, or hardly more.
static int one_wave() { return 2 * num_sms() + num_sms() / 8; }

int launch_distill(const DistillArgs& a, cudaStream_t st) {
  int ctas = row_ctas(a.x.rows, a.x.V, one_wave());
  // With the gradient a row is read twice, the second time from L2 if the rows under way fit there:
  // a CTA has at most about 160 KB of a row (960 rows of 151936 bf16: 2 CTAs 133 us, 1 160; 400 rows
  // of fp32: 4 CTAs 111 us, 2 135, 1 145).
  if (a.grad)
    while (ctas < 8 && (size_t)a.x.V * (a.x.dtype == DF_F32 ? 4 : 2) > ((size_t)160 << 10) * ctas) ctas *= 2;
  return a.x.dtype == DF_F32 ? launch_loss<distill_kernel<float>>(a, ctas, st) : launch_loss<distill_kernel<uint16_t>>(a, ctas, st);
}
int launch_distill_backward(const DistillArgs& a, cudaStream_t st) {
  const int ctas = row_ctas(a.x.rows, a.x.V, one_wave());
  const auto f = a.x.dtype == DF_F32 ? distill_backward_kernel<float> : distill_backward_kernel<uint16_t>;
  DF_TRACE("distill_backward", st);
  return done(launch_k(f, dim3((unsigned)a.x.rows * ctas), dim3(kRowThreads), 0, st, a, ctas));
}
int launch_path_rows(int b, int D, int n_tree, const int32_t* n_new, const int32_t* src_slot, int max_src,
                     const int32_t* cache_len, int32_t* teacher_row, cudaStream_t st) {
  DF_TRACE("path_rows", st);
  const unsigned blocks = (unsigned)(((long long)b * D + 255) / 256);
  return done(launch_k(path_rows_kernel, dim3(blocks), dim3(256), 0, st, b, D, n_tree, n_new, src_slot, max_src, cache_len,
                       teacher_row));
}

}  // namespace df
