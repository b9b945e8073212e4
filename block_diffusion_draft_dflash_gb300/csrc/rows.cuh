// Rows of logits on the device: how a cluster of CTAs reads one, sums and barriers over the
// cluster, and probabilities that are exact enough to decide which token a border falls on.
//
// A row is read in aligned pieces of 16 bytes, whatever its first address: piece i holds the
// row's elements i * VE - head .. (VE = 4 fp32 or 8 bf16 values, head = elements between the
// aligned address below the row and the row).  The CTAs of a cluster take consecutive runs of the
// pieces that lie in the row whole.  The first and the last piece may reach over the row's ends
// (edges, of the first and the last CTA); they are read element by element, and what lies outside
// counts as -inf.
#pragma once
#include "common.cuh"
#include "rows.h"

namespace df {
namespace {   // each file has its own number of threads

#ifndef DF_ROW_THREADS
#define DF_ROW_THREADS 256
#endif
constexpr int kRowThreads = DF_ROW_THREADS;   // of a CTA
constexpr int kRowWarps = kRowThreads / 32;
constexpr uint32_t kNegInfKey = 0x007FFFFFu;   // float_key(-inf)
constexpr uint32_t kPosInfKey = 0xFF800000u;   // float_key(+inf); a NaN's key is above it

// ------------------------------------------------------------------------------ cluster
DF_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
DF_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
DF_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Barrier over the CTAs of a row, with their shared memory.
DF_DEV void row_sync(int ctas) {
  if (ctas == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}
// Address of this shared-memory object in CTA `rank` of the cluster.
DF_DEV uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
DF_DEV void st_remote(uint32_t a, uint32_t v) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
DF_DEV void st_remote(uint32_t a, float v) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
DF_DEV void st_remote(uint32_t a, uint64_t v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }
DF_DEV uint32_t ld_remote(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
DF_DEV uint32_t add_remote(uint32_t a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
  return old;
}
DF_DEV void add_remote(uint32_t a, uint64_t v) { asm volatile("red.shared::cluster.add.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }
DF_DEV void max_remote(uint32_t a, uint32_t v) { asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
DF_DEV void min_remote(uint32_t a, uint32_t v) { asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, int ctas, size_t smem, cudaStream_t st,
                                  Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ------------------------------------------------------------------------------ block sums
template <class V>
DF_DEV V warp_add(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the block, the same in every thread and in a fixed order; `tmp` holds kRowWarps
// entries and may be used again by the next call.
template <class V>
DF_DEV V block_add(V v, V* tmp) {
  v = warp_add(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  V s = tmp[threadIdx.x & (kRowWarps - 1)];
#pragma unroll
  for (int o = kRowWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// Sum over the threads before this one; *total: over all.
template <class V>
DF_DEV V block_scan(V v, V* tmp, V* total) {
  const int lane = threadIdx.x & 31;
  V incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) tmp[threadIdx.x >> 5] = incl;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    const V x = tmp[w];
    if (w < (int)(threadIdx.x >> 5)) before += x;
    all += x;
  }
  *total = all;
  return before + incl - v;
}

// ------------------------------------------------------------------------------ reading
DF_DEV float max_nan(float a, float b) {   // a NaN stays one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
DF_DEV uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <class E>
struct RowOf;
template <>
struct RowOf<float> {
  static constexpr int VE = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static DF_DEV void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static DF_DEV uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static DF_DEV float value(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
  static DF_DEV void set(void* p, long long i, float x) { static_cast<float*>(p)[i] = x; }
  static DF_DEV float largest(const uint4& v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
};
template <>
struct RowOf<uint16_t> {   // bf16
  static constexpr int VE = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static DF_DEV void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static DF_DEV uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
  static DF_DEV float value(const void* p, long long i) { return bf16_to_f(static_cast<const uint16_t*>(p)[i]); }
  static DF_DEV void set(void* p, long long i, float x) { static_cast<uint16_t*>(p)[i] = f_to_bf16(x); }
  static DF_DEV float largest(const uint4& v) {
    const uint32_t m = max_nan2(max_nan2(v.x, v.y), max_nan2(v.z, v.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
};

// One CTA's part of a row.
template <class E>
struct RowPart {
  static constexpr int VE = RowOf<E>::VE;
  const E* row;          // element 0
  const uint4* pieces;   // piece 0 (its first `head` elements lie before the row)
  int head, V;
  int lo, hi;            // whole pieces
  int begin, end;        // with the edges

  DF_DEV RowPart(const E* data, long long ld, long long r, int V_, int rank, int ctas) : V(V_) {
    row = data + r * ld;
    head = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E));
    pieces = reinterpret_cast<const uint4*>(row - head);
    const int first = head > 0, upto = max((V + head) / VE, first);      // whole pieces of the row
    const int each = (upto - first + ctas - 1) / ctas;
    lo = min(first + rank * each, upto);
    hi = min(lo + each, upto);
    begin = rank == 0 ? 0 : lo;
    end = rank == ctas - 1 ? (V + head + VE - 1) / VE : hi;
  }
  DF_DEV int id(int piece, int e) const { return piece * VE + e - head; }
  // Elements of an edge; -inf outside the row.
  DF_DEV uint4 edge(int piece) const {
    float x[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int i = id(piece, e);
      x[e] = (unsigned)i < (unsigned)V ? RowOf<E>::value(row, i) : -INFINITY;
    }
    return RowOf<E>::pack(x);
  }
  DF_DEV uint4 load(int piece) const { return piece >= lo && piece < hi ? pieces[piece] : edge(piece); }
  DF_DEV uint4 whole_or_nothing(int piece) const {
    const uint32_t m = RowOf<E>::kNegInf;
    uint4 v = make_uint4(m, m, m, m);
    if (piece < hi) v = pieces[piece];
    return v;
  }
  // The edge that this thread reads (thread 0 the first, thread 1 the last), or -1.
  DF_DEV int my_edge() const {
    if (threadIdx.x == 0 && begin < lo) return begin;
    if (threadIdx.x == 1 && end > hi) return end - 1;
    return -1;
  }
};

// f(x[VE], piece, on) for every piece of this thread (whole ones lo + t, lo + t + kRowThreads, ...,
// U loads ahead, and its edge).  on: there is such a piece; else x is -inf.
template <int U, class E, class F>
DF_DEV void for_pieces(const RowPart<E>& p, F&& f) {
  float x[RowPart<E>::VE];
  for (int i = p.lo + (int)threadIdx.x; i < p.hi; i += U * kRowThreads) {
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = p.whole_or_nothing(i + j * kRowThreads);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      RowOf<E>::unpack(v[j], x);
      f(x, i + j * kRowThreads, i + j * kRowThreads < p.hi);
    }
  }
  const int edge = p.my_edge();
  if (edge >= 0) {
    RowOf<E>::unpack(p.edge(edge), x);
    f(x, edge, true);
  }
}

// ------------------------------------------------------------------------------ masses
// Which token a border falls on is decided by comparing sums of up to 2^20 probabilities, so a
// probability is made with an error of 2^-35 and sums are exact: a mass is a whole number of
// units of 2^-42 of (about) the largest token's, and the order of a sum does not matter.
//
// 2^y by a table (the method of P. T. P. Tang, "Table-driven implementation of the exponential
// function in IEEE floating-point arithmetic", 1989): y = k / 1024 + r, 2^y = 2^(k / 1024) 2^r.
// y = l c - ref, c = log2(e) / T in two floats; ref is a multiple of 1/1024 (near the largest
// logit's l c), so adding 12288 - ref in one fma rounds y to a multiple of 1/1024, and
// r = l c - (that + ref) comes out of another fma with one rounding of a number below 2^-11.
// Where |l c| reaches 2048 the logits are taken relative to the largest one first, which is exact
// for every logit whose probability is not 0 (they lie within a factor of two of it).
struct Pow2Table {
  float hi[1024], lo[1024];   // 2^(j / 1024) = hi + lo
  constexpr Pow2Table() : hi(), lo() {
    for (int j = 0; j < 1024; ++j) {
      const double x = j / 1024.0 * 0.693147180559945309417232121458;
      double term = 1.0, sum = 1.0;
      for (int n = 1; n < 22; ++n) {
        term *= x / n;
        sum += term;
      }
      hi[j] = (float)sum;
      lo[j] = (float)(sum - (double)(float)sum);
    }
  }
};

constexpr float kMassUnit = 0x1p-42f;

struct MassScale {
  float c_hi, c_lo;    // log2(e) / T
  float base;          // subtracted from a logit first (0, or the largest logit)
  float shift;         // 12288 - ref
  float floor;         // smallest l - base that counts; below it the mass is 0 in any case
  uint32_t top;        // bits of the largest logit's t (see bits())

  // T in [2^-126, 2^100], largest finite.
  DF_DEV void set(float T, float largest) {
    const float l2e = 1.44269502162933349609375f, l2e_lo = 1.92596299112661746887e-8f;
    c_hi = l2e / T;
    c_lo = (fmaf(-c_hi, T, l2e) + l2e_lo) / T;
    const float a = largest * c_hi;
    float ref = 0.f;
    base = largest;
    if (fabsf(a) < 2048.f) {
      base = 0.f;
      ref = rintf(a * 1024.f) * (1.f / 1024.f);
    }
    shift = 12288.f - ref;
    floor = (ref - 63.75f) / c_hi;     // 2^-63.75 counts as 0; bins of 1/64, where they are not cut off, end at 4080
    top = bits(largest);
  }
  DF_DEV float arg(float l) const { return fmaxf(l - base, floor); }
  // y rounded to a multiple of 1/1024, plus 12288, as the bits of a float (units of 1/1024).
  DF_DEV uint32_t bits(float l) const { return __float_as_uint(fmaf(arg(l), c_hi, shift)); }
};

// A thread's share of a mass: two 32-bit sums of the bits of a + 12 (units of 2^-20) and of
// what is left + 1.5 * 2^-19 (units of 2^-42), exact for n <= 512 terms.
struct MassSum {
  uint32_t a = 0, b = 0;
  int n = 0;           // terms in a and b (kept by the caller)
  uint64_t sum = 0;
  DF_DEV void fold() {
    sum += ((int64_t)(int32_t)(a - (uint32_t)n * 0x41400000u) << 22) + (int32_t)(b - (uint32_t)n * 0x36400000u);
    a = b = 0;
    n = 0;
  }
  DF_DEV void room(int more) {
    if (n + more > 512) fold();
  }
};

// The mass of logit l as the terms of a and b; returns c.bits(l).  table[j]: 2^(j / 1024).
template <class Table>
DF_DEV uint32_t mass_terms(const MassScale& c, const Table& table, float l, uint32_t* a, uint32_t* b) {
  const float x = c.arg(l);
  const float t = fmaf(x, c.c_hi, c.shift);
  const float g = t - c.shift;                        // exact
  float r = fmaf(x, c.c_hi, -g);
  r = fmaf(x, c.c_lo, r);
  const uint32_t u = __float_as_uint(t);
  const float2 w = table[u & 1023u];
  const float two_n = __uint_as_float(0x3F800000u + ((u & 0xFFFFFC00u) << 13));
  // 2^r - 1 for |r| <= 2^-11 + 2^-24: the next term is below 2^-50
  const float p = r * fmaf(r, fmaf(r, 0.0555041086648f, 0.2402265069591f), 0.6931471805599f);
  const float hi = w.x * two_n, q = fmaf(hi, p, w.y * two_n);
  const float f1 = (hi + q) + 12.f, f2 = f1 - 12.f;
  const float f3 = ((hi - f2) + q) + 2.86102294921875e-6f;   // 1.5 * 2^-19
  *a = __float_as_uint(f1);
  *b = __float_as_uint(f3);
  return u;
}
// Adds it (the caller counts the term).
template <class Table>
DF_DEV uint32_t add_mass(MassSum& s, const MassScale& c, const Table& table, float l) {
  uint32_t a, b;
  const uint32_t u = mass_terms(c, table, l, &a, &b);
  s.a += a;
  s.b += b;
  return u;
}

}  // namespace
}  // namespace df
