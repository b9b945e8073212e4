// Device helpers of the 4-bit KV cache: decoding and rounding of its rows, tensor-core steps
// on fp16 fragments, untiled bulk copies.
//
// A value is 2^exp * s * c: c one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign (e2m1), s an e4m3
// number shared by 16 values.  s * c has six significant bits and lies between 2^-10 and 2688
// where it is not 0, so it is an fp16 number: the tensor cores multiply the cache's values
// exactly, and 2^exp is folded into the softmax scale (keys) and the output (values).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace df {

// Four code bytes (eight values) -> four fp16x2, low half = low nibble.
DF_DEV void e2m1x8_to_f16(uint32_t x, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(x));
}
DF_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two e4m3 bytes without sign (one in each half of x, the upper byte of a half 0) -> fp16x2:
// the fields moved into fp16's place give the value times 2^-8.  No byte gives an infinity or
// a NaN (0x7F decodes as 480), so a slot that was never written stays finite.
DF_DEV uint32_t e4m3x2_to_f16(uint32_t x) { return hmul2((x & 0x007F007Fu) << 7, 0x5C005C00u); }
DF_DEV float e4m3_to_f(uint32_t byte) {
  const uint32_t h = e4m3x2_to_f16(byte & 0x7Fu);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

// D (16 x 8, fp32) += A (16 x 16, fp16) * B (16 x 8, fp16).
DF_DEV void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DF_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Contiguous copy global -> shared; addresses and size multiples of 16 bytes.
DF_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// The power of two that brings a row whose largest magnitude is `amax` to [2^12, 2^13): the
// bf16 row times it is an fp16 row, exactly, but for what lies 2^26 below the largest.
// `back` is its inverse.  Both stay normal numbers: a row below 2^-114 stays smaller, and one
// without a finite largest takes the powers of the largest numbers.
DF_DEV float f16_row_factor(float amax, float& back) {
  int e = (int)(__float_as_uint(amax) >> 23);   // biased exponent; amax >= 0
  e = min(max(e, 13), 254);
  back = __uint_as_float((uint32_t)(e - 12) << 23);
  return __uint_as_float((uint32_t)(254 - e + 12) << 23);
}

// Slots a sequence may show, or -1 (recorded) where its length does not fit the cache.
DF_DEV int kv4_len(const int32_t* cache_len, int s, int more, int cap, int* status) {
  const int n = cache_len[s];
  if (n >= 0 && n <= cap - more) return n;
  set_status(status, DF_ERR_CAPACITY, s);
  return -1;
}

}  // namespace df
