// fp32 products on the tensor cores: every operand the sum of two tf32 values,
// x = hi + lo (11 significant bits each, rounded to nearest, so
// |x - hi - lo| <= 2^-23 |x|); a product is hi hi + hi lo + lo hi, and the term left
// out is below 2^-22 of it.
#pragma once

#include <stdint.h>

namespace cpa {

__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma_tf32_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// x as hi + lo, each rounded to tf32 (nearest, ties away; the tensor core
// ignores the low 13 bits) by adding half a step to the bits.  In a NaN with all
// its high bits set, the one that fp32 arithmetic here gives among them, that
// addition would run over into the sign and leave a zero.  So what is not
// finite, for which x - hi is NaN, keeps its NaN in lo: whatever it is
// multiplied by is NaN.  (Test and selection cost up to 1 %, both roundings by
// cvt.rna.tf32, which keeps NaN, 8 to 9 %: 4 tokens and a 1000-token chunk, 8 kv heads
// of 128, window 1024 / 4096, 430 / 1501 us now.)
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  const float rest = x - __uint_as_float(hi);
  lo = rest == rest ? __float_as_uint(rest) + 0x1000u : 0x7fffffffu;
}

}  // namespace cpa
