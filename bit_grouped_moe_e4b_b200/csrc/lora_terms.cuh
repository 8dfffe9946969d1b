// fp32 factors of the adapters' products as bf16 terms for the tensor cores.
#pragma once

#include "common.cuh"

namespace e4b {

// (a, b) less (x, y), their leading bits (exact), and 2^-28 of these more.
E4B_DEV void less(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 v, t, c;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\t"
      "fma.rn.f32x2 v, t, c, v;\n\tmov.b64 c, {%5, %5};\n\tfma.rn.f32x2 v, t, c, v;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(-1.f), "f"(0x1p-28f));
}

// The pair (a, b) as three bf16 pairs hi + mid + lo, each the eight leading bits
// of what the terms before it leave and 2^-28 of the term before it. So all terms
// of a value have its sign, and none is zero where the value is not (above 2^-70
// in magnitude): a product with an infinity is one, and not 0 inf or inf - inf.
// The sum is the value up to 2^-27 of it. The terms of an infinity or a NaN are
// the value itself.
E4B_DEV void split_pair(float a, float b, uint32_t (&t)[3]) {
  const bool fa = fabsf(a) < INFINITY, fb = fabsf(b) < INFINITY;
  float ra = a, rb = b;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    t[k] = prmt(__float_as_uint(ra), __float_as_uint(rb), 0x7632);
    if (k == 2) break;
    less(ra, rb, __uint_as_float(__float_as_uint(ra) & 0xFFFF0000u), __uint_as_float(__float_as_uint(rb) & 0xFFFF0000u));
    ra = fa ? ra : a;
    rb = fb ? rb : b;
  }
}

}  // namespace e4b
