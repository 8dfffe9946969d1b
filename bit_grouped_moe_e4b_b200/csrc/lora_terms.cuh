// fp32 factors of the adapters' products as bf16 terms for the tensor cores.
#pragma once

#include "common.cuh"

namespace e4b {

// (a, b) -= the bf16 pair h.
E4B_DEV void less(float& a, float& b, uint32_t h) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"((h << 16) ^ 0x80000000u), "r"((h & 0xFFFF0000u) ^ 0x80000000u));
}

// The pair (a, b) as three bf16 pairs hi + mid + lo, 24 bits of mantissa;
// infinities and NaN have only the first.
E4B_DEV void split_pair(float a, float b, uint32_t (&t)[3]) {
  const uint32_t h = t[0] = pack_bf16x2(a, b);
  less(a, b, h);
  if ((h & 0x7F80u) == 0x7F80u) a = 0.f;
  if ((h & 0x7F800000u) == 0x7F800000u) b = 0.f;
  t[1] = pack_bf16x2(a, b);
  less(a, b, t[1]);
  t[2] = pack_bf16x2(a, b);
}

}  // namespace e4b
