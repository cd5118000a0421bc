// fp32 operands of the bf16 matrix instructions.
#pragma once
#include "mok_device.h"

// Split of fp32 values into three bf16 parts: w = hi + mid + lo, each part the
// truncation of what remains (8 significant bits each, 24 in all), so a product
// of two parts is exact in fp32. Exact from 2^-110 to the largest finite value
// (below, bits under bf16's smallest step, 2^-133, are lost; rounded to the
// nearest instead, what lies above bf16's largest value would become infinite).
// Pairs are packed two bf16 per dword (element 2i in the low half).
MOK_DEV void split3(float w0, float w1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t u0 = __float_as_uint(w0), u1 = __float_as_uint(w1);
  const float r0 = w0 - __uint_as_float(u0 & 0xFFFF0000u), r1 = w1 - __uint_as_float(u1 & 0xFFFF0000u);
  const uint32_t v0 = __float_as_uint(r0), v1 = __float_as_uint(r1);
  const float q0 = r0 - __uint_as_float(v0 & 0xFFFF0000u), q1 = r1 - __uint_as_float(v1 & 0xFFFF0000u);
  hi = (u0 >> 16) | (u1 & 0xFFFF0000u);
  mid = (v0 >> 16) | (v1 & 0xFFFF0000u);
  lo = (__float_as_uint(q0) >> 16) | (__float_as_uint(q1) & 0xFFFF0000u);
}
