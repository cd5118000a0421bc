// Reductions over the lanes of a wavefront in vector instructions (no LDS).
#pragma once
#include "mok_device.h"

namespace {

template <int CTRL>
MOK_DEV float dpp(float v) {
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, true));
}

// The result over each aligned group of L lanes (2 .. 64), in every lane of it:
// pairs, fours, then mirrored halves of 8 and 16 lanes, then the rows of 16 and
// halves of 32 exchanged. Every lane combines the same two values at each step,
// so all of them end with the same bits. `f` is commutative. All lanes take part.
template <int L, class F>
MOK_DEV float lanes_reduce(float v, F f) {
  static_assert(L >= 1 && L <= 64 && (L & (L - 1)) == 0, "a power of two");
  if constexpr (L >= 2) v = f(v, dpp<0xB1>(v));          // lane ^ 1
  if constexpr (L >= 4) v = f(v, dpp<0x4E>(v));          // lane ^ 2
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));         // 7 - lane of 8
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));        // 15 - lane of 16
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
// the sum of 64-bit values over each aligned group of L lanes, by the same exchanges of both their words
template <int CTRL>
MOK_DEV double dpp(double v) {
  const auto w = __builtin_bit_cast(i32x2_t, v);
  return __builtin_bit_cast(double, (i32x2_t){__builtin_amdgcn_update_dpp(w[0], w[0], CTRL, 0xF, 0xF, true),
                                              __builtin_amdgcn_update_dpp(w[1], w[1], CTRL, 0xF, 0xF, true)});
}
template <int L>
MOK_DEV double lanes_sum(double v) {
  static_assert(L >= 1 && L <= 64 && (L & (L - 1)) == 0, "a power of two");
  const auto both = [](const auto& lo, const auto& hi) {
    return __builtin_bit_cast(double, (i32x2_t){(int)lo[0], (int)hi[0]}) +
           __builtin_bit_cast(double, (i32x2_t){(int)lo[1], (int)hi[1]});
  };
  if constexpr (L >= 2) v += dpp<0xB1>(v);
  if constexpr (L >= 4) v += dpp<0x4E>(v);
  if constexpr (L >= 8) v += dpp<0x141>(v);
  if constexpr (L >= 16) v += dpp<0x140>(v);
  if constexpr (L >= 32) {
    const auto w = __builtin_bit_cast(i32x2_t, v);
    v = both(__builtin_amdgcn_permlane16_swap(w[0], w[0], false, false),
             __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false));
  }
  if constexpr (L >= 64) {
    const auto w = __builtin_bit_cast(i32x2_t, v);
    v = both(__builtin_amdgcn_permlane32_swap(w[0], w[0], false, false),
             __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false));
  }
  return v;
}
template <int L>
MOK_DEV float lanes_sum(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
MOK_DEV float lanes_max(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
