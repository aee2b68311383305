// Rows as 8-bit integers with one scale (engram_quantize_i8), on the device:
//
//   s = max_c |x_c| / 127,  q_c = rne(127 x_c / max_c |x_c|)
//
// shared by the quantisation, the product that quantises a few rows itself and
// the gather that writes a layer's rows as codes.
#pragma once

#include <type_traits>

#include "device_util.h"

namespace engram {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// What quantising a row needs: its largest magnitude, and 127 over it.  Both
// and the values are scaled by g, a power of two that keeps 127 / top finite
// for rows of the smallest numbers (exact: nothing is rounded by it).
struct RowScale {
  float top, inv, g;
};

__device__ __forceinline__ RowScale row_factors(float top) {
  const float g = top < 0x1p-60f ? 0x1p80f : 1.0f;
  return RowScale{top * g, 127.0f / (top * g), g};
}

// rne(127 x / top) of exact arithmetic, for |x| <= top.  In float y = x *
// (127 / top) is off by less than 2^-15.  Only within 2^-13 of the middle m
// of two whole numbers could that change the rounding; there 127 x is
// compared with m top, both exact in double (31 and 32 bits).
__device__ __forceinline__ int quantize(float x, const RowScale& r) {
  const float v = x * r.g, y = v * r.inv, n = floorf(y);
  float q = rintf(y);
  if (fabsf(y - n - 0.5f) < 0x1p-13f) {
    const double d = 127.0 * static_cast<double>(v) - (static_cast<double>(n) + 0.5) * static_cast<double>(r.top);
    const float even = 2.0f * rintf(0.5f * (n + 0.5f));   // n or n + 1
    q = d > 0.0 ? n + 1.0f : (d < 0.0 ? n : even);
  }
  return static_cast<int>(q);
}

// Largest magnitude of values held by a group of wavefronts, by its bits: an
// infinity and a NaN order above every finite value.
__device__ __forceinline__ uint32_t wave_top(uint32_t top) {
  // in the registers (DPP): over each row of 16 lanes, then into the rows behind
  auto join = [&](auto ctrl, auto rows) {
    top = max(top, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(top), static_cast<int>(top), decltype(ctrl)::value,
                                                                     decltype(rows)::value, 0xf, false)));
  };
  constexpr int kRowShr = 0x110, kRowBcast15 = 0x142, kRowBcast31 = 0x143;
  join(std::integral_constant<int, kRowShr + 1>{}, std::integral_constant<int, 0xf>{});
  join(std::integral_constant<int, kRowShr + 2>{}, std::integral_constant<int, 0xf>{});
  join(std::integral_constant<int, kRowShr + 4>{}, std::integral_constant<int, 0xf>{});
  join(std::integral_constant<int, kRowShr + 8>{}, std::integral_constant<int, 0xf>{});
  join(std::integral_constant<int, kRowBcast15>{}, std::integral_constant<int, 0xa>{});
  join(std::integral_constant<int, kRowBcast31>{}, std::integral_constant<int, 0xc>{});
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(top), 63));
}

__device__ __forceinline__ float row_scale(uint32_t top) {
  return top < 0x7f800000u ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
}

// Codes of a row whose largest magnitude is `top` (its bits): none where the
// row is zero or holds an infinity or a NaN.
__device__ __forceinline__ bool row_has_codes(uint32_t top) { return top != 0u && top < 0x7f800000u; }

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ u32x2_t quantize8(const float* f, const RowScale& r) {
  u32x2_t w{0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k >> 2] |= (static_cast<uint32_t>(quantize(f[k], r)) & 0xffu) << (8 * (k & 3));
  return w;
}

}  // namespace engram
