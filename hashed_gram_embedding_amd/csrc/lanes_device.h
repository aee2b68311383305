// Reductions over the lanes of a wavefront in registers, and reads of a row of
// logits in runs of four.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "engram.h"

namespace engram {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Cross-lane steps in the registers (DPP) rather than through LDS: every
// reduction of these kernels is on the chain from a row's last load to its
// result (verification of 1 x 4 drafts x 32001 7.8 -> 6.9 us).
//
// x of the lane that CTRL names, in the rows of 16 lanes that ROWS names; `old`
// elsewhere and where there is no such lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float old, float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(x), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane(double old, double x) {
  const uint64_t o = __double_as_longlong(old), b = __double_as_longlong(x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(static_cast<uint32_t>(o), static_cast<uint32_t>(b), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(static_cast<uint32_t>(o >> 32), static_cast<uint32_t>(b >> 32), CTRL, ROWS, 0xf, false);
  return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t from_lane(uint64_t old, uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(static_cast<uint32_t>(old), static_cast<uint32_t>(x), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(static_cast<uint32_t>(old >> 32), static_cast<uint32_t>(x >> 32), CTRL, ROWS, 0xf, false);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// lane - n of the row; lane - 1; the last lane of the row before; lane 31
constexpr int kRowShr = 0x110, kWaveShr1 = 0x138, kRowBcast15 = 0x142, kRowBcast31 = 0x143;

// Inclusive sum over the lanes of a wavefront.
template <typename T>
__device__ __forceinline__ T wave_scan(T x) {
  x += from_lane<kRowShr + 1, 0xf>(T(0), x);
  x += from_lane<kRowShr + 2, 0xf>(T(0), x);
  x += from_lane<kRowShr + 4, 0xf>(T(0), x);
  x += from_lane<kRowShr + 8, 0xf>(T(0), x);
  x += from_lane<kRowBcast15, 0xa>(T(0), x);
  x += from_lane<kRowBcast31, 0xc>(T(0), x);
  return x;
}

__device__ __forceinline__ float at_lane(float x, int lane) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane)); }
__device__ __forceinline__ uint64_t at_lane(uint64_t b, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane), hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ double at_lane(double x, int lane) {
  const uint64_t b = __double_as_longlong(x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane), hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
  return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

// Four logits from any element on, as stored; -inf past the row's end.
template <int DT>
struct Quad;
template <>
struct Quad<ENGRAM_F32> {
  f32x4_t x;
  __device__ __forceinline__ float at(int k) const { return x[k]; }
};
template <>
struct Quad<ENGRAM_BF16> {
  u32x2_t x;
  __device__ __forceinline__ float at(int k) const { return __uint_as_float(k & 1 ? x[k >> 1] & 0xffff0000u : x[k >> 1] << 16); }
};

// Quad i of a row of `quads` whole ones, -inf past the last (no branch around
// the load: it reads the row's first quad instead).
template <int DT>
__device__ __forceinline__ Quad<DT> load_quad(const void* row, int64_t i, int64_t quads) {
  Quad<DT> q;
  const bool in = i < quads;
  const int64_t v = in ? i * 4 : 0;
  if constexpr (DT == ENGRAM_F32) {
    if (quads > 0) __builtin_memcpy(&q.x, static_cast<const float*>(row) + v, 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) q.x[k] = in ? q.x[k] : -__builtin_inff();
  } else {
    if (quads > 0) __builtin_memcpy(&q.x, static_cast<const uint16_t*>(row) + v, 8);
    q.x = in ? q.x : u32x2_t{0xff80ff80u, 0xff80ff80u};
  }
  return q;
}

// The up to three entries behind the last quad are the first threads' own.
template <int DT>
__device__ __forceinline__ float load_tail(const void* row, int64_t v, int64_t V) {
  if (v >= V) return -__builtin_inff();
  if constexpr (DT == ENGRAM_F32) return static_cast<const float*>(row)[v];
  else return bf16_to_f32(static_cast<const uint16_t*>(row)[v]);
}

__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, from_lane<kRowShr + 1, 0xf>(x, x));
  x = fmaxf(x, from_lane<kRowShr + 2, 0xf>(x, x));
  x = fmaxf(x, from_lane<kRowShr + 4, 0xf>(x, x));
  x = fmaxf(x, from_lane<kRowShr + 8, 0xf>(x, x));
  x = fmaxf(x, from_lane<kRowBcast15, 0xa>(x, x));
  x = fmaxf(x, from_lane<kRowBcast31, 0xc>(x, x));
  return at_lane(x, 63);
}

// Largest value over the workgroup, NaN if any thread saw one.
template <int THREADS>
__device__ __forceinline__ float group_max(float x, bool nan, float* red) {
  x = wave_max(x);
  if (__any(nan)) x = __builtin_nanf("");
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) m = m != m || red[w] != red[w] ? __builtin_nanf("") : fmaxf(m, red[w]);
  return m;
}

// Orders a wavefront's LDS accesses before this point and behind it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// bf16 pairs stay packed from pass to pass: without this the compiler keeps
// every unpacked value, then every exponential, for the next pass, twice the
// registers there are.  (float32 rows keep their exponentials in place.)
template <int DT, int N>
__device__ __forceinline__ void forget(Quad<DT> (&x)[N]) {
  if constexpr (DT == ENGRAM_BF16)
#pragma unroll
    for (int n = 0; n < N; ++n) asm volatile("" : "+v"(x[n].x));
}

}  // namespace engram
