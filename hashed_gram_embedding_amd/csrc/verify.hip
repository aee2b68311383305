// Token probabilities and the verification of drafted tokens: the end of a
// speculative decode step whose layers ran over the drafted chunk.
#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "engram_internal.h"
#include "lanes_device.h"

namespace engram {
namespace {

constexpr float kLog2e = 1.44269504088896341f;

// ---- probabilities ----
// p_v = e^((l_v - max) / T) / sum; at T <= 0 the lowest index of the largest
// logit has probability 1.  A row of -inf alone has probabilities 0; one with
// a NaN has NaN throughout, and so has one with +inf at T > 0.
//
// Bound by memory: a row is read once and written once, by one workgroup that
// keeps it in registers between its maximum, its sum and its output (N runs
// of 4 values a thread, all loads in flight together).  The longest bf16 rows
// (N = 32) need more registers than the 128 a thread has: 84 bytes a lane are
// spilled, 16% more bytes written (2048 x 128000: 340 us, 327 by the bytes of
// the row and its outputs alone).
//
// The exponent (l - max) log2(e) / T has four roundings (the difference, the
// constant, the division and the product; the formula itself two) and exp2 is the
// hardware's, one unit off at most: a single probability of exponent x (in powers
// of two) is within (4 ln 2 |x| + 4) 2^-24 of its value, beside the sum's error.

struct ProbsArgs {
  const void* logits;
  const float* temperature;
  float* probs;
  int64_t V;
  int64_t ld;
  int64_t per;
};

__device__ __forceinline__ void store_quad(float* row, int64_t i, int64_t quads, f32x4_t y) {
  if (i < quads) __builtin_memcpy(row + i * 4, &y, 16);
}

template <int THREADS>
__device__ __forceinline__ float group_sum(float x, float* red) {
  x = at_lane(wave_scan(x), 63);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) s += red[w];
  return s;
}

template <int THREADS>
__device__ __forceinline__ int group_min(int x, int* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = min(x, __shfl_xor(x, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  int m = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) m = min(m, red[w]);
  return m;
}

template <int THREADS>
struct ProbsShared {
  float top[THREADS / 64], sum[THREADS / 64];
  int first[THREADS / 64];
};

// What a row without a sum holds throughout, or nothing of the kind.
__device__ __forceinline__ bool constant_row(float top, float temp, float* fill) {
  *fill = top == -__builtin_inff() ? 0.f : __builtin_nanf("");
  return top != top || top == -__builtin_inff() || (top == __builtin_inff() && temp > 0.f);
}

// 2^((l - top) log2(e) / T) of the logits l <= top of a row.  The factor is kept
// finite and above 0: the largest logit's exponent is then 0 and a masked one's
// -inf at the smallest and largest T too.  Finite logits may lie further apart
// than float32 reaches, which matters where T is large enough to bring them
// together again: there the difference is formed of l / 16 and top / 16 (16
// also keeps the factor a normal number up to the largest finite T).  At scale 1
// the multiply-add is the difference itself.
struct Exponent {
  float scale, top, f;
  __device__ __forceinline__ Exponent(float row_top, float temp) {
    scale = temp > 0x1p64f ? 0x1p-4f : 1.0f;
    top = row_top * scale;
    f = fminf(fmaxf(kLog2e / (temp * scale), 0x1p-149f), 0x1.fffffep127f);
  }
  __device__ __forceinline__ float operator()(float l) const { return __builtin_amdgcn_exp2f(fmaf(l, scale, -top) * f); }
};

template <int DT, int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
probs_kernel(ProbsArgs a) {
  __shared__ ProbsShared<THREADS> sh;
  const int64_t row = blockIdx.x, V = a.V;
  constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
  const void* in = static_cast<const char*>(a.logits) + row * a.ld * size;
  float* out = a.probs + row * V;
  const float temp = a.temperature != nullptr ? a.temperature[row / a.per] : 1.0f;
  const int64_t quads = V / 4, vt = quads * 4 + threadIdx.x;   // vt: this thread's entry behind the quads
  const int q0 = threadIdx.x;
  Quad<DT> x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = load_quad<DT>(in, q0 + n * THREADS, quads);
  const float xt = load_tail<DT>(in, vt, V);
  float top = xt;
  bool nan = xt != xt;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float l = x[n].at(k);
      nan |= l != l;
      top = fmaxf(top, l);
    }
  forget(x);
  top = group_max<THREADS>(top, nan, sh.top);
  float fill;
  if (constant_row(top, temp, &fill)) {
    for (int n = 0; n < N; ++n) store_quad(out, q0 + n * THREADS, quads, f32x4_t{fill, fill, fill, fill});
    if (vt < V) out[vt] = fill;
    return;
  }
  if (!(temp > 0.f)) {
    int at = xt == top ? static_cast<int>(vt) : INT32_MAX;
#pragma unroll
    for (int n = N - 1; n >= 0; --n)
#pragma unroll
      for (int k = 3; k >= 0; --k) at = x[n].at(k) == top ? (q0 + n * THREADS) * 4 + k : at;
    at = group_min<THREADS>(at, sh.first);
    for (int n = 0; n < N; ++n) {
      const int d = at - (q0 + n * THREADS) * 4;
      store_quad(out, q0 + n * THREADS, quads, f32x4_t{d == 0 ? 1.f : 0.f, d == 1 ? 1.f : 0.f, d == 2 ? 1.f : 0.f, d == 3 ? 1.f : 0.f});
    }
    if (vt < V) out[vt] = at == vt ? 1.f : 0.f;
    return;
  }
  const Exponent of(top, temp);
  const float et = of(xt);
  float sum = et;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = of(x[n].at(k));
    sum += (e[0] + e[1]) + (e[2] + e[3]);
  }
  forget(x);
  const float inv = 1.0f / group_sum<THREADS>(sum, sh.sum);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    f32x4_t y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = of(x[n].at(k)) * inv;
    store_quad(out, q0 + n * THREADS, quads, y);
  }
  if (vt < V) out[vt] = et * inv;
}

// Rows too long for the registers: one pass for the maximum and the sum (each
// thread's sum is kept relative to its own maximum so far), a second one for
// the output, whose reads mostly meet the caches (2048 x 128000 float32 492 us,
// 436 by the bytes of one read and one write; 2048 x 151936 bf16 413, 388).
template <int DT>
__global__ void __launch_bounds__(1024)
probs_long_kernel(ProbsArgs a) {
  constexpr int THREADS = 1024, U = 8;
  __shared__ ProbsShared<THREADS> sh;
  const int64_t row = blockIdx.x, V = a.V;
  constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
  const void* in = static_cast<const char*>(a.logits) + row * a.ld * size;
  float* out = a.probs + row * V;
  const float temp = a.temperature != nullptr ? a.temperature[row / a.per] : 1.0f;
  const int64_t quads = V / 4, vt = quads * 4 + threadIdx.x;
  const float xt = load_tail<DT>(in, vt, V);
  float top = -__builtin_inff(), sum = 0.f;
  int at = INT32_MAX;
  bool nan = xt != xt;
  for (int64_t q = threadIdx.x; q < quads; q += U * THREADS) {
    Quad<DT> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = load_quad<DT>(in, q + i * THREADS, quads);
    float m = top;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float l = x[i].at(k);
        nan |= l != l;
        if (l > m) at = (static_cast<int32_t>(q) + i * THREADS) * 4 + k;
        m = fmaxf(m, l);
      }
    if (m > -__builtin_inff() && m < __builtin_inff()) {
      const Exponent of(m, temp);
      sum = top > -__builtin_inff() ? sum * of(top) : 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = of(x[i].at(k));
        sum += (e[0] + e[1]) + (e[2] + e[3]);
      }
    }
    top = m;
  }
  const float own = top;
  top = group_max<THREADS>(fmaxf(top, xt), nan, sh.top);
  float fill;
  if (constant_row(top, temp, &fill)) {
    for (int64_t q = threadIdx.x; q < quads; q += THREADS) store_quad(out, q, quads, f32x4_t{fill, fill, fill, fill});
    if (vt < V) out[vt] = fill;
    return;
  }
  if (!(temp > 0.f)) {
    at = group_min<THREADS>(own == top ? at : (xt == top ? static_cast<int32_t>(vt) : INT32_MAX), sh.first);
    for (int64_t q = threadIdx.x; q < quads; q += THREADS) {
      const int64_t d = at - q * 4;
      store_quad(out, q, quads, f32x4_t{d == 0 ? 1.f : 0.f, d == 1 ? 1.f : 0.f, d == 2 ? 1.f : 0.f, d == 3 ? 1.f : 0.f});
    }
    if (vt < V) out[vt] = at == vt ? 1.f : 0.f;
    return;
  }
  const Exponent of(top, temp);
  const float et = of(xt);
  const float part = own > -__builtin_inff() ? sum * of(own) : 0.f;
  const float inv = 1.0f / group_sum<THREADS>(part + et, sh.sum);
  for (int64_t q = threadIdx.x; q < quads; q += U * THREADS) {
    Quad<DT> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = load_quad<DT>(in, q + i * THREADS, quads);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      f32x4_t y;
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = of(x[i].at(k)) * inv;
      store_quad(out, q + i * THREADS, quads, y);
    }
  }
  if (vt < V) out[vt] = et * inv;
}

// Few rows, long ones: kSegment entries a workgroup.  A first launch leaves
// each segment's maximum, its first place and the sum relative to it; a
// second one joins them for its row and writes its segment (read again, from
// the L2).
constexpr int kSegThreads = 256, kSegQuads = 8, kSegment = kSegThreads * kSegQuads * 4;

struct Segment {
  float top, sum;   // NaN where the segment holds one
  int32_t at;
  int32_t pad;
};

template <int DT>
struct SegmentRow {
  const void* in;
  int64_t q0, quads, vt;   // first quad of this thread, whole quads of the row, its entry behind them (last segment)
  __device__ __forceinline__ SegmentRow(const ProbsArgs& a, int64_t row, int seg, int segs) {
    constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
    in = static_cast<const char*>(a.logits) + row * a.ld * size;
    quads = a.V / 4;
    q0 = static_cast<int64_t>(seg) * (kSegment / 4) + threadIdx.x;
    vt = seg == segs - 1 ? quads * 4 + threadIdx.x : a.V;
  }
};

template <int DT>
__global__ void __launch_bounds__(kSegThreads)
probs_segments_kernel(ProbsArgs a, int segs, Segment* __restrict__ part) {
  __shared__ ProbsShared<kSegThreads> sh;
  const int64_t row = blockIdx.x / segs;
  const int seg = static_cast<int>(blockIdx.x % segs);
  const SegmentRow<DT> r(a, row, seg, segs);
  Quad<DT> x[kSegQuads];
#pragma unroll
  for (int n = 0; n < kSegQuads; ++n) x[n] = load_quad<DT>(r.in, r.q0 + n * kSegThreads, r.quads);
  const float temp = a.temperature != nullptr ? a.temperature[row / a.per] : 1.0f;
  const float xt = load_tail<DT>(r.in, r.vt, a.V);
  float top = xt;
  bool nan = xt != xt;
#pragma unroll
  for (int n = 0; n < kSegQuads; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float l = x[n].at(k);
      nan |= l != l;
      top = fmaxf(top, l);
    }
  top = group_max<kSegThreads>(top, nan, sh.top);
  int at = xt == top ? static_cast<int>(r.vt) : INT32_MAX;
#pragma unroll
  for (int n = kSegQuads - 1; n >= 0; --n)
#pragma unroll
    for (int k = 3; k >= 0; --k) at = x[n].at(k) == top ? (static_cast<int>(r.q0) + n * kSegThreads) * 4 + k : at;
  at = group_min<kSegThreads>(at, sh.first);
  float sum = 0.f;
  if (top > -__builtin_inff() && top < __builtin_inff()) {
    const Exponent of(top, temp);
    sum = of(xt);
#pragma unroll
    for (int n = 0; n < kSegQuads; ++n) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = of(x[n].at(k));
      sum += (e[0] + e[1]) + (e[2] + e[3]);
    }
  }
  sum = group_sum<kSegThreads>(sum, sh.sum);
  if (threadIdx.x == 0) part[blockIdx.x] = Segment{top, sum, at, 0};
}

template <int DT>
__global__ void __launch_bounds__(kSegThreads)
probs_join_kernel(ProbsArgs a, int segs, const Segment* __restrict__ part) {
  __shared__ ProbsShared<kSegThreads> sh;
  const int64_t row = blockIdx.x / segs;
  const int seg = static_cast<int>(blockIdx.x % segs);
  const SegmentRow<DT> r(a, row, seg, segs);
  float* out = a.probs + row * a.V;
  Quad<DT> x[kSegQuads];
#pragma unroll
  for (int n = 0; n < kSegQuads; ++n) x[n] = load_quad<DT>(r.in, r.q0 + n * kSegThreads, r.quads);
  const float temp = a.temperature != nullptr ? a.temperature[row / a.per] : 1.0f;
  const float xt = load_tail<DT>(r.in, r.vt, a.V);
  const Segment* mine = part + row * segs;
  float top = -__builtin_inff();
  bool nan = false;
  for (int i = threadIdx.x; i < segs; i += kSegThreads) {
    const float t = mine[i].top;
    nan |= t != t;
    top = fmaxf(top, t);
  }
  top = group_max<kSegThreads>(top, nan, sh.top);
  float fill;
  const bool constant = constant_row(top, temp, &fill);
  if (constant || !(temp > 0.f)) {
    int at = INT32_MAX;
    for (int i = threadIdx.x; i < segs; i += kSegThreads) at = mine[i].top == top ? min(at, mine[i].at) : at;
    at = group_min<kSegThreads>(at, sh.first);
    auto value = [&](int64_t v) { return constant ? fill : (v == at ? 1.f : 0.f); };
    for (int n = 0; n < kSegQuads; ++n) {
      const int64_t q = r.q0 + n * kSegThreads;
      store_quad(out, q, r.quads, f32x4_t{value(q * 4), value(q * 4 + 1), value(q * 4 + 2), value(q * 4 + 3)});
    }
    if (r.vt < a.V) out[r.vt] = value(r.vt);
    return;
  }
  const Exponent of(top, temp);
  float sum = 0.f;
  for (int i = threadIdx.x; i < segs; i += kSegThreads)
    sum += mine[i].top > -__builtin_inff() ? mine[i].sum * of(mine[i].top) : 0.f;
  const float inv = 1.0f / group_sum<kSegThreads>(sum, sh.sum);
#pragma unroll
  for (int n = 0; n < kSegQuads; ++n) {
    f32x4_t y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = of(x[n].at(k)) * inv;
    store_quad(out, r.q0 + n * kSegThreads, r.quads, y);
  }
  if (r.vt < a.V) out[r.vt] = of(xt) * inv;
}

// Rows of a launch: it has fewer than 2^32 work-items (launch_k).  More rows go
// in pieces of whole sequences, or of a part of one: a piece's first row is at
// its first temperature.
constexpr int64_t kMostRows = 1 << 21;

// Few long rows are split.  One workgroup a row / split, in us (float32; bf16
// changes sides within one column of it):
//   V        1 row       16          64          96          128         200
//   32001    6.1/8.0     6.5/8.4     7.3/9.3     8.0/10.5    8.9/11.4    10.5/15.0
//   40000    8.3/7.9     8.8/8.5     10.0/10.1   11.0/11.2   11.8/13.0   15.0/17.2
//   65536    9.1/8.0     9.7/8.7     11.6/11.4   14.2/14.5   17.0/17.2   21.7/27.4
//   128000   22.8/8.1    23.7/9.3    27.4/17.6   30.5/25.4   34.8/31.8   48.0/49.0
//   200000   36.4/8.1    37.5/10.7   43.4/27.3   46.9/38.5   53.4/48.9   77.6/74.6
// (From 128000 on 65 to 128 rows would gain by it too; up to 64 every length past
// 32768 does, 40000 by nothing at 64.)
bool probs_splits(int64_t rows, int64_t V) { return rows <= 64 && V > 32768; }

int probs_segments(int64_t V) { return static_cast<int>((V + kSegment - 1) / kSegment); }

template <int DT>
hipError_t launch_probs_dt(const ProbsArgs& a, int64_t rows, bool split, void* ws, hipStream_t s) {
  if (split) {
    const int segs = probs_segments(a.V);
    const dim3 wide(static_cast<unsigned>(rows * segs));
    prof_stage("token_probs_segments_kernel");
    launch_k(probs_segments_kernel<DT>, wide, dim3(kSegThreads), 0, s, a, segs, static_cast<Segment*>(ws));
    const hipError_t e = launch_error();
    if (e != hipSuccess) return e;
    prof_stage("token_probs_join_kernel");
    launch_k(probs_join_kernel<DT>, wide, dim3(kSegThreads), 0, s, a, segs, static_cast<const Segment*>(ws));
    return launch_error();
  }
  const dim3 grid(static_cast<unsigned>(rows));
  prof_stage("token_probs_kernel");
  // the fewest registers that hold a row
  if (a.V <= 1024 * 2) launch_k((probs_kernel<DT, 256, 2>), grid, dim3(256), 0, s, a);
  else if (a.V <= 1024 * 8) launch_k((probs_kernel<DT, 256, 8>), grid, dim3(256), 0, s, a);
  else if (a.V <= 4096 * 4) launch_k((probs_kernel<DT, 1024, 4>), grid, dim3(1024), 0, s, a);
  else if (a.V <= 4096 * 8) launch_k((probs_kernel<DT, 1024, 8>), grid, dim3(1024), 0, s, a);
  else if (a.V <= 4096 * 16) launch_k((probs_kernel<DT, 1024, 16>), grid, dim3(1024), 0, s, a);
  else if (DT == ENGRAM_BF16 && a.V <= 4096 * 32) launch_k((probs_kernel<ENGRAM_BF16, 1024, 32>), grid, dim3(1024), 0, s, a);
  else launch_k(probs_long_kernel<DT>, grid, dim3(1024), 0, s, a);
  return launch_error();
}

}  // namespace

size_t probs_workspace(int64_t rows, int64_t V) {
  return probs_splits(rows, V) ? static_cast<size_t>(rows) * probs_segments(V) * sizeof(Segment) : 0;
}

hipError_t launch_token_probs(const void* logits, int dtype, int64_t rows, int64_t V, int64_t ld, const float* temperature,
                              int64_t per, float* probs, void* ws, hipStream_t s) {
  const int64_t size = dtype == ENGRAM_BF16 ? 2 : 4;
  const bool split = probs_splits(rows, V);
  for (int64_t r = 0; r < rows;) {
    const int64_t n = std::min(rows - r, per <= kMostRows ? kMostRows / per * per : std::min(kMostRows, per - r % per));
    const ProbsArgs a{static_cast<const char*>(logits) + r * ld * size, temperature != nullptr ? temperature + r / per : nullptr,
                      probs + r * V, V, ld, per};
    const hipError_t e = dtype == ENGRAM_BF16 ? launch_probs_dt<ENGRAM_BF16>(a, n, split, ws, s)
                                              : launch_probs_dt<ENGRAM_F32>(a, n, split, ws, s);
    if (e != hipSuccess) return e;
    r += n;
  }
  return hipSuccess;
}

namespace {

// ---- verification ----
// A draft x_i is accepted while u_i q_i(x_i) < p_i(x_i) (both sides exact in
// double: 24-bit factors).  The next token comes from the row r of the first
// refusal, r = max(p - q, 0), or from p itself behind the last accepted draft
// (and where p - q leaves nothing): the lowest index whose cumulative sum
// passes u * total.  Sums are in double: a border between two tokens then
// moves by about 2^-50 of the total rather than 2^-22.
//
// The row (and the draft's) is read once: every wavefront sums a contiguous
// part of it.  The part in which the cumulative sum passes u * total is then
// read again, by the whole workgroup, to find the token.

struct VerifyArgs {
  const void* target;      // [S][G+1][V]
  const void* draft;       // [S][G][V] or null: each draft had probability 1
  const int32_t* drafted;  // [S][G]
  const int32_t* n_draft;  // [S] or null: G each
  const float* u_accept;   // [S][G]
  const float* u_sample;   // [S]
  int32_t* tokens;         // [S][G+1]
  int32_t* n_accepted;     // [S]
  double* part;            // [S][kParts], split form
  int64_t V;
  int G;
};

constexpr int kParts = 64;        // parts of a row in the split form
constexpr int kVerifyWaves = 16;  // wavefronts of a workgroup; parts of a row in the one-workgroup form

template <int DT>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (DT == ENGRAM_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <int DT>
constexpr int vec_of() { return DT == ENGRAM_BF16 ? 8 : 4; }

// 16 bytes of a row from any element on.
template <int DT>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&f)[vec_of<DT>()]) {
  if constexpr (DT == ENGRAM_BF16) {
    uint4 w;
    __builtin_memcpy(&w, static_cast<const uint16_t*>(p) + i, 16);
    unpack8(w, f);
  } else {
    __builtin_memcpy(f, static_cast<const float*>(p) + i, 16);
  }
}

// The row that the next token is drawn from.
struct Rest {
  const void* p;   // the target's row
  const void* q;   // the draft's, or null
  int32_t drop;    // token with draft probability 1, or -1
};

// An entry of it; a NaN counts as nothing.
__device__ __forceinline__ double entry(double p, double q, bool dropped) {
  const double d = p - q;
  return dropped ? 0.0 : fmax(d, 0.0);
}

template <int DT>
__device__ __forceinline__ double entry_at(const Rest& r, int64_t v) {
  return entry(prob<DT>(r.p, v), r.q != nullptr ? prob<DT>(r.q, v) : 0.0f, v == r.drop);
}

// Accepted drafts of sequence s, and the row for the next token.  Every
// wavefront of the workgroup computes it: lane i looks at draft i.
template <int DT>
__device__ __forceinline__ int accepted(const VerifyArgs& a, int64_t s, Rest* rest) {
  const int lane = threadIdx.x & 63;
  const int32_t x = lane < a.G ? a.drafted[s * a.G + lane] : 0;
  const float u = lane < a.G ? a.u_accept[s * a.G + lane] : 0.f;
  const int n = a.n_draft != nullptr ? min(max(a.n_draft[s], 0), a.G) : a.G;
  bool ok = x >= 0 && x < a.V;
  if (lane < a.G && ok) {
    const double p = prob<DT>(a.target, (s * (a.G + 1) + lane) * a.V + x);
    const double q = a.draft != nullptr ? prob<DT>(a.draft, (s * a.G + lane) * a.V + x) : 1.0f;
    ok = static_cast<double>(u) * q < p;
  }
  const uint64_t bad = __ballot(lane < n && !ok);
  const int acc = bad != 0 ? __builtin_ctzll(bad) : n;
  constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
  rest->p = static_cast<const char*>(a.target) + (s * (a.G + 1) + acc) * a.V * size;
  rest->q = bad != 0 && a.draft != nullptr ? static_cast<const char*>(a.draft) + (s * a.G + acc) * a.V * size : nullptr;
  rest->drop = bad != 0 && a.draft == nullptr ? __shfl(x, acc, 64) : -1;
  return acc;
}

// Length of a part: whole wavefront loads.
template <int DT>
__device__ __forceinline__ int64_t part_len(int64_t V, int parts) {
  constexpr int64_t unit = 64 * vec_of<DT>();
  return ((V + parts - 1) / parts + unit - 1) / unit * unit;
}

// Sum of entries [v0, min(v0 + len, V)) by one wavefront, in every lane.
template <int DT, bool Q>
__device__ __forceinline__ double part_sum(const Rest& r, int64_t v0, int64_t len, int64_t V) {
  constexpr int VEC = vec_of<DT>(), U = 16 / VEC;
  const int lane = threadIdx.x & 63;
  const int64_t end = min(v0 + len, V);
  double s[2] = {0.0, 0.0};
  // U runs of VEC entries a lane, all loads in flight; `whole`: all of them
  // before `end`, else the runs that are not are read from end - VEC on and the
  // entries that a run does not have itself left out
  auto take = [&](int64_t at, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float p[U][VEC], q[U][VEC];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t v = at + (i * 64 + lane) * VEC, from = kWhole ? v : min(v, end - VEC);
      load_vec<DT>(r.p, from, p[i]);
      if constexpr (Q) load_vec<DT>(r.q, from, q[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t v = at + (i * 64 + lane) * VEC, from = kWhole ? v : min(v, end - VEC);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const double x = entry(p[i][k], Q ? q[i][k] : 0.0f, !Q && static_cast<int32_t>(from) + k == r.drop);
        s[k & 1] += kWhole || from + k >= v ? x : 0.0;
      }
    }
  };
  constexpr int64_t step = U * 64 * VEC;
  int64_t at = v0;
  for (; at + step <= end; at += step) take(at, std::true_type{});
  if (at < end) {
    if (V >= VEC) {
      take(at, std::false_type{});
    } else {   // a row shorter than a run
      const int64_t v = at + lane;
      if (v < end) s[0] = entry_at<DT>(r, v);
    }
  }
  return at_lane(wave_scan(s[0] + s[1]), 63);
}

template <int DT>
__device__ __forceinline__ double part_sum(const Rest& r, int64_t v0, int64_t len, int64_t V) {
  return r.q != nullptr ? part_sum<DT, true>(r, v0, len, V) : part_sum<DT, false>(r, v0, len, V);
}

struct PickShared {
  double part[kParts];
  double wave[kVerifyWaves];
  int found[kVerifyWaves], last[kVerifyWaves];
};

// The next token of a row whose part sums are in sh.part (visible to the
// workgroup), -1 where the row holds nothing.  *none: the parts sum to zero.
template <int DT>
__device__ __forceinline__ int64_t pick(const Rest& r, PickShared& sh, int parts, int64_t len, int64_t V, float u, bool* none) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const double x = lane < parts ? sh.part[lane] : 0.0;
  const double scan = wave_scan(x);
  const double total = at_lane(scan, 63), want = static_cast<double>(u) * total;
  *none = !(total > 0.0);
  if (*none || !(total < __builtin_inf())) return -1;
  const uint64_t over = __ballot(x > 0.0 && scan > want), any = __ballot(x > 0.0);
  const bool past = over == 0;   // u not below 1: the last token that has any probability
  const int part = past ? 63 - __builtin_clzll(any) : __builtin_ctzll(over);
  const double left = part > 0 ? at_lane(scan, part - 1) : 0.0;
  // this thread's run of the part
  const int run = static_cast<int>((len + 64 * kVerifyWaves - 1) / (64 * kVerifyWaves));
  const int64_t v0 = part * len + static_cast<int64_t>(tid) * run, v1 = min(min(v0 + run, (part + 1) * len), V);
  constexpr int kKept = 8;
  double e[kKept], sum = 0.0;
#pragma unroll
  for (int i = 0; i < kKept; ++i) e[i] = i < run && v0 + i < v1 ? entry_at<DT>(r, v0 + i) : 0.0;
#pragma unroll
  for (int i = 0; i < kKept; ++i) sum += e[i];
  for (int64_t v = v0 + kKept; v < v1; ++v) sum += entry_at<DT>(r, v);
  const double inside = wave_scan(sum);
  if (lane == 63) sh.wave[wave] = inside;
  __syncthreads();
  double at = left;
  for (int w = 0; w < wave; ++w) at += sh.wave[w];
  at += from_lane<kWaveShr1, 0xf>(0.0, inside);
  // the first of this run that passes (in a chunk of its own kind: offsets
  // within the part fit an int), and the last one that has any probability
  int found = INT32_MAX, last = -1;
  const int base = static_cast<int>(v0 - part * len);
  if (sum > 0.0) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      at += e[i];
      if (e[i] > 0.0) {
        last = base + i;
        if (found == INT32_MAX && !past && at > want) found = base + i;
      }
    }
    for (int64_t v = v0 + kKept; v < v1; ++v) {
      const double d = entry_at<DT>(r, v);
      at += d;
      if (d > 0.0) {
        last = base + static_cast<int>(v - v0);
        if (found == INT32_MAX && !past && at > want) found = last;
      }
    }
  }
  // (runs ascend with the lanes, and with the wavefronts)
  const uint64_t founds = __ballot(found != INT32_MAX), lasts = __ballot(last >= 0);
  found = founds != 0 ? __builtin_amdgcn_readlane(found, __builtin_ctzll(founds)) : INT32_MAX;
  last = lasts != 0 ? __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(lasts)) : -1;
  if (lane == 0) {
    sh.found[wave] = found;
    sh.last[wave] = last;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kVerifyWaves; ++w) {
    found = min(found, sh.found[w]);
    last = max(last, sh.last[w]);
  }
  // the part's sum was formed in another order: by a last bit the second one
  // may not reach what the first reached
  return part * len + (found != INT32_MAX ? found : last);
}

// Part sums of the whole row by this workgroup.
template <int DT>
__device__ __forceinline__ void sum_row(const Rest& r, PickShared& sh, int64_t len, int64_t V) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const double x = part_sum<DT>(r, wave * len, len, V);
  if ((threadIdx.x & 63) == 0) sh.part[wave] = x;
  __syncthreads();
}

// SPLIT: part sums from the workspace (verify_parts_kernel); otherwise this
// workgroup reads the whole row.
template <int DT, bool SPLIT>
__global__ void __launch_bounds__(64 * kVerifyWaves)
verify_kernel(VerifyArgs a) {
  __shared__ PickShared sh;
  const int64_t s = blockIdx.x;
  const int tid = threadIdx.x;
  Rest r;
  const float u = a.u_sample[s];
  const int acc = accepted<DT>(a, s, &r);
  const int parts = SPLIT ? kParts : kVerifyWaves;
  const int64_t len = part_len<DT>(a.V, parts);
  if constexpr (SPLIT) {
    if (tid < kParts) sh.part[tid] = a.part[s * kParts + tid];
    __syncthreads();
  } else {
    sum_row<DT>(r, sh, len, a.V);
  }
  bool none;
  int64_t token = pick<DT>(r, sh, parts, len, a.V, u, &none);
  if (none && (r.q != nullptr || r.drop >= 0)) {   // the draft leaves nothing: from the target's row itself
    __syncthreads();
    r.q = nullptr;
    r.drop = -1;
    const int64_t own = part_len<DT>(a.V, kVerifyWaves);
    sum_row<DT>(r, sh, own, a.V);
    token = pick<DT>(r, sh, kVerifyWaves, own, a.V, u, &none);
  }
  if (tid == 0) a.n_accepted[s] = acc;
  if (tid <= a.G)
    a.tokens[s * (a.G + 1) + tid] = tid < acc ? a.drafted[s * a.G + tid] : (tid == acc ? static_cast<int32_t>(token) : -1);
}

// Split form, first launch: kParts part sums of each sequence's row, one
// wavefront each.
constexpr int kPartWaves = 4;
template <int DT>
__global__ void __launch_bounds__(64 * kPartWaves)
verify_parts_kernel(VerifyArgs a) {
  const int64_t s = blockIdx.x / (kParts / kPartWaves);
  const int part = static_cast<int>(blockIdx.x % (kParts / kPartWaves)) * kPartWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Rest r;
  accepted<DT>(a, s, &r);
  const int64_t len = part_len<DT>(a.V, kParts);
  const double x = part_sum<DT>(r, part * len, len, a.V);
  if ((threadIdx.x & 63) == 0) a.part[s * kParts + part] = x;
}

// Long rows: the sums are split over 16 workgroups a row, in a launch of their
// own.  One launch / two, in us: 1 x 32000 6.6 / 6.8, 1 x 65536 9.4 / 6.9, 1 x 128000
// 15.3 / 7.5, 64 x 65536 10.0 / 9.6, 128 x 65536 15.2 / 16.3, 128 x 128000 28.7 /
// 25.3, 256 x 128000 46.6 / 41.9.
bool verify_splits(int64_t S, int64_t V) { return V > (S <= 64 ? 49152 : 81920); }

template <int DT>
hipError_t launch_verify_dt(const VerifyArgs& a, int64_t S, hipStream_t s) {
  if (verify_splits(S, a.V)) {
    prof_stage("verify_parts_kernel");
    launch_k(verify_parts_kernel<DT>, dim3(static_cast<unsigned>(S * (kParts / kPartWaves))), dim3(64 * kPartWaves), 0, s, a);
    const hipError_t e = launch_error();
    if (e != hipSuccess) return e;
    prof_stage("verify_drafts_kernel");
    launch_k((verify_kernel<DT, true>), dim3(static_cast<unsigned>(S)), dim3(64 * kVerifyWaves), 0, s, a);
  } else {
    prof_stage("verify_drafts_kernel");
    launch_k((verify_kernel<DT, false>), dim3(static_cast<unsigned>(S)), dim3(64 * kVerifyWaves), 0, s, a);
  }
  return launch_error();
}

}  // namespace

size_t verify_workspace(int64_t S, int64_t V) { return verify_splits(S, V) ? static_cast<size_t>(S) * kParts * sizeof(double) : 0; }

hipError_t launch_verify(const void* target, const void* draft, int dtype, const int32_t* drafted, const int32_t* n_draft,
                         const float* u_accept, const float* u_sample, int64_t S, int32_t G, int64_t V, int32_t* tokens,
                         int32_t* n_accepted, void* ws, hipStream_t s) {
  if (S == 0) return hipSuccess;
  const VerifyArgs a{target, draft, drafted, n_draft, u_accept, u_sample, tokens, n_accepted, static_cast<double*>(ws), V, G};
  return dtype == ENGRAM_BF16 ? launch_verify_dt<ENGRAM_BF16>(a, S, s) : launch_verify_dt<ENGRAM_F32>(a, S, s);
}

}  // namespace engram
