// The next token of each row of logits, drawn with temperature, top-k, top-p
// and min-p from a given random number.
//
//   w_v = e^((l_v - max) / T)
//   order: larger logits first, equal ones by index
//   kept: the first top_k of the order; of those the shortest beginning whose
//         weights reach top_p of theirs; and w_v >= min_p
//   token: the lowest index whose running sum of kept weights passes
//          u * (their total)
//
// Weights are whole multiples of 2^-F (F = 45 at 128000 entries): formed in
// double, rounded once, then added as 64-bit integers.  Integer sums do not
// depend on their order, so a row is summed by whichever thread holds an entry
// and binned with LDS atomics, and the token is the same bits each time and
// however the row is split.  In float32 a border between two tokens would move
// by about 2^-24 of the total, which among 128000 tokens changes one draw in
// some hundred; here it moves by about 2^-F.
#include <algorithm>

#include "device_util.h"
#include "engram_internal.h"
#include "lanes_device.h"

namespace engram {
namespace {

struct SampleArgs {
  const void* logits;
  const float* temperature;   // of each sequence (per rows), or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;             // [rows]
  int32_t* tokens;            // [rows]
  float* logprob;             // [rows] or null
  int64_t V;
  int64_t ld;
  int64_t per;
  int32_t fraction;           // F
};

// A float's place among the floats: larger ones have larger keys, -0 is 0.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l == 0.f ? 0.f : l);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }

// 2^f, |f| <= 1/2: the series of e^(f ln 2) to the 11th power (what is left out is below 2^-47).
__device__ __forceinline__ double exp2_half(double f) {
  constexpr double c[12] = {1.0, 0x1.62e42fefa39efp-1, 0x1.ebfbdff82c58fp-3, 0x1.c6b08d704a0c0p-5, 0x1.3b2ab6fba4e77p-7,
                            0x1.5d87fe78a6731p-10, 0x1.430912f86c787p-13, 0x1.ffcbfc588b0c7p-17, 0x1.62c0223a5c824p-20,
                            0x1.b5253d395e7c4p-24, 0x1.e4cf5158b8ecap-28, 0x1.e8cac7351bb25p-32};   // (ln 2)^k / k!
  double p = c[11];
#pragma unroll
  for (int k = 10; k >= 0; --k) p = fma(p, f, c[k]);
  return p;
}

// The weight of a logit and its exponent in powers of two.
struct Weight {
  double top, a;
  int fraction;
  // <= 0; a masked logit's is far below every weight (and not the NaN that -inf at T = inf would give)
  __device__ __forceinline__ double exponent(float l) const { return fmax((static_cast<double>(l) - top) * a, -1100.0); }
  // 2^y in units of 2^-F
  __device__ __forceinline__ uint64_t units(double y) const {
    const double n = rint(y);
    const double w = ldexp(exp2_half(y - n), static_cast<int>(n) + fraction);
    return __double_as_longlong(w + 0x1p52) - __double_as_longlong(0x1p52);
  }
  __device__ __forceinline__ uint64_t operator()(float l) const { return units(exponent(l)); }
};

// A row as its workgroup reads it: each wavefront a contiguous part, in runs
// of 4 a lane.  N > 0: held in registers; N = 0: read again by every pass
// (from the caches, as far as they hold it).
template <int DT, int THREADS, int N>
struct Row {
  const void* in;
  int64_t V, quads, part;   // part: runs of 64 * 4 entries of a wavefront
  Quad<DT> x[N > 0 ? N : 1];
  float xt;                 // the entry behind the quads, the first threads'
  int64_t vt;

  static constexpr int kWaves = THREADS / 64;
  __device__ __forceinline__ int64_t first() const { return (static_cast<int64_t>(threadIdx.x >> 6) * part) * 64 + (threadIdx.x & 63); }
  __device__ __forceinline__ void load(const void* row, int64_t v) {
    in = row;
    V = v;
    quads = v / 4;
    part = N > 0 ? N : (quads + 64 * kWaves - 1) / (64 * kWaves);
    if constexpr (N > 0) {
      const int64_t q0 = first();
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] = load_quad<DT>(in, q0 + n * 64, quads);
    }
    vt = quads * 4 + threadIdx.x;
    xt = load_tail<DT>(in, vt, V);
  }
  // f(l[4], index of the first)
  template <typename F>
  __device__ __forceinline__ void each_quad(F f) {
    const int64_t q0 = first();
    if constexpr (N > 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) l[k] = x[n].at(k);
        f(l, static_cast<uint32_t>(q0 + n * 64) * 4);
      }
      forget(x);
    } else {
      constexpr int U = 4;
      for (int64_t n = 0; n < part; n += U) {
        Quad<DT> y[U];
#pragma unroll
        for (int i = 0; i < U; ++i) y[i] = load_quad<DT>(in, n + i < part ? q0 + (n + i) * 64 : quads, quads);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) l[k] = y[i].at(k);
          f(l, static_cast<uint32_t>(q0 + (n + i) * 64) * 4);
        }
      }
    }
  }
  // f(l, index), the entries behind the quads among them
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    each_quad([&](const float (&l)[4], uint32_t v) {
#pragma unroll
      for (int k = 0; k < 4; ++k) f(l[k], v + k);
    });
    if (vt < V) f(xt, static_cast<uint32_t>(vt));
  }
};

constexpr int kBins = 2048;
constexpr int kListed = 4096;   // entries of one bin that fit the list

template <int THREADS>
struct SampleShared {
  uint64_t bins[kBins];
  uint64_t list[kListed];
  uint64_t wave[THREADS / 64];
  uint64_t part[THREADS / 64 + 1];
  uint64_t low, high, before, total;
  float red[THREADS / 64];
  int first[THREADS / 64];
  int bin;
  int listed;
};

// Sums of the threads before this one; *total: of all.
template <int THREADS>
__device__ __forceinline__ uint64_t group_scan(uint64_t x, uint64_t* wave, uint64_t* total) {
  const uint64_t upto = wave_scan(x);
  __syncthreads();   // (the last call's sums have been read)
  if ((threadIdx.x & 63) == 63) wave[threadIdx.x >> 6] = upto;
  __syncthreads();
  uint64_t before = upto - x, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    before += w < static_cast<int>(threadIdx.x >> 6) ? wave[w] : 0;
    all += wave[w];
  }
  *total = all;
  return before;
}

// The bin in which the bins' running sum (beginning at `before`) reaches `want`, into
// sh.bin, and the sum in front of it into sh.before.  The bins' sums are complete.
template <int THREADS>
__device__ __forceinline__ void find_bin(SampleShared<THREADS>& sh, uint64_t before, uint64_t want) {
  constexpr int kEach = kBins / THREADS;
  uint64_t b[kEach], sum = 0, all;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    b[i] = sh.bins[threadIdx.x * kEach + i];
    sum += b[i];
  }
  uint64_t at = before + group_scan<THREADS>(sum, sh.wave, &all);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (at < want && at + b[i] >= want) {
      sh.bin = threadIdx.x * kEach + i;
      sh.before = at;
    }
    at += b[i];
  }
  __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ void clear_bins(SampleShared<THREADS>& sh) {
#pragma unroll
  for (int i = 0; i < kBins / THREADS; ++i) sh.bins[i * THREADS + threadIdx.x] = 0;
}

// An entry's place in the order: smaller comes first.
struct Place {
  uint32_t top_key;
  __device__ __forceinline__ uint64_t operator()(float l, uint32_t v) const { return static_cast<uint64_t>(top_key - order_key(l)) << 32 | v; }
  __device__ __forceinline__ float logit(uint64_t place) const { return of_key(top_key - static_cast<uint32_t>(place >> 32)); }
};

// The place at which the running sum over the order reaches `want`, given the
// sum `before` of the entries in front of those that `entries` visits (each
// once, as f(place)).  Rounds of kBins bins over the places that are left.
template <int THREADS, typename Entries, typename Amount>
__device__ __forceinline__ uint64_t find_place(SampleShared<THREADS>& sh, uint64_t before, uint64_t want, Entries entries, Amount amount) {
  uint64_t lo = 0, hi = ~uint64_t{0};
  for (;;) {
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.low = ~uint64_t{0};
      sh.high = 0;
    }
    clear_bins<THREADS>(sh);
    __syncthreads();
    uint64_t mn = ~uint64_t{0}, mx = 0;
    entries([&](uint64_t p) {
      if (p >= lo && p <= hi) {
        mn = min(mn, p);
        mx = max(mx, p);
      }
    });
    if (mn <= mx) {
      atomicMin(reinterpret_cast<unsigned long long*>(&sh.low), mn);
      atomicMax(reinterpret_cast<unsigned long long*>(&sh.high), mx);
    }
    __syncthreads();
    mn = sh.low;
    mx = sh.high;
    if (mn >= mx) return mn;
    const int shift = max(64 - __builtin_clzll(mx - mn) - 11, 0);
    entries([&](uint64_t p) {
      if (p >= mn && p <= mx) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[(p - mn) >> shift]), amount(p));
    });
    __syncthreads();
    find_bin<THREADS>(sh, before, want);
    before = sh.before;
    lo = mn + (static_cast<uint64_t>(sh.bin) << shift);
    hi = lo + ((uint64_t{1} << shift) - 1);
    if (shift == 0) return lo;
  }
}

// The last place of the order that stays: SUM ? the entries up to `cut` have
// weights S and stay while the sum in front of them is below top_p S : the
// first top_k of them stay.  First bins over the logits (their distance from
// the largest, in steps of `step`), then the one bin in which it ends.
template <bool SUM, int DT, int THREADS, int N>
__device__ __forceinline__ uint64_t find_cut(SampleShared<THREADS>& sh, Row<DT, THREADS, N>& row, const Weight& weight, const Place& place,
                                             float top, float step, uint64_t cut, uint64_t k, float p) {
  // (non-negative, not decreasing in the distance)
  auto bin_of = [&](float l) { return static_cast<int>(fminf((top - l) * step, kBins - 1.0f)); };
  const float lcut = cut == ~uint64_t{0} ? -__builtin_inff() : place.logit(cut);
  const uint32_t vcut = static_cast<uint32_t>(cut);
  auto in = [&](float l, uint32_t v) { return l >= lcut && (l > lcut || v <= vcut) && l > -__builtin_inff(); };
  __syncthreads();
  clear_bins<THREADS>(sh);
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
  uint64_t rest = 0;   // the last bin takes whatever lies far from the largest: not by atomics
  row.each([&](float l, uint32_t v) {
    if (!in(l, v)) return;
    const int b = bin_of(l);
    const uint64_t x = SUM ? weight(l) : 1;
    if (b == kBins - 1) rest += x;
    else atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[b]), x);
  });
  if (rest > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[kBins - 1]), rest);
  __syncthreads();
  uint64_t want = k;
  {
    uint64_t sum = 0, all;
#pragma unroll
    for (int i = 0; i < kBins / THREADS; ++i) sum += sh.bins[i * THREADS + threadIdx.x];
    group_scan<THREADS>(sum, sh.wave, &all);
    if constexpr (SUM) want = max(static_cast<uint64_t>(ceil(static_cast<double>(p) * static_cast<double>(all))), uint64_t{1});
    if (want >= all) return cut;   // everything stays
  }
  find_bin<THREADS>(sh, 0, want);
  const int bin = sh.bin;
  const uint64_t before = sh.before;
  row.each([&](float l, uint32_t v) {
    if (!in(l, v) || bin_of(l) != bin) return;
    const int at = atomicAdd(&sh.listed, 1);
    if (at < kListed) sh.list[at] = place(l, v);
  });
  __syncthreads();
  const int listed = sh.listed;
  auto amount = [&](uint64_t at) { return SUM ? weight(place.logit(at)) : uint64_t{1}; };
  if (listed <= kListed)
    return find_place<THREADS>(sh, before, want, [&](auto f) {
      for (int i = threadIdx.x; i < listed; i += THREADS) f(sh.list[i]);
    }, amount);
  return find_place<THREADS>(sh, before, want, [&](auto f) {   // (many equal logits)
    row.each([&](float l, uint32_t v) {
      if (in(l, v) && bin_of(l) == bin) f(place(l, v));
    });
  }, amount);
}

template <int DT, int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
sample_kernel(SampleArgs a) {
  __shared__ SampleShared<THREADS> sh;
  const int64_t row_at = blockIdx.x, seq = row_at / a.per, V = a.V;
  constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
  Row<DT, THREADS, N> row;
  row.load(static_cast<const char*>(a.logits) + row_at * a.ld * size, V);
  const float temp = a.temperature != nullptr ? a.temperature[seq] : 1.0f;
  const int32_t k = a.top_k != nullptr ? a.top_k[seq] : 0;
  const float p = a.top_p != nullptr ? a.top_p[seq] : 1.0f;
  const float m = a.min_p != nullptr ? a.min_p[seq] : 0.0f;
  const float u = a.u[row_at];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  float top = -__builtin_inff();
  bool nan = false;
  row.each([&](float l, uint32_t) {
    nan |= l != l;
    top = fmaxf(top, l);
  });
  top = group_max<THREADS>(top, nan, sh.red);
  if (top != top || top == -__builtin_inff() || (top == __builtin_inff() && temp > 0.f)) {
    if (threadIdx.x == 0) {
      a.tokens[row_at] = -1;
      if (a.logprob != nullptr) a.logprob[row_at] = -__builtin_inff();
    }
    return;
  }
  if (!(temp > 0.f)) {
    uint32_t at = ~0u;
    row.each([&](float l, uint32_t v) { at = l == top ? min(at, v) : at; });
    if (threadIdx.x == 0) sh.bin = INT32_MAX;
    __syncthreads();
    if (at != ~0u) atomicMin(&sh.bin, static_cast<int>(at));
    __syncthreads();
    if (threadIdx.x == 0) {
      a.tokens[row_at] = sh.bin;
      if (a.logprob != nullptr) a.logprob[row_at] = 0.f;
    }
    return;
  }

  constexpr double kLog2e = 1.4426950408889634074;
  const Weight weight{top, kLog2e / temp, a.fraction};
  const Place place{order_key(top)};
  // bins of 3/128 of a power of two, 48 powers in all
  const float step = fminf(fmaxf(static_cast<float>(weight.a) * (kBins / 48.0f), 0x1p-126f), 0x1p126f);
  uint64_t cut = ~uint64_t{0};
  if (k > 0 && k < V) cut = find_cut<false>(sh, row, weight, place, top, step, cut, k, 0.f);
  if (p < 1.0f) cut = find_cut<true>(sh, row, weight, place, top, step, cut, 0, p);
  const double least = m > 0.f ? log2(static_cast<double>(fminf(m, 1.0f))) : -__builtin_inf();   // min_p as an exponent
  const float lcut = cut == ~uint64_t{0} ? -__builtin_inff() : place.logit(cut);
  const uint32_t vcut = static_cast<uint32_t>(cut);
  // an entry's weight, 0 where it does not stay
  auto kept = [&](float l, uint32_t v) -> uint64_t {
    if (!(l >= lcut && (l > lcut || v <= vcut))) return 0;
    const double y = weight.exponent(l);
    return y >= least ? weight.units(y) : 0;
  };

  // a wavefront's part of the row each, and the entries behind the quads
  uint64_t sum = 0;
  row.each_quad([&](const float (&l)[4], uint32_t v) {
    if (fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) < lcut) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += kept(l[i], v + i);
  });
  sum = wave_scan(sum);
  uint64_t tail = wave == 0 ? wave_scan(row.vt < V ? kept(row.xt, static_cast<uint32_t>(row.vt)) : uint64_t{0}) : 0;
  __syncthreads();
  if (lane == 63) sh.part[wave] = sum;
  if (threadIdx.x == 63) sh.part[THREADS / 64] = tail;
  __syncthreads();
  uint64_t total = 0;
#pragma unroll
  for (int w = 0; w <= THREADS / 64; ++w) total += sh.part[w];
  // the token is the first whose running sum is above `want`
  const uint64_t want = min(static_cast<uint64_t>(fmax(static_cast<double>(u), 0.0) * static_cast<double>(total)), total - 1);
  uint64_t at = 0;
  int part = 0;
  while (at + sh.part[part] <= want) at += sh.part[part++];
  // that part again, by the whole workgroup
  const int64_t v0 = min(part * row.part * 256, row.quads * 4), v1 = part == THREADS / 64 ? V : min(v0 + row.part * 256, row.quads * 4);
  const int64_t from = part == THREADS / 64 ? row.quads * 4 : v0;
  const int64_t run = (v1 - from + THREADS - 1) / THREADS;
  const int64_t b = min(from + threadIdx.x * run, v1), e = min(b + run, v1);
  auto at_index = [&](int64_t v) {
    if constexpr (DT == ENGRAM_BF16) return bf16_to_f32(static_cast<const uint16_t*>(row.in)[v]);
    else return static_cast<const float*>(row.in)[v];
  };
  uint64_t mine = 0, all;
#pragma unroll 8
  for (int64_t v = b; v < e; ++v) mine += kept(at_index(v), static_cast<uint32_t>(v));
  at += group_scan<THREADS>(mine, sh.wave, &all);
  if (at <= want && want < at + mine) {   // one thread's
    for (int64_t v = b; v < e; ++v) {
      const float l = at_index(v);
      const uint64_t w = kept(l, static_cast<uint32_t>(v));
      at += w;
      if (w > 0 && at > want) {
        a.tokens[row_at] = static_cast<int32_t>(v);
        if (a.logprob != nullptr)
          a.logprob[row_at] = static_cast<float>((weight.exponent(l) - (log2(static_cast<double>(total)) - a.fraction)) * 0.69314718055994530942);
        break;
      }
    }
  }
}

// Rows of a launch: it has fewer than 2^32 work-items (launch_k).
constexpr int64_t kMostRows = 1 << 21;

template <int DT>
hipError_t launch_sample_dt(const SampleArgs& a, int64_t rows, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows));
  prof_stage("sample_tokens_kernel");
  // the fewest registers that hold a row
  if (a.V <= 1024 * 2) launch_k((sample_kernel<DT, 256, 2>), grid, dim3(256), 0, s, a);
  else if (a.V <= 1024 * 8) launch_k((sample_kernel<DT, 256, 8>), grid, dim3(256), 0, s, a);
  else if (a.V <= 4096 * 8) launch_k((sample_kernel<DT, 1024, 8>), grid, dim3(1024), 0, s, a);
  else if (a.V <= 4096 * 16) launch_k((sample_kernel<DT, 1024, 16>), grid, dim3(1024), 0, s, a);
  else if (DT == ENGRAM_BF16 && a.V <= 4096 * 32) launch_k((sample_kernel<ENGRAM_BF16, 1024, 32>), grid, dim3(1024), 0, s, a);
  else launch_k((sample_kernel<DT, 1024, 0>), grid, dim3(1024), 0, s, a);
  return launch_error();
}

}  // namespace

hipError_t launch_sample_tokens(const void* logits, int dtype, int64_t rows, int64_t V, int64_t ld, const float* temperature,
                                const int32_t* top_k, const float* top_p, const float* min_p, int64_t per, const float* u,
                                int32_t* tokens, float* logprob, hipStream_t s) {
  const int64_t size = dtype == ENGRAM_BF16 ? 2 : 4;
  int log_v = 0;
  while ((int64_t{1} << log_v) < V) ++log_v;
  const int fraction = std::min(50, 62 - log_v);   // V weights of up to 1 stay below 2^63, one below the 52 bits of a double
  for (int64_t r = 0; r < rows;) {   // pieces of whole sequences, or of a part of one
    const int64_t n = std::min(rows - r, per <= kMostRows ? kMostRows / per * per : std::min(kMostRows, per - r % per));
    const int64_t q = r / per;
    const SampleArgs a{static_cast<const char*>(logits) + r * ld * size, temperature != nullptr ? temperature + q : nullptr,
                       top_k != nullptr ? top_k + q : nullptr, top_p != nullptr ? top_p + q : nullptr,
                       min_p != nullptr ? min_p + q : nullptr, u + r, tokens + r, logprob != nullptr ? logprob + r : nullptr,
                       V, ld, per, fraction};
    const hipError_t e = dtype == ENGRAM_BF16 ? launch_sample_dt<ENGRAM_BF16>(a, n, s) : launch_sample_dt<ENGRAM_F32>(a, n, s);
    if (e != hipSuccess) return e;
    r += n;
  }
  return hipSuccess;
}

}  // namespace engram
