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

// Weights: 2^y = 2^e T_j 2^f with y = e + j / 128 + f, |f| <= 1/256, T_j = 2^(j / 128)
// from a table in LDS and 2^f by its series to the 4th power (what is left out
// is below 2^-49).  13 instructions in double an entry; the series to the 11th
// power alone, without a table, took 30 with their constants' moves (2048 x
// 128000 without filters 524 us).
constexpr int kTable = 128;

__device__ __forceinline__ double table_entry(int j) { return exp2(j * (1.0 / kTable)); }

// The weight of a logit and its exponent, in steps of 1 / kTable of a power of two.
struct Weight {
  double top, a;         // a: kTable log2(e) / T
  int fraction;
  const double* table;   // LDS
  // <= 0; a masked logit's is far below every weight (and not the NaN that -inf at T = inf would give)
  __device__ __forceinline__ double exponent(float l) const { return fmax((static_cast<double>(l) - top) * a, -60.0 * kTable); }
  // the weight in units of 2^-F
  __device__ __forceinline__ uint64_t units(double y) const {
    constexpr double kWhole = 0x1.8p52;   // added, it leaves a whole number in the low bits
    constexpr double c1 = 0x1.62e42fefa39efp-8, c2 = 0x1.ebfbdff82c58fp-17, c3 = 0x1.c6b08d704a0c0p-26, c4 = 0x1.3b2ab6fba4e77p-35;   // (ln 2 / 128)^k / k!
    const double t = y + kWhole, f = y - (t - kWhole);
    const int n = static_cast<int>(__double_as_longlong(t));
    const double base = table[n & (kTable - 1)];
    const double q = f * fma(fma(fma(c4, f, c3), f, c2), f, c1);
    const uint64_t w = __double_as_longlong(fma(base, q, base)) + (static_cast<uint64_t>(static_cast<uint32_t>((n >> 7) + fraction) << 20) << 32);
    return __double_as_longlong(__longlong_as_double(w) + 0x1p52) - __double_as_longlong(0x1p52);
  }
  __device__ __forceinline__ uint64_t operator()(float l) const { return units(exponent(l)); }
  // ln of an exponent's weight over a sum of weights
  __device__ __forceinline__ float log_share(double y, uint64_t total) const {
    return static_cast<float>((y * (1.0 / kTable) - (log2(static_cast<double>(total)) - fraction)) * 0.69314718055994530942);
  }
};

// A row as its workgroup reads it: each wavefront a contiguous part, in runs
// of 4 a lane.  Every pass reads it again, the first from memory, the others
// from the caches, with the next runs in flight behind the current ones.  (Held
// in registers between the passes a row of 128000 spilled 1.4 KiB a lane,
// and the passes unrolled over it did not fit the instruction cache: 2048 rows
// 2350 us.)
template <int DT, int THREADS>
struct Row {
  const void* in;
  int64_t V, quads, part;   // part: runs of 64 * 4 entries of a wavefront
  float xt;                 // the entry behind the quads, the first threads'
  int64_t vt;

  static constexpr int kWaves = THREADS / 64;
  __device__ __forceinline__ void open(const void* row, int64_t v) {
    in = row;
    V = v;
    quads = v / 4;
    part = (quads + 64 * kWaves - 1) / (64 * kWaves);
    vt = quads * 4 + threadIdx.x;
    xt = load_tail<DT>(in, vt, V);
  }
  // f(l[4], index of the first), -inf past the quads; U runs at a time
  template <int U, typename F>
  __device__ __forceinline__ void each_quad(F f) const {
    const int64_t q0 = static_cast<int64_t>(threadIdx.x >> 6) * part * 64 + (threadIdx.x & 63);
    auto load = [&](Quad<DT> (&x)[U], int64_t n) {
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = load_quad<DT>(in, n + i < part ? q0 + (n + i) * 64 : quads, quads);
    };
    Quad<DT> x[U], next[U];
    load(x, 0);
    for (int64_t n = 0; n < part; n += U) {
      load(next, n + U);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) l[k] = x[i].at(k);
        f(l, static_cast<uint32_t>(q0 + (n + i) * 64) * 4);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = next[i];
    }
  }
  // f(l, index), the entries behind the quads among them
  template <int U, typename F>
  __device__ __forceinline__ void each(F f) const {
    each_quad<U>([&](const float (&l)[4], uint32_t v) {
#pragma unroll
      for (int k = 0; k < 4; ++k) f(l[k], v + k);
    });
    if (vt < V) f(xt, static_cast<uint32_t>(vt));
  }
};

// What a workgroup of THREADS keeps in LDS: two of 512 fit a CU; a row of a
// workgroup of 256 (4096 entries at most) always fits its list.
template <int THREADS>
struct SampleShared {
  static constexpr int kBinBits = THREADS <= 256 ? 9 : 11, kBins = 1 << kBinBits;
  static constexpr int kListed = THREADS <= 256 ? 5120 : 7552;   // entries of the list
  static constexpr int kOneBin = THREADS <= 256 ? 1024 : 2048;   // of them, at its end, those of the bin in which a cut lies
  uint64_t bins[kBins];
  uint64_t list[kListed];
  double table[kTable];
  uint64_t few[64];
  uint64_t wave[THREADS / 64], wave2[THREADS / 64];
  uint64_t part[THREADS / 64 + 1];
  uint64_t before;
  float red[THREADS / 64];
  int bin;
  int listed;
  int few_n;
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

// Smallest and largest of the workgroup's values.
template <int THREADS>
__device__ __forceinline__ void group_range(SampleShared<THREADS>& sh, uint64_t* lo, uint64_t* hi) {
  uint64_t a = *lo, b = *hi;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    a = min(a, static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(a), off, 64)));
    b = max(b, static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(b), off, 64)));
  }
  if ((threadIdx.x & 63) == 0) {
    sh.wave[threadIdx.x >> 6] = a;
    sh.wave2[threadIdx.x >> 6] = b;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    a = min(a, sh.wave[w]);
    b = max(b, sh.wave2[w]);
  }
  *lo = a;
  *hi = b;
}

// The bin in which the bins' running sum (beginning at `before`) reaches `want`, into
// sh.bin, and the sum in front of it into sh.before.  The bins' sums are complete.
template <int THREADS>
__device__ __forceinline__ void find_bin(SampleShared<THREADS>& sh, uint64_t before, uint64_t want) {
  constexpr int kEach = SampleShared<THREADS>::kBins / THREADS;
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
  for (int i = 0; i < SampleShared<THREADS>::kBins / THREADS; ++i) sh.bins[i * THREADS + threadIdx.x] = 0;
}

// An entry's place in the order: smaller comes first.
struct Place {
  uint32_t top_key;
  __device__ __forceinline__ uint64_t operator()(float l, uint32_t v) const { return static_cast<uint64_t>(top_key - order_key(l)) << 32 | v; }
  __device__ __forceinline__ float logit(uint64_t place) const { return of_key(top_key - static_cast<uint32_t>(place >> 32)); }
};

// The place at which the running sum over the places' order reaches `want`
// (it does), given the sum `before` of those in front of the ones that
// `entries` visits (each once, as f(place), all in lo .. hi).  Rounds of kBins
// bins over the places that are left; the last 64 of them in registers.
template <int THREADS, typename Entries, typename Amount>
__device__ __forceinline__ uint64_t find_place(SampleShared<THREADS>& sh, uint64_t lo, uint64_t hi, uint64_t before, uint64_t want,
                                               Entries entries, Amount amount) {
  for (;;) {
    const int shift = max(64 - __builtin_clzll((hi - lo) | 1) - SampleShared<THREADS>::kBinBits, 0);
    __syncthreads();
    clear_bins<THREADS>(sh);
    if (threadIdx.x == 0) sh.few_n = 0;
    __syncthreads();
    entries([&](uint64_t p) {
      if (p >= lo && p <= hi) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[(p - lo) >> shift]), amount(p));
    });
    __syncthreads();
    find_bin<THREADS>(sh, before, want);
    before = sh.before;
    lo += static_cast<uint64_t>(sh.bin) << shift;
    hi = lo + ((uint64_t{1} << shift) - 1);
    if (shift == 0) return lo;
    entries([&](uint64_t p) {
      if (p >= lo && p <= hi) {
        const int at = atomicAdd(&sh.few_n, 1);
        if (at < 64) sh.few[at] = p;
      }
    });
    __syncthreads();
    const int n = sh.few_n;
    if (n <= 64) {   // every wavefront: a place a lane, what lies in front of it from the other lanes
      const int lane = threadIdx.x & 63;
      const uint64_t mine = lane < n ? sh.few[lane] : ~uint64_t{0}, own = lane < n ? amount(mine) : 0;
      uint64_t at = before;
      for (int i = 0; i < n; ++i) {
        const uint64_t p = at_lane(mine, i), x = at_lane(own, i);
        at += p < mine ? x : 0;
      }
      const uint64_t here = __ballot(lane < n && at < want && at + own >= want);
      return at_lane(mine, __builtin_ctzll(here));
    }
    // (a bin's places are seldom spread over all of it)
    uint64_t mn = ~uint64_t{0}, mx = 0;
    entries([&](uint64_t p) {
      if (p >= lo && p <= hi) {
        mn = min(mn, p);
        mx = max(mx, p);
      }
    });
    group_range<THREADS>(sh, &mn, &mx);
    lo = mn;
    hi = mx;
  }
}

// What a row's passes know of it.
template <int DT, int THREADS>
struct Draw {
  static constexpr int kBins = SampleShared<THREADS>::kBins, kListed = SampleShared<THREADS>::kListed;
  SampleShared<THREADS>& sh;
  Row<DT, THREADS> row;
  Weight weight;
  Place place;
  float top, step;          // bins over the logits: their distance from the largest in steps
  uint64_t cut;             // the last place that stays
  float lcut;               // its logit
  double least;             // min_p as an exponent
  float floor_l;            // below it nothing stays by min_p

  // (not decreasing in the distance)
  __device__ __forceinline__ int bin_of(float l) const { return static_cast<int>(fminf((top - l) * step, kBins - 1.0f)); }
  __device__ __forceinline__ bool in(float l, uint32_t v) const {
    return l >= lcut && (l > lcut || v <= static_cast<uint32_t>(cut)) && l > -__builtin_inff();
  }
  // an entry's weight, 0 where it does not stay
  __device__ __forceinline__ uint64_t kept(float l, uint32_t v) const {
    const double y = weight.exponent(l);
    const uint64_t w = weight.units(y);
    return l >= lcut && (l > lcut || v <= static_cast<uint32_t>(cut)) && y >= least ? w : 0;
  }
  __device__ __forceinline__ void set_cut(uint64_t c) {
    cut = c;
    lcut = place.logit(c);
  }
  __device__ __forceinline__ uint64_t share(float p, uint64_t all) const {
    return max(static_cast<uint64_t>(ceil(static_cast<double>(p) * static_cast<double>(all))), uint64_t{1});
  }
  // All entries with a logit of `least_l` and more (any order) into the list; false: too many.
  __device__ __forceinline__ bool collect(float least_l, int* n) {
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    row.template each_quad<4>([&](const float (&l)[4], uint32_t v) {
      if (!(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= least_l)) return;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (l[k] >= least_l && l[k] > -__builtin_inff()) {
          const int at = atomicAdd(&sh.listed, 1);
          if (at < kListed) sh.list[at] = place(l[k], v + k);
        }
    });
    if (row.vt < row.V && row.xt >= least_l && row.xt > -__builtin_inff()) {
      const int at = atomicAdd(&sh.listed, 1);
      if (at < kListed) sh.list[at] = place(row.xt, static_cast<uint32_t>(row.vt));
    }
    __syncthreads();
    *n = sh.listed;
    return *n <= kListed;
  }
};

// f(place) of the list's entries up to a cut.
template <int THREADS>
struct Listed {
  const SampleShared<THREADS>& sh;
  int n;
  uint64_t cut;
  template <typename F>
  __device__ __forceinline__ void operator()(F f) const {
    for (int i = threadIdx.x; i < n; i += THREADS)
      if (sh.list[i] <= cut) f(sh.list[i]);
  }
};

// The cut of a row: SUM ? where the weights reach top_p of all up to the cut
// so far : where the first top_k end.  Bins over the logits, then the places in
// the one bin in which it ends.  The entries up to that bin come into the list,
// its own entries at the list's end; *listed: how many there are, -1 where
// they do not fit.
template <bool SUM, int DT, int THREADS>
__device__ __forceinline__ void cut_row(Draw<DT, THREADS>& d, uint64_t k, float p, int* listed) {
  SampleShared<THREADS>& sh = d.sh;
  using Sh = SampleShared<THREADS>;
  constexpr int kBins = Sh::kBins, kOneBin = Sh::kOneBin, kFront = Sh::kListed - kOneBin;
  *listed = -1;
  __syncthreads();
  clear_bins<THREADS>(sh);
  if (threadIdx.x == 0) sh.listed = sh.few_n = 0;
  __syncthreads();
  uint64_t rest = 0;   // the last bin takes whatever lies far from the largest: not by atomics
  auto count = [&](float l, uint32_t v, uint64_t w) {
    const int b = d.bin_of(l);
    const bool in = d.in(l, v);
    rest += in && b == kBins - 1 ? w : 0;
    if (in && b < kBins - 1) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[b]), w);
  };
  d.row.template each_quad<2>([&](const float (&l)[4], uint32_t v) {
    uint64_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = SUM ? d.weight(l[i]) : 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) count(l[i], v + i, w[i]);
  });
  if (d.row.vt < d.row.V) count(d.row.xt, static_cast<uint32_t>(d.row.vt), SUM ? d.weight(d.row.xt) : 1);
  if (rest > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[kBins - 1]), rest);
  __syncthreads();
  uint64_t want = k;
  {
    uint64_t sum = 0, all;
#pragma unroll
    for (int i = 0; i < kBins / THREADS; ++i) sum += sh.bins[i * THREADS + threadIdx.x];
    group_scan<THREADS>(sum, sh.wave, &all);
    if constexpr (SUM) want = d.share(p, all);
    if (want >= all) return;   // everything stays
  }
  find_bin<THREADS>(sh, 0, want);
  const int bin = sh.bin;
  const uint64_t before = sh.before;
  uint64_t lo = ~uint64_t{0}, hi = 0;
  d.row.template each<4>([&](float l, uint32_t v) {
    if (!d.in(l, v) || d.bin_of(l) > bin) return;
    const uint64_t q = d.place(l, v);
    if (d.bin_of(l) < bin) {
      const int at = atomicAdd(&sh.listed, 1);
      if (at < kFront) sh.list[at] = q;
    } else {
      lo = min(lo, q);
      hi = max(hi, q);
      const int at = atomicAdd(&sh.few_n, 1);
      if (at < kOneBin) sh.list[kFront + at] = q;
    }
  });
  group_range<THREADS>(sh, &lo, &hi);   // (its barrier: the list is complete)
  const int front = sh.listed, one = sh.few_n;
  auto amount = [&](uint64_t at) { return SUM ? d.weight(d.place.logit(at)) : uint64_t{1}; };
  if (one <= kOneBin) {
    d.set_cut(find_place<THREADS>(sh, lo, hi, before, want, [&](auto f) {
      for (int i = threadIdx.x; i < one; i += THREADS) f(sh.list[kFront + i]);
    }, amount));
    if (front > kFront) return;
    // the bin's entries behind the others
    uint64_t q[kOneBin / THREADS];
#pragma unroll
    for (int i = 0; i < kOneBin / THREADS; ++i) q[i] = sh.list[kFront + i * THREADS + threadIdx.x];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOneBin / THREADS; ++i) {
      const int at = i * THREADS + threadIdx.x;
      if (at < one) sh.list[front + at] = q[i];
    }
    __syncthreads();
    *listed = front + one;
    return;
  }
  d.set_cut(find_place<THREADS>(sh, lo, hi, before, want, [&](auto f) {   // (many equal logits)
    d.row.template each<2>([&](float l, uint32_t v) {
      if (d.in(l, v) && d.bin_of(l) == bin) f(d.place(l, v));
    });
  }, amount));
}

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 4)   // (four wavefronts a SIMD: two workgroups of 512 a CU)
sample_kernel(SampleArgs a) {
  __shared__ SampleShared<THREADS> sh;
  const int64_t row_at = blockIdx.x, seq = row_at / a.per, V = a.V;
  constexpr int size = DT == ENGRAM_BF16 ? 2 : 4;
  Row<DT, THREADS> row;
  row.open(static_cast<const char*>(a.logits) + row_at * a.ld * size, V);
  const float temp = a.temperature != nullptr ? a.temperature[seq] : 1.0f;
  const int32_t top_k = a.top_k != nullptr ? a.top_k[seq] : 0;
  const float p = a.top_p != nullptr ? a.top_p[seq] : 1.0f;
  const float m = a.min_p != nullptr ? a.min_p[seq] : 0.0f;
  const float u = a.u[row_at];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  float own = row.xt;   // this thread's largest
  bool nan = own != own;
  row.template each_quad<8>([&](const float (&l)[4], uint32_t) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      nan |= l[k] != l[k];
      own = fmaxf(own, l[k]);
    }
  });
  const float top = group_max<THREADS>(own, nan, sh.red);
  if (top != top || top == -__builtin_inff() || (top == __builtin_inff() && temp > 0.f)) {
    if (threadIdx.x == 0) {
      a.tokens[row_at] = -1;
      if (a.logprob != nullptr) a.logprob[row_at] = -__builtin_inff();
    }
    return;
  }
  if (!(temp > 0.f)) {
    uint32_t at = ~0u;
    if (own == top) row.template each<4>([&](float l, uint32_t v) { at = l == top ? min(at, v) : at; });
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

  if (threadIdx.x < kTable) sh.table[threadIdx.x] = table_entry(threadIdx.x);   // (a barrier follows before its first use)
  constexpr double kLog2e = 1.4426950408889634074;
  // bins over 48 powers of two
  Draw<DT, THREADS> d{sh, row, Weight{top, kTable * kLog2e / temp, a.fraction, sh.table}, Place{order_key(top)}, top, 0.f, ~uint64_t{0},
                      -__builtin_inff(), m > 0.f ? kTable * log2(static_cast<double>(fminf(m, 1.0f))) : -__builtin_inf(), -__builtin_inff()};
  d.step = fminf(fmaxf(static_cast<float>(d.weight.a) * (d.kBins / 48.0f / kTable), 0x1p-126f), 0x1p126f);
  if (m > 0.f && d.weight.a > 0.0) {   // the logit at which min_p ends, and a margin for the roundings
    const double at = top + d.least / d.weight.a;
    d.floor_l = static_cast<float>(at - 1e-6 * (fabs(at) + fabs(static_cast<double>(top))));
  }
  const bool by_k = top_k > 0 && top_k < V, by_p = p < 1.0f;

  // Few entries stay (a small top_k): then a list holds them, and the rest is done on
  // the list.  The threads' largest logits bound the top_k-th from below.
  int listed = -1;
  if (by_k && top_k <= THREADS / 2 && V >= 4 * THREADS) {
    // (a thread without a finite entry counts as the last place)
    const uint64_t mine = own > -__builtin_inff() ? d.place(own, threadIdx.x) : ~uint64_t{0};
    uint64_t lo = mine, hi = mine;
    group_range<THREADS>(sh, &lo, &hi);
    const uint64_t kth = find_place<THREADS>(sh, lo, hi, 0, top_k, [&](auto f) { f(mine); }, [](uint64_t) { return uint64_t{1}; });
    const float least_l = kth == ~uint64_t{0} ? -__builtin_inff() : d.place.logit(kth);
    int n;
    if (d.collect(least_l, &n)) {
      listed = n;
      if (n > top_k) {
        d.set_cut(find_place<THREADS>(sh, 0, d.place(least_l, ~0u), 0, top_k, Listed<THREADS>{sh, n, ~uint64_t{0}},
                                      [](uint64_t) { return uint64_t{1}; }));
      }
    }
  }
  if (by_k && listed < 0) cut_row<false>(d, top_k, 0.f, &listed);
  bool p_left = by_p;
  if (by_p && listed < 0) {
    cut_row<true>(d, 0, p, &listed);
    p_left = false;
  }
  if (m > 0.f && !by_k && !by_p) {   // few entries stay by min_p alone
    int n;
    if (d.collect(d.floor_l, &n)) listed = n;
  }
  __syncthreads();
  if (listed >= 0) {
    auto weight_of = [&](uint64_t q) { return d.weight(d.place.logit(q)); };
    const uint64_t last = d.lcut > -__builtin_inff() ? d.place(d.lcut, ~0u) : ~uint64_t{0};
    if (p_left) {
      uint64_t sum = 0, all;
      Listed<THREADS>{sh, listed, d.cut}([&](uint64_t q) { sum += weight_of(q); });
      group_scan<THREADS>(sum, sh.wave, &all);
      d.set_cut(find_place<THREADS>(sh, 0, last, 0, d.share(p, all),
                                    Listed<THREADS>{sh, listed, d.cut}, weight_of));
    }
    auto stays = [&](uint64_t q) {
      const double y = d.weight.exponent(d.place.logit(q));
      return y >= d.least ? d.weight.units(y) : 0;
    };
    const Listed<THREADS> entries{sh, listed, d.cut};
    uint64_t sum = 0, total;
    entries([&](uint64_t q) { sum += stays(q); });
    group_scan<THREADS>(sum, sh.wave, &total);
    const uint64_t want = min(static_cast<uint64_t>(fmin(fmax(static_cast<double>(u), 0.0), 1.0) * static_cast<double>(total)), total - 1);
    // by index: the entry's place with its halves exchanged
    const uint64_t found = find_place<THREADS>(sh, 0, static_cast<uint64_t>(V) << 32 | ~0u, 0, want + 1, [&](auto f) {
      entries([&](uint64_t q) { f(q << 32 | q >> 32); });
    }, [&](uint64_t q) { return stays(q << 32 | q >> 32); });
    if (threadIdx.x == 0) {
      a.tokens[row_at] = static_cast<int32_t>(found >> 32);
      if (a.logprob != nullptr)
        a.logprob[row_at] = d.weight.log_share(d.weight.exponent(d.place.logit(found << 32)), total);
    }
    return;
  }

  // a wavefront's part of the row each, and the entries behind the quads
  const float lowest = fmaxf(d.lcut, d.floor_l);
  uint64_t sum = 0;
  row.template each_quad<2>([&](const float (&l)[4], uint32_t v) {
    if (!(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= lowest)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += d.kept(l[i], v + i);
  });
  sum = wave_scan(sum);
  uint64_t tail = wave == 0 ? wave_scan(row.vt < V ? d.kept(row.xt, static_cast<uint32_t>(row.vt)) : uint64_t{0}) : 0;
  __syncthreads();
  if (lane == 63) sh.part[wave] = sum;
  if (threadIdx.x == 63) sh.part[THREADS / 64] = tail;
  __syncthreads();
  uint64_t total = 0;
#pragma unroll
  for (int w = 0; w <= THREADS / 64; ++w) total += sh.part[w];
  // the token is the first whose running sum is above `want`
  const uint64_t want = min(static_cast<uint64_t>(fmin(fmax(static_cast<double>(u), 0.0), 1.0) * static_cast<double>(total)), total - 1);
  uint64_t at = 0;
  int part = 0;
  while (at + sh.part[part] <= want) at += sh.part[part++];
  // that part again, by the whole workgroup
  const bool behind = part == THREADS / 64;
  const int64_t v0 = behind ? row.quads * 4 : min(part * row.part * 256, row.quads * 4);
  const int64_t v1 = behind ? V : min(v0 + row.part * 256, row.quads * 4);
  const int64_t run = (v1 - v0 + THREADS - 1) / THREADS;
  const int64_t b = min(v0 + threadIdx.x * run, v1), e = min(b + run, v1);
  auto at_index = [&](int64_t v) {
    if constexpr (DT == ENGRAM_BF16) return bf16_to_f32(static_cast<const uint16_t*>(row.in)[v]);
    else return static_cast<const float*>(row.in)[v];
  };
  uint64_t mine = 0, all;
#pragma unroll 4
  for (int64_t v = b; v < e; ++v) mine += d.kept(at_index(v), static_cast<uint32_t>(v));
  at += group_scan<THREADS>(mine, sh.wave, &all);
  if (at <= want && want < at + mine) {   // one thread's
    for (int64_t v = b; v < e; ++v) {
      const float l = at_index(v);
      const uint64_t w = d.kept(l, static_cast<uint32_t>(v));
      at += w;
      if (w > 0 && at > want) {
        a.tokens[row_at] = static_cast<int32_t>(v);
        if (a.logprob != nullptr)
          a.logprob[row_at] = d.weight.log_share(d.weight.exponent(l), total);
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
  if (a.V <= 1024 * 4) launch_k((sample_kernel<DT, 256>), grid, dim3(256), 0, s, a);
  else if (rows <= 256) launch_k((sample_kernel<DT, 1024>), grid, dim3(1024), 0, s, a);
  else launch_k((sample_kernel<DT, 512>), grid, dim3(512), 0, s, a);
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
