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
#include "sample_values.h"

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

// Bins over the weights: 32 a power of two (8 in the small workgroup); the last
// one, 60 powers below the largest weight, holds weights of 0.
constexpr int kSteps = 60 * kTable;

// The weights of a bf16 row's table of values (sample_values.h) lie in LDS, and
// an entry's weight is one read.
struct Weight {
  double top, a;         // a: kTable log2(e) / T
  int fraction;
  int bin_shift;
  const double* table;   // LDS
  uint64_t* values;      // LDS, [2][kValues], or null
  uint32_t base;         // the first value's bits
  // A logit's exponent in steps of 1 / kTable of a power of two, <= 0; a masked logit's is below every weight (and not
  // the NaN that -inf at T = inf would give)
  __device__ __forceinline__ double exponent(float l) const { return fmax((static_cast<double>(l) - top) * a, -static_cast<double>(kSteps)); }
  // Its weight in units of 2^-F (below 2^52), its bin in the bits above.
  __device__ __forceinline__ uint64_t formed(float l) const {
    constexpr double kWhole = 0x1.8p52;   // added, it leaves a whole number in the low bits
    constexpr double c1 = 0x1.62e42fefa39efp-8, c2 = 0x1.ebfbdff82c58fp-17, c3 = 0x1.c6b08d704a0c0p-26, c4 = 0x1.3b2ab6fba4e77p-35;   // (ln 2 / 128)^k / k!
    const double y = exponent(l), t = y + kWhole, f = y - (t - kWhole);
    const int n = static_cast<int>(__double_as_longlong(t));
    const double one = table[n & (kTable - 1)];
    const double q = f * fma(fma(fma(c4, f, c3), f, c2), f, c1);
    const uint64_t w = __double_as_longlong(fma(one, q, one)) + (static_cast<uint64_t>(static_cast<uint32_t>((n >> 7) + fraction) << 20) << 32);
    const uint64_t whole = __double_as_longlong(__longlong_as_double(w) + 0x1p52);
    return whole + (static_cast<uint64_t>((static_cast<uint32_t>(-n >> bin_shift) << 20) - 0x43300000u) << 32);
  }
  __device__ __forceinline__ int bin_formed(float l) const {
    return -static_cast<int>(__double_as_longlong(exponent(l) + 0x1.8p52)) >> bin_shift;
  }
  static __device__ __forceinline__ uint64_t units(uint64_t formed) { return formed & ((uint64_t{1} << 52) - 1); }
  static __device__ __forceinline__ int bin(uint64_t formed) { return static_cast<int>(formed >> 52); }
  __device__ __forceinline__ uint64_t operator()(float l) const { return units(formed(l)); }
  // the same, from the values
  template <bool VALUES>
  __device__ __forceinline__ uint64_t look(float l) const {
    if constexpr (!VALUES) return formed(l);
    const uint32_t bits = __float_as_uint(l) >> 16, at = (bits & 0x7fff) - base;
    uint64_t w = values[min(at, kValues - 1u) + (bits >> 15) * kValues];
    if (at >= kValues) w = l == -__builtin_inff() ? static_cast<uint64_t>(kSteps >> bin_shift) << 52 : formed(l);
    return w;
  }
  // An entry counted by value; f(l) for one of another magnitude.  Lanes that count one value wait for one another: 2048 x
  // 128000 with top_p take 318 us of spread logits, 2500 where half of them are zeros, 3060 of zeros alone (a row with more
  // than kOthers entries below the table's magnitudes is counted a second time).
  template <typename F>
  static __device__ __forceinline__ void count(uint32_t* counts, uint32_t from, float l, F f) {
    const uint32_t bits = __float_as_uint(l) >> 16, at = (bits & 0x7fff) - from;
    if (at < kValues) atomicAdd(&counts[at + (bits >> 15) * kValues], 1u);
    else if (l > -__builtin_inff()) f(l);
  }
  // zeros: the largest logit is 0, and so are most others.
  template <int THREADS>
  __device__ __forceinline__ void form_values(float row_top, bool zeros) {
    base = first_value(__float_as_uint(row_top) >> 23 & 0xffu, zeros);
    for (int i = threadIdx.x; i < 2 * kValues; i += THREADS) {
      const uint32_t bits = (base + (i < kValues ? i : i - kValues)) | (i < kValues ? 0 : 0x8000);
      const float l = __uint_as_float(bits << 16);
      values[i] = l <= row_top ? formed(l) : 0;
    }
    __syncthreads();
  }
  // ln of a logit's weight over a sum of weights
  __device__ __forceinline__ float log_share(float l, uint64_t total) const {
    return static_cast<float>((exponent(l) * (1.0 / kTable) - (log2(static_cast<double>(total)) - fraction)) * 0.69314718055994530942);
  }
};

// The smallest float that `holds` (it does for larger ones, and for +inf), next to a guess of it.
template <typename F>
__device__ __forceinline__ float smallest(float guess, F holds) {
  const int lane = threadIdx.x & 63;
  uint32_t lo = order_key(-__builtin_inff()), hi = order_key(__builtin_inff());   // keys: lo .. hi hold at hi
  uint32_t at = min(max(order_key(guess), lo + 32), hi - 32) - 32;
  uint32_t stride = 1;
  for (;;) {   // 64 keys at a time: around the guess, then over what is left
    const uint32_t key = min(at + lane * stride, hi);
    const uint64_t yes = __ballot(holds(of_key(key)));
    const int first = yes != 0 ? __builtin_ctzll(yes) : 64;
    if (first < 64) hi = min(hi, at + first * stride);
    if (first > 0) lo = max(lo, min(at + (first - 1) * stride, hi) + 1);
    if (lo >= hi) return of_key(hi);
    stride = max((hi - lo) / 63, 1u);
    at = lo;
  }
}

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
  // The runs that `mark` marks are read a second time for f, which the whole wavefront calls (with -inf in lanes
  // that have none left): few runs, so that the pass itself is a short loop.
  template <int U, typename M, typename F>
  __device__ __forceinline__ void marked(M mark, F f) const {
    const int64_t q0 = static_cast<int64_t>(threadIdx.x >> 6) * part * 64 + (threadIdx.x & 63);
    auto load = [&](Quad<DT> (&x)[U], int64_t n) {
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = load_quad<DT>(in, n + i < part ? q0 + (n + i) * 64 : quads, quads);
    };
    auto values = [](const Quad<DT>& x, float (&l)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) l[k] = x.at(k);
    };
    Quad<DT> x[U], next[U];
    load(x, 0);
    for (int64_t n0 = 0; n0 < part; n0 += 32) {
      uint32_t marks = 0;
#pragma unroll 1
      for (int n = 0; n < 32 && n0 + n < part; n += U) {
        load(next, n0 + n + U);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float l[4];
          values(x[i], l);
          marks |= mark(l) ? 1u << (n + i) : 0;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = next[i];
      }
      if (part - n0 < 32) marks &= (1u << (part - n0)) - 1;   // (behind the part -inf was read, which may be marked)
#pragma unroll 1
      while (__any(marks != 0)) {
        const int64_t q = marks != 0 ? q0 + (n0 + __builtin_ctz(marks)) * 64 : quads;
        const Quad<DT> y = load_quad<DT>(in, q, quads);
        float l[4];
        values(y, l);
        f(l, static_cast<uint32_t>(q) * 4);
        marks &= marks - 1;
      }
    }
  }
  // f(l[4], index of the first) in the order of the row (the workgroup's runs side by side): for the
  // pass from memory, which streams a row faster so than in a part for each wavefront.
  template <int U, typename F>
  __device__ __forceinline__ void stream(F f) const {
    Quad<DT> x[U], next[U];
    auto load = [&](Quad<DT> (&y)[U], int64_t q) {
#pragma unroll
      for (int i = 0; i < U; ++i) y[i] = load_quad<DT>(in, q + i * THREADS, quads);
    };
    load(x, threadIdx.x);
    for (int64_t q = threadIdx.x; q < quads; q += U * THREADS) {
      load(next, q + U * THREADS);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) l[k] = x[i].at(k);
        f(l, static_cast<uint32_t>(q + i * THREADS) * 4);
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

// What a workgroup of THREADS keeps in LDS: two of 512 fit a CU.  A list need
// not hold a whole row, in no workgroup (one of 256 takes rows of up to 8192
// entries, its list 5120): entries that do not fit are read from the row again.
template <int DT, int THREADS>
struct SampleShared {
  static constexpr bool kLooks = DT == ENGRAM_BF16 && THREADS > 256;   // weights of values
  static constexpr int kBinBits = THREADS <= 256 ? 9 : 11, kBins = 1 << kBinBits;
  static constexpr int kBinShift = THREADS <= 256 ? 4 : 2, kLastBin = kSteps >> kBinShift;
  static constexpr int kListed = THREADS <= 256 ? 5120 : kLooks ? 2560 : 6400;   // entries of the list
  uint64_t bins[kBins];
  uint64_t list[kListed];
  uint64_t values[kLooks ? 2 * kValues : 1];
  double table[kTable];
  uint64_t few[512];
  float queue[THREADS / 64][128];
  uint64_t wave[THREADS / 64], wave2[THREADS / 64];
  uint64_t part[THREADS / 64 + 1];
  uint64_t before;
  float red[THREADS / 64];
  int bin;
  int listed;
  int few_n;
};
static_assert(kSteps >> 2 < 2048 && kSteps >> 4 < 512, "every bin has its place");

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
template <int THREADS, typename Sh>
__device__ __forceinline__ void group_range(Sh& sh, uint64_t* lo, uint64_t* hi) {
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
template <int THREADS, typename Sh>
__device__ __forceinline__ void find_bin(Sh& sh, uint64_t before, uint64_t want) {
  constexpr int kEach = Sh::kBins / THREADS;
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

template <int THREADS, typename Sh>
__device__ __forceinline__ void clear_bins(Sh& sh) {
#pragma unroll
  for (int i = 0; i < Sh::kBins / THREADS; ++i) sh.bins[i * THREADS + threadIdx.x] = 0;
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
template <int THREADS, typename Sh, typename Entries, typename Amount>
__device__ __forceinline__ uint64_t find_place(Sh& sh, uint64_t lo, uint64_t hi, uint64_t before, uint64_t want,
                                               Entries entries, Amount amount) {
  for (;;) {
    const int shift = max(64 - __builtin_clzll((hi - lo) | 1) - Sh::kBinBits, 0);
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

// What a row's passes know of it.  The entries that stay are those up to a
// place of the order; min_p ends at one too.
template <int DT, int THREADS>
struct Draw {
  using Sh = SampleShared<DT, THREADS>;
  Sh& sh;
  Row<DT, THREADS> row;
  Weight weight;
  Place place;
  uint64_t cut;      // the last place that stays
  float lcut;        // its logit
  uint32_t vcut;     // its index

  __device__ __forceinline__ void set_cut(uint64_t c) {
    cut = c;
    lcut = c == ~uint64_t{0} ? -__builtin_inff() : place.logit(c);
    vcut = static_cast<uint32_t>(c);
  }
  __device__ __forceinline__ bool in(float l, uint32_t v) const { return l >= lcut && (l > lcut || v <= vcut); }
  // f(l, index, whether it is up to the cut) of the row's entries.  Equal logits
  // matter only in the run in which the cut's index lies: in those before it
  // entries equal to the cut's stay, in those behind it they do not.
  template <int U, bool CUT, typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (!CUT) {
      row.template each<U>([&](float l, uint32_t v) { f(l, v, true); });
    } else {
      const float above = lcut == __builtin_inff() ? lcut : of_key(order_key(lcut) + 1);
      row.template each_quad<U>([&](const float (&l)[4], uint32_t v) {
        const uint32_t v0 = __builtin_amdgcn_readfirstlane(v);   // 256 entries of a wavefront from here
        const float from = v0 + 255 <= vcut ? lcut : above;
        const bool mixed = v0 <= vcut && vcut < v0 + 255;
        if (!__any(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= lcut)) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) f(l[i], v + i, l[i] >= from || (mixed && in(l[i], v + i)));
      });
      if (row.vt < row.V) f(row.xt, static_cast<uint32_t>(row.vt), in(row.xt, static_cast<uint32_t>(row.vt)));
    }
  }
  __device__ __forceinline__ uint64_t look(float l) const { return weight.template look<Sh::kLooks>(l); }
  // What the weights have to reach for top_p, at least one unit: a negative top_p keeps the first entry, as 0 does (and a
  // negative number has no value as an unsigned one).
  __device__ __forceinline__ uint64_t share(float p, uint64_t all) const {
    return static_cast<uint64_t>(fmax(ceil(static_cast<double>(p) * static_cast<double>(all)), 1.0));
  }
  // Those of a run whose bit of `which` is set into the list from `at` on, which holds `most` of them; *n counts them.
  // One LDS atomic a wavefront and run.
  __device__ __forceinline__ void append(const float (&l)[4], uint32_t v, uint32_t which, int at, int most, int* n) const {
    if (!__any(which != 0)) return;
    const uint64_t below = (uint64_t{1} << (threadIdx.x & 63)) - 1;
    int mine = 0, all = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t b = __ballot(which >> k & 1);
      mine += __popcll(b & below);
      all += __popcll(b);
    }
    int first = 0;
    if ((threadIdx.x & 63) == 0) first = atomicAdd(n, all);
    mine += __builtin_amdgcn_readfirstlane(first);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (which >> k & 1) {
        if (mine < most) sh.list[at + mine] = place(l[k], v + k);
        ++mine;
      }
  }
  // All entries with a logit of `from` and more (any order) into the list; false: too many.
  __device__ __forceinline__ bool collect(float from, int* n) {
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    auto which = [&](float l, int k) { return l >= from && l > -__builtin_inff() ? 1u << k : 0u; };
    row.template marked<8>([&](const float (&l)[4]) { return fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= from; },
                           [&](const float (&l)[4], uint32_t v) {
      append(l, v, which(l[0], 0) | which(l[1], 1) | which(l[2], 2) | which(l[3], 3), 0, Sh::kListed, &sh.listed);
    });
    if (row.vt < row.V && which(row.xt, 0)) {
      const int at = atomicAdd(&sh.listed, 1);
      if (at < Sh::kListed) sh.list[at] = place(row.xt, static_cast<uint32_t>(row.vt));
    }
    __syncthreads();
    *n = sh.listed;
    return *n <= Sh::kListed;
  }
};

// f(place) of the list's entries up to a cut.
template <int THREADS, typename Sh>
struct Listed {
  const Sh& sh;
  int n;
  uint64_t cut;
  template <typename F>
  __device__ __forceinline__ void operator()(F f) const {
    for (int i = threadIdx.x; i < n; i += THREADS)
      if (sh.list[i] <= cut) f(sh.list[i]);
  }
};

// The cut of a row whose entries that stay are not few: SUM ? where the weights
// reach top_p of all up to the cut so far : where the first top_k end.  Bins
// over the weights; then the places in the one bin in which it ends, in the
// list (at most kListed of them), and, where SUM, in the same pass the sums of
// the weights in front of that bin (*sum, each wavefront's part; *tail, the
// entries behind the quads), to which those of the bin that stay are added in
// sh.part.  False: everything stays.  counted: the entries' values are counted
// already (in the list's place), those of other magnitudes in sh.few.
template <bool SUM, bool CUT, int DT, int THREADS>
__device__ __forceinline__ bool cut_row(Draw<DT, THREADS>& d, uint64_t k, float p, bool counted = false) {
  using Sh = SampleShared<DT, THREADS>;
  Sh& sh = d.sh;
  constexpr int kBins = Sh::kBins, kWaves = THREADS / 64;
  __syncthreads();
  clear_bins<THREADS>(sh);
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
  if constexpr (Sh::kLooks && !CUT) {
    // entries counted by value (half the LDS work of adding up their weights), the values binned afterwards
    uint32_t* counts = reinterpret_cast<uint32_t*>(sh.list);
    static_assert(sizeof(sh.list) >= 2 * kValues * 4, "the counts fit");
    auto other = [&](float l) {
      const uint64_t w = d.weight.formed(l);
      if (d.weight.bin(w) < Sh::kLastBin) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[d.weight.bin(w)]), SUM ? d.weight.units(w) : 1);
    };
    if (counted) {
      for (int i = threadIdx.x; i < sh.few_n; i += THREADS) other(reinterpret_cast<const float*>(sh.few)[i]);
    } else {
      for (int i = threadIdx.x; i < 2 * kValues; i += THREADS) counts[i] = 0;
      __syncthreads();
      const uint32_t base = d.weight.base;
      d.template each<4, CUT>([&](float l, uint32_t, bool) { Weight::count(counts, base, l, other); });
      __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * kValues; i += THREADS) {
      const uint64_t n = counts[i], w = sh.values[i];
      if (n > 0 && d.weight.bin(w) < Sh::kLastBin)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[d.weight.bin(w)]), SUM ? d.weight.units(w) * n : n);
    }
  } else {
    d.template each<2, CUT>([&](float l, uint32_t, bool in) {
      const uint64_t w = d.look(l);
      if (in && d.weight.bin(w) < Sh::kLastBin)   // (entries of weight 0 count for nothing)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[d.weight.bin(w)]), SUM ? d.weight.units(w) : 1);
    });
  }
  __syncthreads();
  uint64_t want = k;
  {
    uint64_t sum = 0, all;
#pragma unroll
    for (int i = 0; i < kBins / THREADS; ++i) sum += sh.bins[i * THREADS + threadIdx.x];
    group_scan<THREADS>(sum, sh.wave, &all);
    if constexpr (SUM) want = d.share(p, all);
    if (want >= all) return false;   // everything of any weight stays
  }
  find_bin<THREADS>(sh, 0, want);
  const int bin = sh.bin;
  const uint64_t before = sh.before;
  // the smallest logits of the bin and of the one before
  auto first_of = [&](int b) {
    return smallest(static_cast<float>(d.weight.top - (((b + 1) << Sh::kBinShift) - 0.5) / d.weight.a), [&](float l) { return l >= d.weight.top || d.weight.bin_formed(l) <= b; });
  };
  const float from = first_of(bin), front_from = bin > 0 ? first_of(bin - 1) : __builtin_inff();
  uint64_t lo = ~uint64_t{0}, hi = 0, sum = 0, tail = 0;
  // (the entries in front of the bin are queued, so that their weights are formed or looked up 64 at a time)
  float* queue = sh.queue[threadIdx.x >> 6];
  int queued = 0;
  auto take_queue = [&]() {   // 64 of them, or what is there
    const int lane = threadIdx.x & 63;
    wave_sync();
    const float l = queue[lane], later = queue[64 + lane];
    if (lane < queued) sum += d.weight.units(d.look(l));
    wave_sync();
    if (lane < queued - 64) queue[lane] = later;
    queued = max(queued - 64, 0);
    wave_sync();
  };
  auto in_bin = [&](float l, uint32_t v) { return l >= from && !(l >= front_from) && (!CUT || d.in(l, v)); };
  auto range = [&](uint64_t q) {
    lo = min(lo, q);
    hi = max(hi, q);
  };
  d.row.template marked<4>([&](const float (&l)[4]) {
    float x = -__builtin_inff();   // the largest behind those in front of the bin
    if (!SUM || !__any(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= front_from)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x = fmaxf(x, l[i] >= front_from ? x : l[i]);
    } else {   // (a cut before this one lies behind every entry in front of the bin)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool front = l[i] >= front_from;
        const uint64_t b = __ballot(front);
        if (front) queue[queued + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(b >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(b), 0))] = l[i];
        queued += __popcll(b);
        if (queued >= 64) take_queue();
        x = fmaxf(x, front ? x : l[i]);
      }
    }
    return x >= from;
  }, [&](const float (&l)[4], uint32_t v) {
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in_bin(l[i], v + i)) {
        which |= 1u << i;
        range(d.place(l[i], v + i));
      }
    d.append(l, v, which, 0, Sh::kListed, &sh.listed);
  });
  if (SUM && queued > 0) take_queue();
  if (d.row.vt < d.row.V) {
    const float l = d.row.xt;
    const uint32_t v = static_cast<uint32_t>(d.row.vt);
    if (in_bin(l, v)) {
      range(d.place(l, v));
      const int at = atomicAdd(&sh.listed, 1);
      if (at < Sh::kListed) sh.list[at] = d.place(l, v);
    }
    if (SUM && l >= front_from) tail = d.weight(l);
  }
  group_range<THREADS>(sh, &lo, &hi);   // (its barrier: the list is complete)
  const int listed = sh.listed;
  auto amount = [&](uint64_t at) { return SUM ? d.weight(d.place.logit(at)) : uint64_t{1}; };
  const bool fits = listed <= Sh::kListed;
  const Listed<THREADS, Sh> entries{sh, listed, ~uint64_t{0}};
  auto of_row = [&](auto f) {   // (many equal logits)
    d.row.template each<2>([&](float l, uint32_t v) {
      if (in_bin(l, v)) f(d.place(l, v));
    });
  };
  const uint64_t cut = fits ? find_place<THREADS>(sh, lo, hi, before, want, entries, amount) : find_place<THREADS>(sh, lo, hi, before, want, of_row, amount);
  if constexpr (SUM) {
    sum = wave_scan(sum);
    tail = wave_scan(tail);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh.part[threadIdx.x >> 6] = sum;
    if (threadIdx.x == 63) sh.part[kWaves] = tail;
    __syncthreads();
    auto add = [&](uint64_t q) {
      const uint32_t v = static_cast<uint32_t>(q);
      if (q <= cut) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.part[v < d.row.quads * 4 ? v / (static_cast<uint32_t>(d.row.part) * 256) : kWaves]), amount(q));
    };
    if (fits) entries(add);
    else of_row(add);
    __syncthreads();
  }
  d.set_cut(cut);
  return true;
}

// The n-th largest of the lanes' values (1 <= n <= 64).
__device__ __forceinline__ float wave_nth(float x, int n) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int size = 2; size <= 64; size *= 2) {
#pragma unroll
    for (int step = size / 2; step > 0; step /= 2) {
      const float other = __shfl_xor(x, step, 64);
      const bool up = (lane & size) == 0, lower = (lane & step) == 0;
      x = up == lower ? fmaxf(x, other) : fminf(x, other);   // descending
    }
  }
  return __shfl(x, n - 1, 64);
}

constexpr int kShort = 512;     // places of a list that one wavefront finishes
constexpr int kOthers = 1024;   // entries of a counted row that are no value of the table: sh.few holds so many floats

// The list's n <= kShort places in ascending order, into sh.few: a wavefront
// counts, for every kWaves-th place, those before it.  (What a workgroup runs
// once is fetched from the L2 as it goes, at some 5 cycles a byte: a sorting
// network over 256 places took 8000 cycles, this loop 2500.)
template <int THREADS, typename Sh>
__device__ __forceinline__ void order_list(Sh& sh, int n) {
  const int lane = threadIdx.x & 63;
  uint64_t x[kShort / 64];
#pragma unroll
  for (int i = 0; i < kShort / 64; ++i) x[i] = i * 64 + lane < n ? sh.list[i * 64 + lane] : ~uint64_t{0};
#pragma unroll 1
  for (int e = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); e < n; e += THREADS / 64) {
    const uint64_t p = sh.list[e];
    int before = 0;
#pragma unroll
    for (int i = 0; i < kShort / 64; ++i)
      if (i * 64 < n) before += __popcll(__ballot(x[i] < p));
    if (lane == 0) sh.few[before] = p;
  }
  __syncthreads();
}

// Bound by the vector instructions of the passes over a row, where there are many
// (the first pass from memory, the others from the L2: a row is fetched once).  2048 x
// 128000 bf16 takes 93 us greedy (memory: 5.6 TB/s), 272 without filters, 217 with
// top_k, 340 with top_p, in 7, 35, 17 and 37 instructions to 64 entries; at 4 cycles
// each the issue of 35 is 235 us, and LDS conflicts keep a CU's LDS busy for 35 to 40
// more.  Double precision is 1.1 of those 35 and 0.5 of the 37, since weights come
// from the table of values.  A row of 32001 float32 takes 9, 17, 21 and 25 us, a
// chain of passes by one workgroup, each weight formed in double.  (1024 threads
// have 128 registers: 53 spilled, 60 bytes a lane.)
template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 4)   // (four wavefronts a SIMD: two workgroups of 512 a CU)
sample_kernel(SampleArgs a) {
  using Sh = SampleShared<DT, THREADS>;
  __shared__ Sh sh;
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

  // this thread's largest, and the first run of four that holds it
  float own = -__builtin_inff();
  uint32_t own_v = 0;
  bool nan = row.xt != row.xt;
  auto seen = [&](const float (&l)[4], uint32_t v) {
    nan |= __builtin_isunordered(l[0], l[1]) | __builtin_isunordered(l[2], l[3]);
    const float x = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
    own_v = x > own ? v : own_v;
    own = fmaxf(own, x);
  };
  // runs in flight: 16 wavefronts have enough with 4 (256 x 128000 bf16 greedy 14.6 us, 16.5 with 8; no filters 45, 47)
  constexpr int kFirst = THREADS == 1024 ? 4 : 8;
  // a bf16 row that is going to be cut by top_p alone: its values are counted on the way
  bool counted = Sh::kLooks && p < 1.0f && temp > 0.f && !(top_k > 0 && top_k < V);
  if constexpr (Sh::kLooks) {
    if (counted) {
      uint32_t* counts = reinterpret_cast<uint32_t*>(sh.list);
      for (int i = threadIdx.x; i < 2 * kValues; i += THREADS) counts[i] = 0;
      if (threadIdx.x == 0) sh.few_n = 0;
      __syncthreads();
      auto other = [&](float l) {
        const int at = atomicAdd(&sh.few_n, 1);
        if (at < kOthers) reinterpret_cast<float*>(sh.few)[at] = l;
      };
      row.template stream<4>([&](const float (&l)[4], uint32_t v) {
        seen(l, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) Weight::count(counts, kFirstBase, l[i], other);
      });
      if (row.vt < V) Weight::count(counts, kFirstBase, row.xt, other);
    } else {
      row.template stream<kFirst>(seen);
    }
  } else {
    row.template stream<kFirst>(seen);
  }
  const float quads_own = own;
  own = fmaxf(own, row.xt);
  const float top = group_max<THREADS>(own, nan, sh.red);
  if (top != top || top == -__builtin_inff() || (top == __builtin_inff() && temp > 0.f)) {
    if (threadIdx.x == 0) {
      a.tokens[row_at] = -1;
      if (a.logprob != nullptr) a.logprob[row_at] = -__builtin_inff();
    }
    return;
  }
  auto at_index = [&](int64_t v) {
    if constexpr (DT == ENGRAM_BF16) return bf16_to_f32(static_cast<const uint16_t*>(row.in)[v]);
    else return static_cast<const float*>(row.in)[v];
  };
  if (!(temp > 0.f)) {
    if (threadIdx.x == 0) sh.bin = INT32_MAX;
    __syncthreads();
    if (quads_own == top) {
      while (at_index(own_v) != top) ++own_v;
      atomicMin(&sh.bin, static_cast<int>(own_v));
    } else if (own == top) {
      atomicMin(&sh.bin, static_cast<int>(row.vt));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      a.tokens[row_at] = sh.bin;
      if (a.logprob != nullptr) a.logprob[row_at] = 0.f;
    }
    return;
  }

  if (threadIdx.x < kTable) sh.table[threadIdx.x] = table_entry(threadIdx.x);   // (a barrier follows before its first use)
  constexpr double kLog2e = 1.4426950408889634074;
  Draw<DT, THREADS> d{sh, row, Weight{top, kTable * kLog2e / temp, a.fraction, Sh::kBinShift, sh.table, sh.values, 0u}, Place{order_key(top)},
                      ~uint64_t{0}, -__builtin_inff(), ~0u};
  const bool by_k = top_k > 0 && top_k < V, by_p = p < 1.0f, by_m = m > 0.f;
  const auto one = [](uint64_t) { return uint64_t{1}; };
  const auto weight_of = [&](uint64_t q) { return d.weight(d.place.logit(q)); };

  // Few entries stay (a small top_k): then a list holds them, and the rest is done on
  // the list.  Every wavefront has `each` lanes whose largest logits reach the
  // smallest of their `each`-th largest ones, so top_k entries reach it.  (top_k of 20 in a row of 32001: 14.2 us, 29.8
  // by bins; of 100 in 2048 rows of 128000: 206 and 384.)
  int listed = -1;
  constexpr int kWaves = THREADS / 64;
  if (by_k && top_k <= 32 * kWaves && V >= 4 * THREADS) {
    const int each = (top_k + kWaves - 1) / kWaves;
    const float nth = wave_nth(own, each);
    __syncthreads();
    if (lane == 0) sh.red[wave] = nth;
    __syncthreads();
    float from = sh.red[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) from = fminf(from, sh.red[w]);
    int n;
    if (d.collect(from, &n)) listed = n;
  }
  float least = -__builtin_inff();   // where min_p ends
  if (by_m) {
    __syncthreads();                 // the table
    const double y = kTable * log2(static_cast<double>(fminf(m, 1.0f)));
    least = smallest(static_cast<float>(top + y / d.weight.a), [&](float l) { return l >= top || d.weight.exponent(l) >= y; });
  }
  if (by_m && !by_k && !by_p) {      // few entries stay by min_p alone
    int n;
    if (d.collect(least, &n)) listed = n;
  }
  __syncthreads();                   // the table, the list
  auto wanted = [&](uint64_t total) {   // the token is the first whose running sum is above this
    return min(static_cast<uint64_t>(fmin(fmax(static_cast<double>(u), 0.0), 1.0) * static_cast<double>(total)), total - 1);
  };
  // the thread that finds the token keeps it for the end
  bool found_it = false;
  uint32_t token = 0;
  float logit = 0.f;
  uint64_t weights = 1;
  auto write = [&](uint32_t v, float l, uint64_t total) {
    found_it = true;
    token = v;
    logit = l;
    weights = total;
  };
  if (listed >= 0 && listed <= kShort) {   // one wavefront does it without a barrier, lane i the order's i-th, i + 64-th, ..
    order_list<THREADS>(sh, listed);
    if (wave == 0) {
      const int rounds = (listed + 63) / 64;
      auto round_place = [&](int i) { return i * 64 + lane < listed ? sh.few[i * 64 + lane] : ~uint64_t{0}; };
      uint64_t all = 0;
#pragma unroll 1
      for (int i = 0; i < rounds; ++i) {
        const int rank = i * 64 + lane;
        const uint64_t w = rank < listed && !(by_k && rank >= top_k) ? weight_of(sh.few[rank]) : 0;
        sh.list[rank] = w;
        all += at_lane(wave_scan(w), 63);
      }
      wave_sync();
      const uint64_t share = by_p ? d.share(p, all) : all;
      uint64_t sum = 0, total = 0;
      int stay = 0;   // they are the first of the order
#pragma unroll 1
      for (int i = 0; i < rounds; ++i) {
        const uint64_t w = sh.list[i * 64 + lane], upto = wave_scan(w);
        const bool stays = w > 0 && sum + upto - w < share && d.place.logit(round_place(i)) >= least;
        sum += at_lane(upto, 63);
        total += at_lane(wave_scan(stays ? w : uint64_t{0}), 63);
        stay += __popcll(__ballot(stays));
      }
      const uint64_t want = wanted(total);
      if (stay <= 64) {   // what lies in front of each by index, from the other lanes
        const uint64_t mine = round_place(0), own_w = lane < stay ? sh.list[lane] : 0;
        uint64_t before = 0;
#pragma unroll 1
        for (int j = 0; j < stay; ++j) {
          const uint64_t q = at_lane(mine, j), y = at_lane(own_w, j);
          before += static_cast<uint32_t>(q) < static_cast<uint32_t>(mine) ? y : 0;
        }
        if (own_w > 0 && before <= want && want < before + own_w) write(static_cast<uint32_t>(mine), d.place.logit(mine), total);
      } else {            // bit by bit: the first index up to which the weights pass `want`
        uint32_t found = 0;
#pragma unroll 1
        for (int b = 31 - __builtin_clz(static_cast<uint32_t>(V - 1) | 1); b >= 0; --b) {
          const uint32_t upto = found + (1u << b) - 1;
          uint64_t part = 0;
#pragma unroll 2
          for (int i = lane; i < stay; i += 64) part += static_cast<uint32_t>(sh.few[i]) <= upto ? sh.list[i] : 0;
          if (at_lane(wave_scan(part), 63) <= want) found += 1u << b;
        }
        for (int i = lane; i < stay; i += 64)
          if (static_cast<uint32_t>(sh.few[i]) == found) write(found, d.place.logit(sh.few[i]), total);
      }
    }
  } else if (listed >= 0) {   // a longer list
    if (by_k && listed > top_k) d.set_cut(find_place<THREADS>(sh, 0, ~uint64_t{0}, 0, top_k, Listed<THREADS, Sh>{sh, listed, ~uint64_t{0}}, one));
    if (by_p) {
      uint64_t sum = 0, all;
      Listed<THREADS, Sh>{sh, listed, d.cut}([&](uint64_t q) { sum += weight_of(q); });
      group_scan<THREADS>(sum, sh.wave, &all);
      d.set_cut(find_place<THREADS>(sh, 0, d.lcut > -__builtin_inff() ? d.place(d.lcut, ~0u) : ~uint64_t{0}, 0, d.share(p, all),
                                    Listed<THREADS, Sh>{sh, listed, d.cut}, weight_of));
    }
    if (least > d.lcut) d.set_cut(d.place(least, ~0u));
    const Listed<THREADS, Sh> entries{sh, listed, d.cut};
    uint64_t sum = 0, total;
    entries([&](uint64_t q) { sum += weight_of(q); });
    group_scan<THREADS>(sum, sh.wave, &total);
    // by index: the entry's place with its halves exchanged
    const uint64_t found = find_place<THREADS>(sh, 0, static_cast<uint64_t>(V) << 32 | ~0u, 0, wanted(total) + 1, [&](auto f) {
      entries([&](uint64_t q) { f(q << 32 | q >> 32); });
    }, [&](uint64_t q) { return weight_of(q << 32 | q >> 32); });
    if (threadIdx.x == 0) write(static_cast<uint32_t>(found >> 32), d.place.logit(found << 32), total);
  } else {
    // Sums of a wavefront's part of the row each, and of the entries behind the quads.
    if constexpr (Sh::kLooks) {
      // A row whose largest is 0 holds logits less their largest, or little but zeros, which are in the table of the
      // smallest magnitudes alone; its first entries tell (it is longer than THREADS).  2048 x 128000 without filters,
      // logits less their largest and zeros: 252 us and 430 by the table up to 128, 435 and 251 by the other.
      bool zeros = false;
      if (top == 0.f) zeros = 2 * __syncthreads_count(at_index(threadIdx.x) == 0.f) > THREADS;
      d.weight.template form_values<THREADS>(top, zeros);
    }
    bool summed = false;
    if (by_k) cut_row<false, false>(d, top_k, 0.f);
    counted = counted && d.weight.base == kFirstBase && sh.few_n <= kOthers;
    if (by_p) summed = d.cut == ~uint64_t{0} ? cut_row<true, false>(d, 0, p, counted) : cut_row<true, true>(d, 0, p);
    if (least > d.lcut) {
      d.set_cut(d.place(least, ~0u));
      summed = false;
    }
    if (!summed) {
      uint64_t sum = 0, tail = 0;
      auto add = [&](float l, uint32_t v, bool in) {
        const uint64_t w = d.weight.units(d.look(l));
        (v < row.quads * 4 ? sum : tail) += in ? w : 0;
      };
      constexpr int U = Sh::kLooks ? 4 : 2;
      if (d.cut == ~uint64_t{0}) d.template each<U, false>(add);
      else d.template each<U, true>(add);
      sum = wave_scan(sum);
      tail = wave_scan(tail);
      __syncthreads();
      if (lane == 63) sh.part[wave] = sum;
      if (threadIdx.x == 63) sh.part[kWaves] = tail;
      __syncthreads();
    }
    uint64_t total = 0;
#pragma unroll
    for (int w = 0; w <= kWaves; ++w) total += sh.part[w];
    const uint64_t want = wanted(total);
    uint64_t at = 0;
    int part = 0;
    while (at + sh.part[part] <= want) at += sh.part[part++];
    // that part again, by the whole workgroup, kRun runs a thread at a time
    constexpr int kRun = 2;
    if (part == kWaves) {
      const uint64_t w = row.vt < V && d.in(row.xt, static_cast<uint32_t>(row.vt)) ? d.weight(row.xt) : 0;
      uint64_t all;
      const uint64_t before = at + group_scan<THREADS>(w, sh.wave, &all);
      if (before <= want && want < before + w) write(static_cast<uint32_t>(row.vt), row.xt, total);
    } else {
      const int64_t q0 = part * row.part * 64, q1 = min(q0 + row.part * 64, row.quads);
      for (int64_t from = q0; from < q1; from += THREADS * kRun) {
        const int64_t q = from + threadIdx.x * kRun;
        Quad<DT> x[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) x[i] = load_quad<DT>(row.in, q + i, q1);
        uint64_t w[kRun * 4], mine = 0, all;
#pragma unroll
        for (int i = 0; i < kRun * 4; ++i) {
          const float l = x[i >> 2].at(i & 3);
          w[i] = d.in(l, static_cast<uint32_t>(q * 4 + i)) ? d.weight.units(d.look(l)) : 0;
          mine += w[i];
        }
        uint64_t sum = at + group_scan<THREADS>(mine, sh.wave, &all);
        if (sum <= want && want < sum + mine) {   // one thread's
#pragma unroll
          for (int i = 0; i < kRun * 4; ++i) {
            sum += w[i];
            if (!found_it && sum > want) write(static_cast<uint32_t>(q * 4 + i), x[i >> 2].at(i & 3), total);
          }
        }
        at += all;
        if (at > want) break;
      }
    }
  }
  if (found_it) {
    a.tokens[row_at] = static_cast<int32_t>(token);
    if (a.logprob != nullptr) a.logprob[row_at] = d.weight.log_share(logit, weights);
  }
}

// Rows of a launch: it has fewer than 2^32 work-items (launch_k).
constexpr int64_t kMostRows = 1 << 21;

template <int DT>
hipError_t launch_sample_dt(const SampleArgs& a, int64_t rows, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows));
  prof_stage("sample_tokens_kernel");
  // Threads: the passes over a row want many, the steps between them few, and several rows a CU hide each other's steps.
  // us for 256 / 512 / 1024 threads, no filters and top_p: 2048 x 8192 33 / 51 / 117 and 63 / 84 / 179, x 32001 bf16 101 / 92 / 152
  // and 169 / 142 / 244; 1 x 8192 7.6 / 9.6 / 14.3 and 17.4 / 17.3 / 21.8, x 32001 18.9 / 15.5 / 17.4 and 43 / 26 / 27; 256 x 65536
  // - / 27 / 27 and - / 54 / 50.  512 / 1024 threads at 128000 bf16 entries, no filters, top_p of 0.9 and top_k of 100: 256 rows
  // 51 / 44, 69 / 56 and 41 / 43; 320 rows 70 / 78, 88 / 105 and 54 / 70; 512 rows 77 / 83, 90 / 108 and 57 / 78; 1024 rows
  // 139 / 163, 169 / 213 and 105 / 148.
  if (a.V <= (rows > 256 ? 8192 : 4096)) launch_k((sample_kernel<DT, 256>), grid, dim3(256), 0, s, a);
  else if (a.V > 65536 && rows <= 256) launch_k((sample_kernel<DT, 1024>), grid, dim3(1024), 0, s, a);
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
