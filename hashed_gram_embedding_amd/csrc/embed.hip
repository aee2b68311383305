// Token embeddings beside the layer's own tables: the lookup with scaling that
// makes the first hidden states, and its gradient.
//
//   H[i][m][:] = scale E[id_i][:]                                  (m < M)
//   dE[v][:]   = scale sum_{i : id_i = v} sum_m dH[i][m][:]
//
// An id outside [0, V) (padding) has a row of zeros and no gradient.
#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "engram_internal.h"
#include "lanes_device.h"

namespace engram {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int64_t kL2Bytes = 32 << 20;   // 8 XCDs x 4 MiB

// A row's columns go to the lanes in chunks of 8: the lanes of a row are the
// power of two that covers its chunks, at most a workgroup; longer rows take
// more than one turn.
int row_lanes_log2(int64_t dim) {
  int log = 0;
  while ((1 << log) < kThreads && (int64_t{8} << log) < dim) ++log;
  return log;
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (DT == ENGRAM_BF16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), f);
  } else {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = a[k];
      f[k + 4] = b[k];
    }
  }
}

// PAST: lines that are not to stay in the L2.
template <int DT, bool PAST = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  auto store = [](auto v, auto* q) {
    if constexpr (PAST) __builtin_nontemporal_store(v, q);
    else *q = v;
  };
  if constexpr (DT == ENGRAM_BF16) {
    store(__builtin_bit_cast(u32x4_t, pack8(f)), reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i));
  } else {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i);
    store(f32x4_t{f[0], f[1], f[2], f[3]}, q);
    store(f32x4_t{f[4], f[5], f[6], f[7]}, q + 1);
  }
}

struct EmbedArgs {
  const int32_t* ids;
  const void* table;
  void* out;
  int64_t n;
  int64_t V;
  int64_t dim;
  int32_t branches;
  int32_t log_lanes;
  float scale;
};

// One row of the table is read once and written M times.  Bound by memory: 32763
// tokens x 4 x 1024 in bf16 43 us (6.8 TB/s) with outputs stored past the L2 (PAST),
// 51 through it; 256 x 1 x 1024 2.5 us, a launch and two loads in a chain, either way.
template <int IN, int OUT, bool PAST>
__global__ void __launch_bounds__(kThreads)
embed_kernel(EmbedArgs a) {
  const int lanes = 1 << a.log_lanes;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
  if (i >= a.n) return;
  const int64_t id = a.ids[i];
  const bool has = id >= 0 && id < a.V;
  for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < a.dim; c += lanes * 8) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (has) {
      load8<IN>(a.table, id * a.dim + c, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= a.scale;
    }
    for (int m = 0; m < a.branches; ++m) store8<OUT, PAST>(a.out, (i * a.branches + m) * a.dim + c, f);
  }
}

// ---- the gradient ----
// Tokens are sorted by id, equal ids by position, and the sums run over that
// order: whichever workgroup adds them, every sum has the same terms in the
// same order, so results are the same bits each time and no two workgroups
// add to one row.

// Zeros for the gradient's table, written by the workgroups behind a sorting
// launch's own: the sort is a chain of small launches, and the table is the
// larger part of what a call writes.
struct Fill {
  char* at;        // 16-byte aligned
  int64_t bytes;   // a multiple of 16
};
constexpr int64_t kFillBytes = 256;   // of one thread

__device__ __forceinline__ void fill_zeros(const Fill& f, int64_t group, int threads) {
  const int64_t end = min(f.bytes, (group + 1) * threads * kFillBytes);
  for (int64_t b = group * threads * kFillBytes + threadIdx.x * 16; b < end; b += threads * 16)
    *reinterpret_cast<u32x4_t*>(f.at + b) = u32x4_t{0, 0, 0, 0};
}

// What the sort orders: an id, V for one without a row.
__device__ __forceinline__ uint32_t key_of(int32_t id, uint32_t V) { return static_cast<uint32_t>(id) < V ? static_cast<uint32_t>(id) : V; }

// Few ids: each one's place is the number of ids before it in the order,
// counted over all of them.  16 ids a workgroup, so that few ids still fill the
// GPU; its other 64 lanes to an id take every 64th 4 of the ids, kRankAhead loads
// of 16 bytes in flight.  Bound by the comparisons, 3 instructions each.  (64
// ids a workgroup, the others read as scalars: 17.8 us at 4096 ids, 65 at 16384.)
constexpr int kRankThreads = 1024, kRankIds = 16, kRankParts = kRankThreads / kRankIds, kRankAhead = 8;
__global__ void __launch_bounds__(kRankThreads)
rank_kernel(const int32_t* __restrict__ ids, int n, uint32_t V, uint32_t* __restrict__ key_out, uint32_t* __restrict__ pos_out,
            int groups, Fill fill) {
  if (static_cast<int>(blockIdx.x) >= groups) return fill_zeros(fill, blockIdx.x - groups, kRankThreads);
  __shared__ int share[kRankThreads / 64][kRankIds];
  const int at = threadIdx.x % kRankIds, part = threadIdx.x / kRankIds;
  const int i = blockIdx.x * kRankIds + at, own = i & ~3;
  const uint32_t key = i < n ? key_of(ids[i], V) : 0;
  const int whole = n / 4;
  int before = 0;
  // equal ids count where they are in front; of i's own four only smaller ones do here
  auto four = [&](int j, u32x4_t x) {
    const uint32_t bound = key + (j < own ? 1 : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) before += min(x[k], V) < bound;
  };
  for (int c0 = part; c0 < whole; c0 += kRankParts * kRankAhead) {
    u32x4_t x[kRankAhead];
#pragma unroll
    for (int u = 0; u < kRankAhead; ++u) {
      const int c = min(c0 + u * kRankParts, whole - 1);
      __builtin_memcpy(&x[u], ids + c * 4, 16);   // (ids are aligned to 4 bytes)
    }
#pragma unroll
    for (int u = 0; u < kRankAhead; ++u)
      if (c0 + u * kRankParts < whole) four((c0 + u * kRankParts) * 4, x[u]);
  }
  before += __shfl_xor(before, 16, 64);
  before += __shfl_xor(before, 32, 64);
  if ((threadIdx.x & 63) < kRankIds) share[threadIdx.x / 64][at] = before;
  __syncthreads();
  if (threadIdx.x < kRankIds && i < n) {
    int rank = 0;
#pragma unroll
    for (int w = 0; w < kRankThreads / 64; ++w) rank += share[w][at];
    for (int j = whole * 4; j < n; ++j) rank += key_of(ids[j], V) < key;
    for (int j = own; j < i; ++j) rank += key_of(ids[j], V) == key;
    key_out[rank] = key;
    pos_out[rank] = i;
  }
}

// More ids: stable passes over digits of the key, lowest first.  A pass counts
// each block's digits, sums the counts (digit by digit, block by block) and
// moves every id to its place.
constexpr int kSortThreads = 256, kSortWaves = kSortThreads / 64;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits, kDigitsEach = kDigits / kSortThreads;
// ROUNDS * kSortThreads ids a workgroup: 4 rounds up to kShortSort ids (more
// workgroups), 16 above (fewer counts to sum).  A pass of 131072 ids takes 26 us
// with 4 and 23 with 16, one of 1048576 ids 160 and 60; 32768 ids take 13 with 4.
constexpr int64_t kShortSort = 1 << 16;

struct SortPass {
  const int32_t* ids;       // first pass: the caller's ids (pos is the index itself)
  const uint32_t* key;      // later passes
  const uint32_t* pos;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* counts;         // [kDigits][blocks]
  int64_t n;
  uint32_t V;
  int32_t shift;
  int32_t blocks;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& a, int64_t i) { return a.ids != nullptr ? key_of(a.ids[i], a.V) : a.key[i]; }

template <int ROUNDS>
__global__ void __launch_bounds__(kSortThreads)
digit_count_kernel(SortPass a, Fill fill) {
  if (static_cast<int>(blockIdx.x) >= a.blocks) return fill_zeros(fill, blockIdx.x - a.blocks, kSortThreads);
  __shared__ uint32_t hist[kDigits];
#pragma unroll
  for (int k = 0; k < kDigitsEach; ++k) hist[k * kSortThreads + threadIdx.x] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * ROUNDS * kSortThreads;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = i0 + r * kSortThreads + threadIdx.x;
    if (i < a.n) atomicAdd(&hist[(sort_key(a, i) >> a.shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kDigitsEach; ++k) {
    const int digit = k * kSortThreads + threadIdx.x;
    a.counts[static_cast<int64_t>(digit) * a.blocks + blockIdx.x] = hist[digit];
  }
}

__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t x) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const uint32_t y = __shfl_up(x, off, 64);
    x += lane >= off ? y : 0;
  }
  return x;
}

// Exclusive sums of the counts, in place: one workgroup, kScanRun counts a
// thread at a time (16384 counts 31 us read one after another, 12 so).
constexpr int kScanThreads = 1024, kScanRun = 16;
__global__ void __launch_bounds__(kScanThreads)
digit_scan_kernel(uint32_t* __restrict__ counts, int64_t m, Fill fill) {
  if (blockIdx.x > 0) return fill_zeros(fill, blockIdx.x - 1, kScanThreads);
  __shared__ uint32_t part[kScanThreads / 64];
  uint32_t carry = 0;
  for (int64_t from = 0; from < m; from += kScanThreads * kScanRun) {
    const int64_t i0 = from + threadIdx.x * kScanRun;
    u32x4_t x[kScanRun / 4];
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kScanRun / 4; ++i) x[i] = i0 + i * 4 < m ? *reinterpret_cast<const u32x4_t*>(counts + i0 + i * 4) : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kScanRun / 4; ++i) sum += x[i][0] + x[i][1] + x[i][2] + x[i][3];
    const uint32_t upto = wave_scan_u32(sum);
    __syncthreads();   // (the last turn's sums have been read)
    if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = upto;
    __syncthreads();
    uint32_t at = carry + upto - sum;
#pragma unroll
    for (int w = 0; w < kScanThreads / 64; ++w) {
      at += w < static_cast<int>(threadIdx.x >> 6) ? part[w] : 0;
      carry += part[w];
    }
#pragma unroll
    for (int i = 0; i < kScanRun / 4; ++i) {
      u32x4_t y;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = at;
        at += x[i][k];
      }
      if (i0 + i * 4 < m) *reinterpret_cast<u32x4_t*>(counts + i0 + i * 4) = y;
    }
  }
}

// Each wavefront takes a contiguous quarter of the block's ids, 64 at a time;
// lanes with the same digit find one another by a ballot for each digit bit.
template <int ROUNDS>
__global__ void __launch_bounds__(kSortThreads)
digit_move_kernel(SortPass a, Fill fill) {
  if (static_cast<int>(blockIdx.x) >= a.blocks) return fill_zeros(fill, blockIdx.x - a.blocks, kSortThreads);
  __shared__ uint32_t at[kSortWaves][kDigits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w)
#pragma unroll
    for (int k = 0; k < kDigitsEach; ++k) at[w][k * kSortThreads + threadIdx.x] = 0;
  __syncthreads();
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kSortWaves + wave) * ROUNDS * 64;
  uint32_t key[ROUNDS], pos[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = i0 + r * 64 + lane;
    key[r] = i < a.n ? sort_key(a, i) : 0;
    pos[r] = a.ids != nullptr || i >= a.n ? static_cast<uint32_t>(i) : a.pos[i];
    if (i < a.n) atomicAdd(&at[wave][(key[r] >> a.shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kDigitsEach; ++k) {   // where each wavefront's ids of each digit begin
    const int digit = k * kSortThreads + threadIdx.x;
    uint32_t from = a.counts[static_cast<int64_t>(digit) * a.blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t x = at[w][digit];
      at[w][digit] = from;
      from += x;
    }
  }
  __syncthreads();
  const uint64_t below = (uint64_t{1} << lane) - 1;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = i0 + r * 64 + lane;
    const uint32_t digit = (key[r] >> a.shift) & (kDigits - 1);
    uint64_t same = __ballot(i < a.n);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
      const uint64_t set = __ballot((digit >> b) & 1);
      same &= (digit >> b) & 1 ? set : ~set;
    }
    if (i < a.n) {
      const uint32_t to = at[wave][digit] + __popcll(same & below);
      a.key_out[to] = key[r];
      a.pos_out[to] = pos[r];
    }
    wave_sync();   // every lane has read its digit's place before the digit's last lane moves it on
    if (i < a.n && (same >> lane) == 1) at[wave][digit] += __popcll(same);
    wave_sync();
  }
}

struct SumArgs {
  const uint32_t* key;    // [n] sorted
  const uint32_t* pos;    // [n]
  const void* dout;       // [n][M][dim]
  void* dtable;           // [V][dim]
  float* part;            // [tiles][2][dim]
  int64_t n;
  int64_t dim;
  int64_t tiles;
  uint32_t V;
  int32_t branches;
  int32_t log_lanes;
  int32_t tile;           // sorted tokens of a tile
  int32_t accumulate;
  float scale;
};

template <int OUT>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, int64_t c, float (&sum)[8]) {
  const int64_t i = key * a.dim + c;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] *= a.scale;
  if (a.accumulate) {
    float old[8];
    load8<OUT>(a.dtable, i, old);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += old[k];
  }
  store8<OUT>(a.dtable, i, sum);
}

// Sums over tiles of the sorted tokens.  A run of equal ids inside a tile is
// written to its row; one that came in from the tile before, or goes on in
// the next, leaves its part sum (slot 0: came in, slot 1: begins here).  Bound
// by memory: kAhead rows of dout are in flight for every chunk of columns, and
// where they are more than the L2 holds they are read past it (PAST), so that
// the lines of the table's zeros, which the sorting launches have just written,
// need not make room for them: 32763 x 4 x 1024 bf16 68 us (4.6 TB/s), through the
// L2 112 (then one row at a time 148; 4 or 16 rows, tiles of 16 tokens or two
// buffers of rows 107-119, no different).  The 0.5 MB of 509 x 256 float32 take
// 5.9 us past the L2 and 4.8 through it.
constexpr int kAhead = 8;
constexpr int kLeastLanes = 2;   // log2: of a tile
template <int IN>
struct Chunk {   // 8 columns as stored
  u32x4_t x[IN == ENGRAM_BF16 ? 1 : 2];
  template <bool PAST>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p) + i * (IN == ENGRAM_BF16 ? 2 : 4));
    x[0] = PAST ? __builtin_nontemporal_load(q) : q[0];
    if constexpr (IN == ENGRAM_F32) x[1] = PAST ? __builtin_nontemporal_load(q + 1) : q[1];
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (IN == ENGRAM_BF16) return __uint_as_float(k & 1 ? x[0][k >> 1] & 0xffff0000u : x[0][k >> 1] << 16);
    else return __uint_as_float(x[k >> 2][k & 3]);
  }
};

template <int IN, int OUT, int TILE, bool PAST>
__global__ void __launch_bounds__(kThreads)
tile_sum_kernel(SumArgs a) {
  constexpr int kMost = (kThreads >> kLeastLanes) * TILE;   // sorted tokens of a workgroup
  __shared__ uint32_t keys[kMost + 2], pos[kMost];           // keys[0]: of the token before
  const int tiles = kThreads >> a.log_lanes, mine = threadIdx.x >> a.log_lanes;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * tiles * TILE;
  const int here = static_cast<int>(min(static_cast<int64_t>(tiles) * TILE, a.n - first));
  for (int i = threadIdx.x; i < here + 2; i += kThreads) {
    const int64_t p = first + i - 1;
    keys[i] = p >= 0 && p < a.n ? a.key[p] : ~0u;
    if (i < here) pos[i] = a.pos[first + i];
  }
  __syncthreads();
  const int p0 = mine * TILE, p1 = min(p0 + TILE, here);
  const int64_t c = ((static_cast<int64_t>(blockIdx.y) << a.log_lanes) + (threadIdx.x & ((1 << a.log_lanes) - 1))) * 8;
  if (p0 >= here || c >= a.dim) return;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * tiles + mine;
  int end = p1;   // ids without a row come last
  while (end > p0 && keys[end] >= a.V) --end;
  const int64_t step = a.branches * a.dim;
  const int items = (end - p0) * a.branches;   // (token, branch) pairs
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool begun = keys[p0] != keys[p0 + 1];       // the run begins in this tile
  int p = p0, m = 0;                           // of the next to be added
  int q = p0, b = 0;                           // of the next to be loaded
  for (int i0 = 0; i0 < items; i0 += kAhead) {
    Chunk<IN> x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      x[i].template load<PAST>(a.dout, pos[q] * step + b * a.dim + c);
      if (i0 + i + 1 < items && ++b == a.branches) {   // (behind the last one it is loaded again)
        b = 0;
        ++q;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= items) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += x[i].at(k);
      if (++m < a.branches) continue;
      m = 0;
      const uint32_t key = keys[p + 1];
      const bool ends = keys[p + 2] != key;
      if (ends || p + 1 == p1) {
        if (begun && ends) write_row<OUT>(a, key, c, sum);
        else store8<ENGRAM_F32>(a.part, (tile * 2 + (begun ? 1 : 0)) * a.dim + c, sum);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = 0.f;
        begun = true;
      }
      ++p;
    }
  }
}

// Runs over more than one tile: the tile in which one ends joins its parts,
// kJoinGroups of them side by side (each a contiguous share, joined in order).
constexpr int kJoinThreads = 256, kJoinLanes = 16, kJoinGroups = kJoinThreads / kJoinLanes;
template <int OUT>
__global__ void __launch_bounds__(kJoinThreads)
tile_join_kernel(SumArgs a) {
  __shared__ float share[kJoinGroups][kJoinLanes][9];
  __shared__ int back[kJoinThreads / 64];
  const int64_t t = static_cast<int64_t>(blockIdx.x) + 1;
  const int64_t p0 = t * a.tile, p1 = min(p0 + a.tile, a.n);
  const uint32_t key = a.key[p0];
  if (key >= a.V || a.key[p0 - 1] != key || (p1 < a.n && a.key[p1] == key && a.key[p1 - 1] == key)) return;
  // the tiles before this one that begin inside the run, kJoinThreads of them a turn
  int64_t begin = t;
  for (;;) {
    const int64_t u = begin - 1 - threadIdx.x;
    const uint64_t other = __ballot(u < 0 || a.key[u * a.tile] != key);
    if ((threadIdx.x & 63) == 0) back[threadIdx.x >> 6] = other != 0 ? __builtin_ctzll(other) : 64;
    __syncthreads();
    int n = 0;
    for (int w = 0; w < kJoinThreads / 64; ++w) {
      n += back[w];
      if (back[w] < 64) break;
    }
    __syncthreads();
    begin -= n;
    if (n < kJoinThreads) break;
  }
  const int64_t t0 = begin > 0 && a.key[begin * a.tile - 1] == key ? begin - 1 : begin;
  const int64_t parts = t - t0 + 1, per = (parts + kJoinGroups - 1) / kJoinGroups;
  const int lane = threadIdx.x % kJoinLanes, group = threadIdx.x / kJoinLanes;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * kJoinLanes + lane) * 8;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.dim) {
    const int64_t from = t0 + group * per, to = min(from + per, t + 1);
#pragma unroll 4
    for (int64_t q = from; q < to; ++q) {
      float f[8];
      load8<ENGRAM_F32>(a.part, (q * 2 + (q == t0 ? 1 : 0)) * a.dim + c, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += f[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) share[group][lane][k] = sum[k];
  __syncthreads();
  if (group != 0 || c >= a.dim) return;
  for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += share[g][lane][k];
  write_row<OUT>(a, key, c, sum);
}

// Ids up to this number take rank_kernel: 8192 ids 13.8 us against 13 a pass of
// the sort (two passes of a table of 32001 rows, three of 646400), 12288 25, 16384
// 43.
constexpr int64_t kMostRanked = 12288;

int64_t sort_blocks(int64_t n) {
  const int64_t block = kSortThreads * (n <= kShortSort ? 4 : 16);
  return (n + block - 1) / block;
}

int sort_passes(int64_t V) {   // digits that hold the keys 0..V
  int passes = 1;
  while (passes * kDigitBits < 32 && (V >> (passes * kDigitBits)) > 0) ++passes;
  return passes;
}

// Sorted tokens of a tile: long ones leave fewer part sums, short ones more
// tiles to fill the GPU.  At 16384 tokens x 4 x 1024 columns, where the rule
// changes, sums and joins take 45.6 us short and 44.4 long; at 8192 x 4 x 1024 26
// and 42, at 16384 x 4 x 64 14 and 34.
constexpr int kShortTile = 8, kLongTile = 32;
int tile_tokens(int64_t n, int64_t dim) { return n * ((dim + 7) / 8) <= int64_t{1} << 21 ? kShortTile : kLongTile; }

size_t up256(size_t x) { return (x + 255) & ~size_t{255}; }

struct GradSpace {
  uint32_t *key[2], *pos[2], *counts;
  float* part;
  size_t bytes;
};

GradSpace carve_grad(void* ws, int64_t n, int64_t dim) {
  GradSpace g{};
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char* p = ws == nullptr ? nullptr : static_cast<char*>(ws) + used;
    used += up256(bytes);
    return p;
  };
  const bool ranked = n <= kMostRanked;
  for (int i = 0; i < (ranked ? 1 : 2); ++i) {
    g.key[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
    g.pos[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
  }
  if (!ranked) g.counts = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(sort_blocks(n)) * kDigits * 4));
  const int64_t tile = tile_tokens(n, dim), tiles = (n + tile - 1) / tile;
  g.part = reinterpret_cast<float*>(take(static_cast<size_t>(tiles) * 2 * dim * 4));
  g.bytes = used;
  return g;
}

template <typename F>
hipError_t by_types(int in, int out, F f) {
  if (in == ENGRAM_BF16) return out == ENGRAM_BF16 ? f(std::integral_constant<int, ENGRAM_BF16>{}, std::integral_constant<int, ENGRAM_BF16>{})
                                                   : f(std::integral_constant<int, ENGRAM_BF16>{}, std::integral_constant<int, ENGRAM_F32>{});
  return out == ENGRAM_BF16 ? f(std::integral_constant<int, ENGRAM_F32>{}, std::integral_constant<int, ENGRAM_BF16>{})
                            : f(std::integral_constant<int, ENGRAM_F32>{}, std::integral_constant<int, ENGRAM_F32>{});
}

// The next share of the zeros: of what is left, one part in `launches`.
struct Zeros {
  char* at;
  int64_t bytes;
  int64_t given = 0;
  Fill next(int launches) {
    const int64_t left = bytes - given, share = launches <= 1 ? left : left / launches / 16 * 16;
    const Fill f{at + given, share};
    given += f.bytes;
    return f;
  }
};
unsigned fill_groups(const Fill& f, int threads) { return static_cast<unsigned>((f.bytes + threads * kFillBytes - 1) / (threads * kFillBytes)); }

__global__ void __launch_bounds__(kThreads)
fill_kernel(Fill fill) { fill_zeros(fill, blockIdx.x, kThreads); }

}  // namespace

hipError_t launch_embed(const int32_t* ids, int64_t n, const void* table, int dtype, int64_t V, int64_t dim, float scale,
                        int32_t branches, int out_dtype, void* out, hipStream_t s) {
  const int log_lanes = row_lanes_log2(dim);
  const int64_t per = kThreads >> log_lanes, most = (int64_t{1} << 23) * per;   // tokens of a launch (2^31 work-items)
  const int64_t row = branches * dim * (out_dtype == ENGRAM_BF16 ? 2 : 4);
  const bool past = n * row > kL2Bytes;   // the next kernel will not find them there anyway
  for (int64_t i = 0; i < n; i += most) {
    const int64_t m = std::min(most, n - i);
    const EmbedArgs a{ids + i, table, static_cast<char*>(out) + i * row, m, V, dim, branches, log_lanes, scale};
    const hipError_t e = by_types(dtype, out_dtype, [&](auto in, auto to) {
      launch_k(past ? embed_kernel<decltype(in)::value, decltype(to)::value, true> : embed_kernel<decltype(in)::value, decltype(to)::value, false>, dim3(static_cast<unsigned>((m + per - 1) / per)), dim3(kThreads), 0, s, a);
      return launch_error();
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t embed_backward_workspace(int64_t n, int64_t dim) { return carve_grad(nullptr, n, dim).bytes; }

hipError_t launch_embed_backward(const int32_t* ids, int64_t n, const void* dout, int dtype, int64_t V, int64_t dim, float scale,
                                 int32_t branches, bool accumulate, int out_dtype, void* dtable, void* ws, hipStream_t s) {
  Zeros zeros{static_cast<char*>(dtable), accumulate ? 0 : V * dim * (out_dtype == ENGRAM_BF16 ? 2 : 4)};
  hipError_t e;
  if (n == 0) {
    if (zeros.bytes == 0) return hipSuccess;
    const Fill f = zeros.next(1);
    prof_stage("fill_kernel");
    launch_k(fill_kernel, dim3(fill_groups(f, kThreads)), dim3(kThreads), 0, s, f);
    return launch_error();
  }
  const GradSpace g = carve_grad(ws, n, dim);
  int sorted = 0;
  if (n <= kMostRanked) {
    const Fill f = zeros.next(1);
    const int groups = static_cast<int>((n + kRankIds - 1) / kRankIds);
    prof_stage("rank_kernel");
    launch_k(rank_kernel, dim3(groups + fill_groups(f, kRankThreads)), dim3(kRankThreads), 0, s, ids, static_cast<int>(n), static_cast<uint32_t>(V),
             g.key[0], g.pos[0], groups, f);
    if ((e = launch_error()) != hipSuccess) return e;
  } else {
    const int passes = sort_passes(V);
    const int blocks = static_cast<int>(sort_blocks(n));
    int left = passes * 3;
    for (int p = 0; p < passes; ++p) {
      const int from = sorted, to = p == 0 ? 0 : 1 - sorted;
      const SortPass a{p == 0 ? ids : nullptr, g.key[from], g.pos[from], g.key[to], g.pos[to], g.counts, n, static_cast<uint32_t>(V),
                       p * kDigitBits, blocks};
      Fill f = zeros.next(left--);
      prof_stage("digit_count_kernel");
      launch_k(n <= kShortSort ? digit_count_kernel<4> : digit_count_kernel<16>, dim3(blocks + fill_groups(f, kSortThreads)), dim3(kSortThreads), 0, s, a, f);
      if ((e = launch_error()) != hipSuccess) return e;
      f = zeros.next(left--);
      prof_stage("digit_scan_kernel");
      launch_k(digit_scan_kernel, dim3(1 + fill_groups(f, kScanThreads)), dim3(kScanThreads), 0, s, g.counts, int64_t{blocks} * kDigits, f);
      if ((e = launch_error()) != hipSuccess) return e;
      f = zeros.next(left--);
      prof_stage("digit_move_kernel");
      launch_k(n <= kShortSort ? digit_move_kernel<4> : digit_move_kernel<16>, dim3(blocks + fill_groups(f, kSortThreads)), dim3(kSortThreads), 0, s, a, f);
      if ((e = launch_error()) != hipSuccess) return e;
      sorted = to;
    }
  }
  const int log_lanes = std::max(row_lanes_log2(dim), kLeastLanes), lanes = 1 << log_lanes;
  const int tile = tile_tokens(n, dim);
  const int64_t tiles = (n + tile - 1) / tile, per = kThreads / lanes;
  const SumArgs a{g.key[sorted], g.pos[sorted], dout, dtable, g.part, n, dim, tiles, static_cast<uint32_t>(V), branches, log_lanes, tile,
                  accumulate ? 1 : 0, scale};
  prof_stage("tile_sum_kernel");
  const bool past = n * branches * dim * (dtype == ENGRAM_BF16 ? 2 : 4) > kL2Bytes;
  e = by_types(dtype, out_dtype, [&](auto in, auto to) {
    constexpr int I = decltype(in)::value, O = decltype(to)::value;
    launch_k(tile == kShortTile ? (past ? tile_sum_kernel<I, O, kShortTile, true> : tile_sum_kernel<I, O, kShortTile, false>)
                                : (past ? tile_sum_kernel<I, O, kLongTile, true> : tile_sum_kernel<I, O, kLongTile, false>),
             dim3(static_cast<unsigned>((tiles + per - 1) / per), static_cast<unsigned>((dim + lanes * 8 - 1) / (lanes * 8))), dim3(kThreads), 0, s, a);
    return launch_error();
  });
  if (e != hipSuccess || tiles == 1) return e;
  prof_stage("tile_join_kernel");
  const dim3 grid(static_cast<unsigned>(tiles - 1), static_cast<unsigned>((dim + kJoinLanes * 8 - 1) / (kJoinLanes * 8)));
  if (out_dtype == ENGRAM_BF16) launch_k(tile_join_kernel<ENGRAM_BF16>, grid, dim3(kJoinThreads), 0, s, a);
  else launch_k(tile_join_kernel<ENGRAM_F32>, grid, dim3(kJoinThreads), 0, s, a);
  return launch_error();
}

}  // namespace engram
