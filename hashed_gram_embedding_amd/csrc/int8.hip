// 8-bit integer products (W8A8) beside the bf16 and MXFP8 ones of Step 5
// ("DeepSeek Engram series guide": k_t = W_K e_t, v_t = W_V e_t) and for the
// vocabulary product that follows the layers.
//
//   s_t = max_c |x_tc| / 127,  q_tc = rne(127 x_tc / max_c |x_tc|)
//   out_to = (sum_c q_tc w_oc) s_t s_o
//
// The sum is exact in int32 (|q|, |w| <= 128 and at most 131071 columns), so
// its order is free: the kernels permute and split the columns as it suits
// them and results do not depend on it.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device_util.h"
#include "engram_internal.h"
#include "hash_device.h"
#include "int8_device.h"

namespace engram {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at any output
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// ---- quantisation of rows (int8_device.h) ----

// Eight values of a row from any element on.
template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float* f) {
  if constexpr (DT == ENGRAM_BF16) {
    uint4 v;
    __builtin_memcpy(&v, static_cast<const uint16_t*>(x) + i, 16);
    unpack8(v, f);
  } else {
    __builtin_memcpy(f, static_cast<const float*>(x) + i, 32);
  }
}

template <int DT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if constexpr (DT == ENGRAM_BF16) return bf16_to_f32(static_cast<const uint16_t*>(x)[i]);
  else return static_cast<const float*>(x)[i];
}

// Where a row's codes go.  Plain rows keep their columns.  In the product's
// own layout (tail) the last, incomplete run of 16 columns lies right-aligned
// in its 16 bytes, zeros before it: the product reads W's last 16 columns
// there, and the zeros leave out those that the run before holds.
struct CodeRow {
  int8_t* dst;
  int whole, shift;
  __device__ __forceinline__ CodeRow(int8_t* row, int cols, bool tail)
      : dst(row), whole(cols / 16 * 16), shift(tail && cols % 16 != 0 ? 16 - cols % 16 : 0) {}
  __device__ __forceinline__ int8_t* at(int64_t c) const { return dst + (c < whole ? c : c + shift); }
};

// Rows of fewer than 512 N + 8 columns: one wavefront a row, runs of 8, every
// value read once, all loads in flight together; up to 7 columns behind the
// last run are the first lanes' own.  A row of zeros has scale 0, one holding
// an infinity or a NaN codes 0 and scale NaN.  Bound by memory: bf16 rows of
// 32768 x 1024 19.7 us (5.1 TB/s), 65536 x 4100 165 (4.9), float32 27.0 (6.2) and
// 254 (5.3); 4096 x 1024 bf16 4.5, one chain of loads and the launch.
template <int DT, int N>
__device__ __forceinline__ void quantize_rows(int64_t group, const void* __restrict__ x, int64_t rows, int cols, int8_t* __restrict__ q,
                                              int64_t ldq, int tail, float* __restrict__ scale) {
  const int64_t row = group * 4 + (threadIdx.x >> 6), base = row * cols;
  const int lane = threadIdx.x & 63, c8 = cols / 8 * 8, ct = c8 + lane;
  if (row >= rows) return;
  float f[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * 64 + lane) * 8;
    if (c < c8) {
      load8<DT>(x, base + c, f[n]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[n][k] = 0.f;
    }
  }
  const float ft = ct < cols ? load1<DT>(x, base + ct) : 0.f;
  uint32_t top = magnitude(ft);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, magnitude(f[n][k]));
  top = wave_top(top);
  if (lane == 0) scale[row] = row_scale(top);
  const bool codes = row_has_codes(top);
  const RowScale rs = row_factors(__uint_as_float(top));
  const CodeRow out(q + row * ldq, cols, tail != 0);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * 64 + lane) * 8;
    const u32x2_t w = codes ? quantize8(f[n], rs) : u32x2_t{0, 0};
    if (c < c8) __builtin_memcpy(out.at(c), &w, 8);
  }
  if (ct < cols) *out.at(ct) = static_cast<int8_t>(codes ? quantize(ft, rs) : 0);
  if (lane < out.shift) out.dst[out.whole + lane] = 0;
}

// Longer rows: one workgroup a row, which reads it twice (the second time
// from the L2, as far as the rows in work fit there: bf16 32768 x 8192 154 us
// (5.2 TB/s by one read), 8192 x 16384 97 (4.2), 8192 x 16387 118 (3.4: runs of 8
// at odd addresses), 4096 x 131071 621 (2.6)).
template <int DT>
__device__ __forceinline__ void quantize_long(int64_t row, const void* __restrict__ x, int cols, int8_t* __restrict__ q, int64_t ldq,
                                              int tail, float* __restrict__ scale) {
  __shared__ uint32_t part[4];
  const int t = threadIdx.x;
  const int64_t base = row * cols, c8 = cols / 8 * 8, ct = c8 + t;   // (rows up to 2^31 - 1 columns: no step past them in 32 bits)
  const float ft = ct < cols ? load1<DT>(x, base + ct) : 0.f;
  uint32_t top = magnitude(ft);
#pragma unroll 4
  for (int64_t c = t * 8; c < c8; c += 256 * 8) {
    float f[8];
    load8<DT>(x, base + c, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, magnitude(f[k]));
  }
  top = wave_top(top);
  if ((t & 63) == 0) part[t >> 6] = top;
  __syncthreads();
  top = max(max(part[0], part[1]), max(part[2], part[3]));
  if (t == 0) scale[row] = row_scale(top);
  const bool codes = row_has_codes(top);
  const RowScale rs = row_factors(__uint_as_float(top));
  const CodeRow out(q + row * ldq, cols, tail != 0);
#pragma unroll 4
  for (int64_t c = t * 8; c < c8; c += 256 * 8) {
    float f[8];
    load8<DT>(x, base + c, f);
    const u32x2_t w = codes ? quantize8(f, rs) : u32x2_t{0, 0};
    __builtin_memcpy(out.at(c), &w, 8);
  }
  if (ct < cols) *out.at(ct) = static_cast<int8_t>(codes ? quantize(ft, rs) : 0);
  if (t < out.shift) out.dst[out.whole + t] = 0;
}

// ---- product ----

struct ProjectI8Args {
  const int8_t* q;       // [n_tok][ldq]
  const float* q_scale;  // [n_tok]
  const int8_t* w;       // [n_out][K]
  const float* w_scale;  // [n_out]
  void* out;             // [n_tok][n_out]
  int64_t n_tok;
  int64_t ldq;
  int64_t n_out;
  int K;
  int tailed;            // q's last run of 16 columns is right-aligned and zero-filled
  // Step 5 of a layer with Step 6's sums instead of outputs (GATE forms): out
  // is v [n_tok][d] float32, n_out = (1 + M) d
  const uint16_t* H;     // [n_tok][M][d] bf16 (read only)
  float4* stats;         // [n_tok][nq]
  int d;
  int M;
  int nq;
  StateAdvance adv;      // ring form only
};

// Which bytes of a row's last 16 belong to its last chunk: all of them, or
// the K % 16 behind the ones that the chunk before holds.
__device__ __forceinline__ u32x4_t tail_mask(int K) {
  const int twice = (16 - K % 16) % 16;
  u32x4_t m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(max(twice - 4 * i, 0), 4);
    m[i] = n == 4 ? 0u : 0xffffffffu << (8 * n);
  }
  return m;
}

// Chunk c (16 columns) of a row of K >= 16 codes at any alignment; the last
// one right-aligned, zeros before it.
__device__ __forceinline__ u32x4_t load_chunk(const int8_t* row, int c, int K) {
  u32x4_t v;
  __builtin_memcpy(&v, row + min(c * 16, K - 16), 16);
  return c * 16 + 16 > K ? v & tail_mask(K) : v;
}

// Rows whose length is no multiple of 16 into the product's own layout: whole
// aligned chunks, the last one right-aligned behind zeros.  A thread takes
// kAlignItems chunks, 256 apart.  A load from an address that is no multiple of
// 4 takes the memory pipeline several times as long, so the 5 words around such
// a chunk are read and shifted into place, except at the array's two ends.
// (Reading odd rows into the tiles through registers instead took 46 us at
// 2000 x 4099 x 2000, where the copy and the product take 38, and 94 against 87
// at 1795 x 1001 x 32000; at 76 x 2823 x 70852, where the copy moves more than
// the product, 113 against 149.)
constexpr int kAlignItems = 4;

struct AlignJob {
  const int8_t* x;   // [rows][K]
  u32x4_t* y;        // [rows][chunks]
  int64_t rows;
  int64_t groups;    // workgroups: rows * chunks / (256 kAlignItems), rounded up
};

__device__ __forceinline__ void align_rows(const AlignJob& j, int64_t group, int K, int chunks) {
  const int64_t n = j.rows * chunks, base = group * 256 * kAlignItems;
  const int64_t row0 = base / chunks, id0 = base + threadIdx.x;
  const uint32_t c0 = static_cast<uint32_t>(base - row0 * chunks) + threadIdx.x, width = static_cast<uint32_t>(chunks);
  const int8_t* const end = j.x + j.rows * K;
  u32x4_t v[kAlignItems];
  uint32_t behind[kAlignItems];
  int past[kAlignItems];
  int keep[kAlignItems];   // of the chunk: all, its last K % 16, nothing
#pragma unroll
  for (int i = 0; i < kAlignItems; ++i) {
    const bool in = id0 + i * 256 < n;
    const uint32_t down = (c0 + i * 256) / width;
    const int64_t r = in ? row0 + down : 0;
    const int c = in ? static_cast<int>(c0 + i * 256 - down * width) : 0;
    const int8_t* p = j.x + r * K + min(c * 16, K - 16);
    past[i] = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
    if (p - past[i] < j.x || p - past[i] + 20 > end) past[i] = 0;
    keep[i] = c * 16 + 16 <= K ? 2 : c * 16 < K ? 1 : 0;
    p -= past[i];
    __builtin_memcpy(&v[i], p, 16);
    __builtin_memcpy(&behind[i], past[i] != 0 ? p + 16 : p, 4);
  }
#pragma unroll
  for (int i = 0; i < kAlignItems; ++i) {
    const uint32_t by = static_cast<uint32_t>(past[i]);
    const u32x4_t x{__builtin_amdgcn_alignbyte(v[i][1], v[i][0], by), __builtin_amdgcn_alignbyte(v[i][2], v[i][1], by),
                    __builtin_amdgcn_alignbyte(v[i][3], v[i][2], by), __builtin_amdgcn_alignbyte(behind[i], v[i][3], by)};
    const u32x4_t none{0, 0, 0, 0};
    if (id0 + i * 256 < n) j.y[id0 + i * 256] = keep[i] == 2 ? x : keep[i] == 1 ? x & tail_mask(K) : none;
  }
}

__global__ void __launch_bounds__(256)
align_rows_kernel(AlignJob a, AlignJob b, int K, int chunks) {
  const bool first = blockIdx.x < a.groups;
  align_rows(first ? a : b, blockIdx.x - (first ? 0 : a.groups), K, chunks);
}

// Rows to codes, one wavefront a row (N > 0) or one workgroup (N = 0).  ALIGN:
// the first workgroups copy W's odd rows, which nothing here reads, so the
// product waits for one launch instead of two (55 x 2271 x 1676 18.0 -> 15.6 us, 2000 x
// 4099 x 2000 44.6 -> 41.0).
struct QuantizeArgs {
  const void* x;
  int64_t rows;
  int8_t* q;
  int64_t ldq;
  float* scale;
  int cols;
  int tail;
};

template <int DT, int N, bool ALIGN>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(QuantizeArgs a, AlignJob w, int chunks) {
  int64_t group = blockIdx.x;
  if constexpr (ALIGN) {
    if (group < w.groups) {
      align_rows(w, group, a.cols, chunks);
      return;
    }
    group -= w.groups;
  }
  if constexpr (N > 0) quantize_rows<DT, N>(group, a.x, a.rows, a.cols, a.q, a.ldq, a.tail, a.scale);
  else quantize_long<DT>(group, a.x, a.cols, a.q, a.ldq, a.tail, a.scale);
}

template <typename OutT>
__device__ __forceinline__ OutT to_out(float f) {
  if constexpr (sizeof(OutT) == 2) return f32_to_bf16(f);
  else return f;
}

// Sum over the 16 lanes of a DPP row, in all of them (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row_sum(float x) {
  auto turned = [](float v, auto by) {
    constexpr int kRowRor = 0x120;
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), kRowRor + decltype(by)::value, 0xf, 0xf, false));
  };
  x += turned(x, std::integral_constant<int, 8>{});
  x += turned(x, std::integral_constant<int, 4>{});
  x += turned(x, std::integral_constant<int, 2>{});
  x += turned(x, std::integral_constant<int, 1>{});
  return x;
}

// What four columns of a projection row add to a token's gate sums (h.h, k.k,
// h.k, v.v): value columns their squares, key columns those of h and k.
__device__ __forceinline__ float4 gate_terms(const f32x4_t& x, bool is_v, uint2 h) {
  const float xx = x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
  if (is_v) return make_float4(0.f, 0.f, 0.f, xx);
  const float h0 = __uint_as_float(h.x << 16), h1 = __uint_as_float(h.x & 0xffff0000u);
  const float h2 = __uint_as_float(h.y << 16), h3 = __uint_as_float(h.y & 0xffff0000u);
  return make_float4(h0 * h0 + h1 * h1 + h2 * h2 + h3 * h3, xx, h0 * x[0] + h1 * x[1] + h2 * x[2] + h3 * x[3], 0.f);
}

__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Tiled product for the sizes that fill the chip.  A workgroup of WF x WT
// wavefronts forms TF outputs x TT tokens; W rows are the A operand of
// v_mfma_i32_32x32x32_i8 and token rows the B operand, so a lane ends with
// runs of four consecutive outputs of one token.  Columns come in slices of
// 128 through two LDS buffers: while one is multiplied the next is in flight.
// Chunk c (16 bytes) of a slice's row r lies at c ^ ((r >> 1) & 7), so that
// the operand reads of 16 lanes (16 rows, one chunk) spread over all banks.
//
// Workgroups are persistent: each walks its share of the tiles, and the first
// slice of the next tile is on its way while the last one of this tile is
// multiplied and its outputs are scaled and stored.  (One workgroup per tile
// left the matrix cores idle at both ends of every tile: with 1024 columns a
// tile has 8 slices, and 32763 x 1024 x 5120 took 227 us instead of 195.)
// Tiles go to the XCDs in contiguous shares of an order that walks bands of
// kBand token tiles, tokens fastest: the 32 tiles that an XCD works on at one
// time span 8 x 4, so both operands are re-read from its L2 (tokens fastest
// over all of them, 128 x 1/4 at that size: 218 us, outputs fastest, 20 x
// 1.6: 202, bands: 185).  Outputs of the large tiles are stored past the L2
// (nontemporal): written through it they drive the operands out, 300 -> 265
// us at 1795 x 1024 x 128000.
//
// Slices go from memory straight into LDS, so both operands are 16-byte
// aligned rows of whole chunks.
//
// GATE: Step 5 of a layer.  Value columns are stored, and instead of the keys
// the sums that Step 6 takes of them and of h leave the kernel, one float4 per
// token and run of 64 x (2 or 4) columns, so that the keys' float32 rows are
// neither written nor read again (4096 tokens, one branch: 25.3 us for the
// product and the sums apart, 18.1 together; 8192 tokens, 4 branches, with the
// conv 148 against 116).  These forms spill 52 (256 x 256) and 36 bytes a lane
// around the epilogue.
constexpr int kBand = 8;

template <typename OutT, int TF, int TT, int WF, int WT, bool GATE>
__global__ void __launch_bounds__(64 * WF * WT) __attribute__((amdgpu_waves_per_eu(2, 2)))
project_i8_tile_kernel(ProjectI8Args a, int tiles_f, int tiles_t) {
  constexpr int NT = 64 * WF * WT;
  constexpr int I = TF / WF / 32, J = TT / WT / 32;   // 32 x 32 blocks of a wavefront
  constexpr int WC = TF * 8, QC = TT * 8;             // chunks of a slice
  constexpr int NW = WC / NT, NQ = QC / NT;           // chunks a thread loads
  constexpr int RC = TF / WF * static_cast<int>(sizeof(OutT)) / 16;   // chunks of a wavefront's output row
  static_assert(RC >= 8 && (RC & (RC - 1)) == 0 && WF * WT * 32 * RC <= WC + QC, "outputs turn around in one buffer");
  static_assert((TF + TT) % NT == 0 || NT % (TF + TT) == 0, "scales per thread");
  extern __shared__ u32x4_t lds[];
  float* const sc = reinterpret_cast<float*>(lds + 2 * (WC + QC));   // [2][TF + TT] scales: outputs, then tokens
  float4* const red = reinterpret_cast<float4*>(sc + 2 * (TF + TT));  // GATE: [WF][TT] sums of the wavefronts' columns

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wf = wave % WF, wt = wave / WF, lr = lane & 31, lh = lane >> 5;
  const int K = a.K, chunks = K / 16, ksteps = (chunks + 7) / 8;
  const int n_tiles = tiles_f * tiles_t, share = (n_tiles + 7) / 8;
  const int xcd = blockIdx.x & 7, stride = gridDim.x >> 3;

  // whole 128-byte lines of the output leave past the L2; pieces of lines are
  // put together there
  const bool stream = a.n_out * static_cast<int64_t>(sizeof(OutT)) % 128 == 0 && reinterpret_cast<uintptr_t>(a.out) % 128 == 0;

  struct Tile {
    int64_t f0, t0;
  };
  // Round n of an XCD's share is `stride` tiles; a workgroup's place in it
  // moves by one each round, so that no workgroup gets a band's ragged last
  // tile (or a whole one) every time.
  auto tile_of = [&](int round, Tile* t) {
    const int local = round * stride + (static_cast<int>(blockIdx.x >> 3) + round) % stride;
    const int id = xcd * share + local;
    if (local >= share || id >= n_tiles) return false;
    const int band = id / (kBand * tiles_f), b0 = band * kBand, rows = min(kBand, tiles_t - b0);
    const int in = id - band * kBand * tiles_f;
    t->t0 = static_cast<int64_t>(b0 + in % rows) * TT;
    t->f0 = static_cast<int64_t>(in / rows) * TF;
    return true;
  };

  // This thread's chunk of a slice: row r0 (and every NT / 8 rows from there),
  // source chunk ch, into LDS slot tid.  The rows of one thread are 16 n
  // apart, so one source chunk serves all of them.
  static_assert(NT / 8 % 16 == 0, "the swizzle repeats every 16 rows");
  const int r0 = tid >> 3, ch = (tid & 7) ^ ((r0 >> 1) & 7);
  const int ldq = static_cast<int>(a.ldq);

  // Rows past the operand's end and chunks past the last one are out of the
  // buffer's range and read as zeros (a W chunk past the row's end may read
  // the next row instead: the tokens' zeros leave it out).
  auto issue = [&](const Tile& t, int kt, int buf) {
    const int w_bytes = static_cast<int>(min(static_cast<int64_t>(TF), a.n_out - t.f0)) * K;
    const int q_bytes = static_cast<int>(min(static_cast<int64_t>(TT), a.n_tok - t.t0)) * ldq;
    const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.w + t.f0 * K), 0, w_bytes, 0x00020000);
    const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q + t.t0 * ldq), 0, q_bytes, 0x00020000);
    u32x4_t* dst = lds + buf * (WC + QC) + wave * 64;
    const bool in = kt * 8 + ch < chunks;
    const int wo = r0 * K + ch * 16, qo = in ? r0 * ldq + ch * 16 : 0x7fff0000;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (__attribute__((address_space(3))) void*)(dst + i * NT), 16,
                                               wo + i * (NT / 8) * K, kt * 128, 0, 0);
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (__attribute__((address_space(3))) void*)(dst + WC + i * NT), 16,
                                               in ? qo + i * (NT / 8) * ldq : qo, kt * 128, 0, 0);
  };
  auto scales = [&](const Tile& t, int par) {
#pragma unroll
    for (int b = 0; b < (TF + TT) / 64; b += WF * WT) {
      const int seg = b + wave;   // 64 scales per wavefront instruction
      if (seg < (TF + TT) / 64) {
        const int r = seg * 64 + lane;
        const float* src = seg < TF / 64 ? a.w_scale + min(t.f0 + r, a.n_out - 1) : a.q_scale + min(t.t0 + (r - TF), a.n_tok - 1);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                         (__attribute__((address_space(3))) void*)(sc + par * (TF + TT) + seg * 64), 4, 0, 0);
      }
    }
  };

  Tile cur, next{0, 0};
  int round = 0;
  const int rounds = (share + stride - 1) / stride;
  while (round < rounds && !tile_of(round, &cur)) ++round;   // a last round may leave a place empty
  if (round >= rounds) return;
  int buf = 0, par = 0;
  scales(cur, 0);
  issue(cur, 0, 0);
  // One tile; `whole`: every block of this wavefront holds tokens.  (Two
  // copies of the loop rather than a choice inside it, between whose sides the
  // accumulators would have to move.)
  bool more = false;
  int jn = J;   // blocks of 32 tokens that this wavefront has in the tile
  auto process = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    i32x16_t acc[I][J];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    i32x4_t fa[2][I], fb[2][J];   // operands of two steps of 32 columns
    auto multiply = [&](int set) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
    };
    for (int kt = 0; kt < ksteps; ++kt) {
      // this lane's part of the slice has landed and its reads of the other
      // buffer are done; after the barrier, every lane's
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (kt + 1 < ksteps) {
        issue(cur, kt + 1, buf ^ 1);
      } else if (more) {
        issue(next, 0, buf ^ 1);
        scales(next, par ^ 1);
      }
      const u32x4_t* Ws = lds + buf * (WC + QC);
      const u32x4_t* Qs = Ws + WC;
      auto operands = [&](int set, int ks) {
        const int kc = (ks * 2 + lh) ^ ((lr >> 1) & 7);
#pragma unroll
        for (int i = 0; i < I; ++i) fa[set][i] = __builtin_bit_cast(i32x4_t, Ws[(wf * (TF / WF) + i * 32 + lr) * 8 + kc]);
#pragma unroll
        for (int j = 0; j < J; ++j) fb[set][j] = __builtin_bit_cast(i32x4_t, Qs[(wt * (TT / WT) + j * 32 + lr) * 8 + kc]);
      };
      if constexpr (kWhole) {
        // The operands of step ks + 1 are read while step ks multiplies, one
        // LDS read behind each of the first products; those of a slice's first
        // step while the last step of the slice before multiplies, which so
        // waits behind the barrier (32763 x 1024 x 5120 191 -> 183 us, 32763 x 128 x
        // 5120 82 -> 77).
        operands(0, 0);
        if (kt > 0) multiply(1);
#pragma unroll
        for (int ks = 0; ks < 3; ++ks) {
          operands((ks + 1) & 1, ks + 1);
          multiply(ks & 1);
        }
        if constexpr (I * J >= I + J) {
          constexpr int kMfma = 0x8, kLdsRead = 0x100;
#pragma unroll
          for (int ks = 0; ks < 3; ++ks) {
#pragma unroll
            for (int z = 0; z < I + J; ++z) {
              __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
              __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
            }
            if constexpr (I * J > I + J) __builtin_amdgcn_sched_group_barrier(kMfma, I * J - I - J, 0);
          }
        }
      } else {   // only the blocks that hold tokens
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          operands(0, ks);
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (j < jn)
#pragma unroll
              for (int i = 0; i < I; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[0][i], fb[0][j], acc[i][j], 0, 0, 0);
        }
      }
      buf ^= 1;
    }
    // Outputs: every wavefront turns a block of 32 tokens around in its part
    // of the buffer that was multiplied last, so that it stores runs of
    // TF / WF outputs of one token.  acc[i][j][4g + e] is output 32i + 8g +
    // 4 lh + e of token 32j + lr.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the buffer's last reads are done
    if constexpr (kWhole) multiply(1);
    u32x4_t* E = lds + (buf ^ 1) * (WC + QC) + wave * 32 * RC;
    const float* sw = sc + par * (TF + TT) + wf * (TF / WF);
    const float* sq = sc + par * (TF + TT) + TF + wt * (TT / WT);
    constexpr int EPC = 16 / static_cast<int>(sizeof(OutT));   // outputs of a chunk
    const int64_t fw = cur.f0 + wf * (TF / WF);
    // every output of the wavefront is one of the product's: its first chunk
    // of each block, rows apart by a stride that all lanes share
    const bool inside = !GATE && fw + TF / WF <= a.n_out && cur.t0 + (wt + 1) * (TT / WT) <= a.n_tok;
    OutT* const first = static_cast<OutT*>(a.out) + (cur.t0 + wt * (TT / WT) + lane / RC) * a.n_out + fw + lane % RC * EPC;
    // GATE: this wavefront's columns are v's, or one branch's keys
    const bool is_v = GATE && fw < a.d;
    const int branch = GATE && !is_v ? static_cast<int>(fw / a.d) - 1 : 0;
    const int64_t col = GATE ? fw - static_cast<int64_t>(is_v ? 0 : 1 + branch) * a.d : 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!kWhole && j >= jn) break;
      uint2 h[GATE ? 32 * RC / 64 : 1];
      if constexpr (GATE) {
#pragma unroll
        for (int it = 0; it < 32 * RC / 64; ++it) {
          h[it] = make_uint2(0u, 0u);
          const int rr = (it * 64 + lane) / RC, c = (it * 64 + lane) % RC;
          const int64_t tok = min(cur.t0 + wt * (TT / WT) + j * 32 + rr, a.n_tok - 1);
          if (!is_v && fw < a.n_out) h[it] = *reinterpret_cast<const uint2*>(a.H + (tok * a.M + branch) * a.d + col + c * 4);
        }
      }
      const float st = sq[j * 32 + lr];
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4_t s4 = *reinterpret_cast<const f32x4_t*>(sw + i * 32 + g * 8 + lh * 4);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(acc[i][j][4 * g + e]) * st * s4[e];
          if constexpr (sizeof(OutT) == 2)
            reinterpret_cast<u32x2_t*>(E + lr * RC + ((i * 4 + g) ^ (lr & 7)))[lh] = u32x2_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
          else
            E[lr * RC + ((i * 8 + g * 2 + lh) ^ (lr & 7))] = __builtin_bit_cast(u32x4_t, f32x4_t{x[0], x[1], x[2], x[3]});
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wavefront's block is in LDS
      constexpr int NIT = 32 * RC / 64;
      u32x4_t v[NIT];
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        const int rr = (it * 64 + lane) / RC, c = (it * 64 + lane) % RC;
        v[it] = E[rr * RC + (c ^ (rr & 7))];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // and read, before the next block's writes
      if constexpr (!GATE) {
        if (inside) {
#pragma unroll
          for (int it = 0; it < NIT; ++it) {
            OutT* dst = first + (j * 32 + it * (64 / RC)) * a.n_out;
            if (TF * TT >= 65536 && stream)
              __builtin_nontemporal_store(v[it], reinterpret_cast<u32x4_any_t*>(dst));
            else
              __builtin_memcpy(dst, &v[it], 16);
          }
          continue;
        }
      }
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        const int rr = (it * 64 + lane) / RC, c = (it * 64 + lane) % RC;
        const int64_t tok = cur.t0 + wt * (TT / WT) + j * 32 + rr, o = fw + c * EPC;
        if constexpr (GATE) {
          const f32x4_t x = __builtin_bit_cast(f32x4_t, v[it]);
          if (is_v && tok < a.n_tok) __builtin_memcpy(static_cast<float*>(a.out) + tok * a.d + o, &x, 16);
          float4 p = gate_terms(x, is_v, h[it]);
          p = make_float4(row_sum(p.x), row_sum(p.y), row_sum(p.z), row_sum(p.w));
          if (c == 0) red[wf * TT + wt * (TT / WT) + j * 32 + rr] = p;
        } else if (tok < a.n_tok && o < a.n_out) {
          OutT* dst = static_cast<OutT*>(a.out) + tok * a.n_out + o;
          if (o + EPC <= a.n_out) {
            if (TF * TT >= 65536 && stream)
              __builtin_nontemporal_store(v[it], reinterpret_cast<u32x4_any_t*>(dst));
            else
              __builtin_memcpy(dst, &v[it], 16);
          } else {
            const int left = static_cast<int>(a.n_out - o);
#pragma unroll
            for (int e = 0; e < EPC - 1; ++e) {
              OutT x;
              if constexpr (sizeof(OutT) == 2) x = static_cast<uint16_t>(v[it][e >> 1] >> (16 * (e & 1)));
              else x = __uint_as_float(v[it][e]);
              if (e < left) dst[e] = x;
            }
          }
        }
      }
    }
    if constexpr (GATE) {
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const int join = static_cast<int>(a.n_out / (TF / WF)) / a.nq;   // wavefronts' sums in one: 2 or 4
      for (int i = tid; i < TT * WF / join; i += NT) {
        const int t = i % TT, g = i / TT * join;
        if (cur.t0 + t < a.n_tok && cur.f0 + g * (TF / WF) < a.n_out) {
          float4 p = add4(red[g * TT + t], red[(g + 1) * TT + t]);
          if (join == 4) p = add4(p, add4(red[(g + 2) * TT + t], red[(g + 3) * TT + t]));
          a.stats[(cur.t0 + t) * a.nq + (cur.f0 / (TF / WF) + g) / join] = p;
        }
      }
    }
  };
  for (;;) {
    more = false;
    while (++round < rounds && !(more = tile_of(round, &next))) {
    }
    const int64_t left = a.n_tok - cur.t0 - wt * (TT / WT);
    jn = static_cast<int>(min(max((left + 31) / 32, int64_t{0}), static_cast<int64_t>(J)));
    if (jn == J) process(std::true_type{});
    else process(std::false_type{});
    if (!more) break;
    cur = next;
    par ^= 1;
  }
}

// Small products of aligned operands, bound by latency: one tile of 64
// outputs x 64 tokens a workgroup, four wavefronts of 32 x 32, and a ring of
// kRing slices of 128 columns in LDS that are all in flight from the start
// (the tiles' two buffers wait for each slice in turn: 256 x 1024 x 2048 8.5
// us there, 5.9 here).  Only while every tile has its place on the chip at once:
// with four tiles a CU at 1024 columns it is the slower (19.6 against 10.0 us).
// kRingLoads memory instructions a wavefront and slice.
constexpr int kRing = 8, kRingLoads = 4;

// Waits until at most `slices` of this wavefront's younger slices are in flight.
__device__ __forceinline__ void wait_for_slice(int slices) {
  switch (slices) {
    case 0: asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); break;
    case 1: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kRingLoads) : "memory"); break;
    case 2: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kRingLoads) : "memory"); break;
    case 3: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * kRingLoads) : "memory"); break;
    case 4: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * kRingLoads) : "memory"); break;
    case 5: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(5 * kRingLoads) : "memory"); break;
    case 6: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(6 * kRingLoads) : "memory"); break;
    default: asm volatile("s_waitcnt vmcnt(%0)" ::"n"(7 * kRingLoads) : "memory"); break;
  }
}

template <typename OutT, bool GATE>
__global__ void __launch_bounds__(256)
project_i8_ring_kernel(ProjectI8Args a, int tiles_f) {
  extern __shared__ u32x4_t lds[];   // [kRing][64 W rows, 64 token rows][8 chunks]
  __shared__ float4 red[GATE ? 64 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lh = lane >> 5, wf = wave & 1, wt = wave >> 1;
  if constexpr (GATE) advance_state(a.adv, blockIdx.x);
  const int64_t f0 = static_cast<int64_t>(blockIdx.x % tiles_f) * 64, t0 = static_cast<int64_t>(blockIdx.x / tiles_f) * 64;
  const int K = a.K, chunks = K / 16, ksteps = (chunks + 7) / 8, ldq = static_cast<int>(a.ldq);
  const int r0 = tid >> 3, ch = (tid & 7) ^ ((r0 >> 1) & 7);
  const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.w + f0 * K), 0,
                                                    static_cast<int>(min(int64_t{64}, a.n_out - f0)) * K, 0x00020000);
  const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q + t0 * ldq), 0,
                                                    static_cast<int>(min(int64_t{64}, a.n_tok - t0)) * ldq, 0x00020000);
  // rows past the end and the chunks past the last one read zeros, as in the tiles
  auto issue = [&](int kt) {
    u32x4_t* dst = lds + (kt % kRing) * 1024 + wave * 64;
    const bool in = kt * 8 + ch < chunks;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (__attribute__((address_space(3))) void*)(dst + i * 256), 16,
                                               (r0 + i * 32) * K + ch * 16, kt * 128, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (__attribute__((address_space(3))) void*)(dst + 512 + i * 256), 16,
                                               in ? (r0 + i * 32) * ldq + ch * 16 : 0x7fff0000, kt * 128, 0, 0);
  };
  // the scales first: they have landed when the first slice has
  float so[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) so[i] = a.w_scale[min(f0 + wf * 32 + (i >> 2) * 8 + lh * 4 + (i & 3), a.n_out - 1)];
  const int64_t tok = t0 + wt * 32 + lr;
  const float st = a.q_scale[min(tok, a.n_tok - 1)];
  asm volatile("" ::: "memory");
#pragma unroll
  for (int p = 0; p < kRing - 1; ++p)
    if (p < ksteps) issue(p);
  i32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0;
  for (int kt = 0; kt < ksteps; ++kt) {
    wait_for_slice(min(kRing - 2, ksteps - 1 - kt));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // everyone's part; slot kt - 1 has been read
    if (kt + kRing - 1 < ksteps) issue(kt + kRing - 1);
    const u32x4_t* Ws = lds + (kt % kRing) * 1024;
    const u32x4_t* Qs = Ws + 512;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int kc = (ks * 2 + lh) ^ ((lr >> 1) & 7);
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, Ws[(wf * 32 + lr) * 8 + kc]),
                                                  __builtin_bit_cast(i32x4_t, Qs[(wt * 32 + lr) * 8 + kc]), acc, 0, 0, 0);
    }
  }
  if constexpr (GATE) {
    // the tile's 64 columns are v's, or one branch's keys
    const bool is_v = f0 < a.d;
    const int branch = is_v ? 0 : static_cast<int>(f0 / a.d) - 1;
    const int64_t row = min(tok, a.n_tok - 1);
    const int64_t c0 = f0 - static_cast<int64_t>(is_v ? 0 : 1 + branch) * a.d + wf * 32 + lh * 4;
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint2 h = make_uint2(0u, 0u);
      if (!is_v) h = *reinterpret_cast<const uint2*>(a.H + (row * a.M + branch) * a.d + c0 + g * 8);
      f32x4_t x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(acc[4 * g + e]) * st * so[4 * g + e];
      if (is_v && tok < a.n_tok) __builtin_memcpy(static_cast<float*>(a.out) + tok * a.d + c0 + g * 8, &x, 16);
      p = add4(p, gate_terms(x, is_v, h));
    }
    p = add4(p, make_float4(__shfl_xor(p.x, 32, 64), __shfl_xor(p.y, 32, 64), __shfl_xor(p.z, 32, 64), __shfl_xor(p.w, 32, 64)));
    if (wf == 1 && lh == 0) red[wt * 32 + lr] = p;
    __syncthreads();
    if (wf == 0 && lh == 0 && tok < a.n_tok) a.stats[tok * a.nq + f0 / 64] = add4(p, red[wt * 32 + lr]);
    return;
  }
  if (tok >= a.n_tok) return;
  OutT* out = static_cast<OutT*>(a.out) + tok * a.n_out;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int64_t o = f0 + wf * 32 + g * 8 + lh * 4;
    OutT x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = to_out<OutT>(static_cast<float>(acc[4 * g + e]) * st * so[4 * g + e]);
    if (o + 4 <= a.n_out) {
      __builtin_memcpy(out + o, x, sizeof(x));
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (o + e < a.n_out) out[o + e] = x[e];
    }
  }
}

// LDS of a workgroup, and how many of them a CU holds.
inline int ring_bytes(int64_t K) { return static_cast<int>(std::min<int64_t>(kRing, (K + 127) / 128)) * 1024 * 16; }
inline int ring_places(int64_t K) { return std::min(4, (160 << 10) / ring_bytes(K)); }

template <typename OutT, bool GATE = false>
hipError_t launch_ring(const ProjectI8Args& a, hipStream_t s) {
  constexpr int kLds = kRing * 1024 * 16;
  auto* const fn = project_i8_ring_kernel<OutT, GATE>;
  static std::atomic<uint64_t> attr_set{0};   // > 64 KiB of dynamic LDS, raised once per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if ((attr_set.load() & bit) == 0) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit);
  }
  const int64_t tf = (a.n_out + 63) / 64, tt = (a.n_tok + 63) / 64;
  launch_k(fn, dim3(static_cast<unsigned>(tf * tt)), dim3(256), ring_bytes(a.K), s, a, static_cast<int>(tf));
  return launch_error();
}

// Fewer than 16 columns: one thread an output.
template <typename OutT>
__global__ void __launch_bounds__(256)
project_i8_short_kernel(ProjectI8Args a) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= a.n_tok * a.n_out) return;
  const int64_t t = id / a.n_out, o = id - t * a.n_out;
  const int8_t* q = a.q + t * a.ldq + (a.tailed ? a.ldq - a.K : 0);   // right-aligned in its 16 bytes
  const int8_t* w = a.w + o * a.K;
  int sum = 0;
  for (int c = 0; c < a.K; ++c) sum += static_cast<int>(q[c]) * static_cast<int>(w[c]);
  static_cast<OutT*>(a.out)[id] = to_out<OutT>(static_cast<float>(sum) * a.q_scale[t] * a.w_scale[o]);
}

// Few tokens: bound by reading W once, or by latency.  Every wavefront streams
// 16 rows of W from memory straight into the operand registers of v_mfma_i32_16x16x64_i8 (lane l: row l & 15, bytes 16 (l >> 4)
// of each run of 64), 16 loads (1024 columns) in flight, while the codes of
// up to 16 NB tokens sit in LDS.  A row of codes starts 16 bytes further
// round the banks than the one before (stride 16 modulo 256), so the 16 rows
// of an operand read are free of conflicts.
// E_DT: type of e.  Up to 16 float rows of together 32,768 columns are
// quantised here, by every workgroup, behind the first loads of W: it saves a
// launch (9 x 1024 x 2048 9.5 -> 8.7 us).  More take longer than a launch of
// their own (32 x 1024 x 2048 13.4 against 11.3 us, 16 x 4096 x 2000 17.9 against
// 16.1).
// 1 x 1024 x 128000 takes 24.3 us (5.4 TB/s), 32 x 1024 x 128000 29.4; past 32
// tokens the tiles are faster (64 tokens: 46 against 36 us).  Held to 128
// registers (4 wavefronts a SIMD) the aligned form of up to 16 tokens spills 20
// bytes a lane.
constexpr int kFewWaves = 8;
constexpr int kFewLds = 140 << 10;
constexpr int kFewShared = 512;   // groups up to which a workgroup shares each

__host__ __device__ inline int few_stride(int K) { return (K + 255) / 256 * 256 + 16; }

// Rows wave, wave + 8, .. of e (R of them per wavefront) to codes and scales
// in LDS; two passes over the rows, the loads of all of them together.
template <int E_DT, int R>
__device__ __forceinline__ void quantize_into(const void* e, int rows, int K, u32x4_t* lds, int stride, float* sq) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c8 = K / 8 * 8, ct = c8 + lane, chunks = (K + 15) / 16;
  uint32_t top[R];
  float ft[R];
  int64_t base[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    base[i] = static_cast<int64_t>(min(wave + i * kFewWaves, rows - 1)) * K;   // rows past the last repeat it
    ft[i] = ct < K ? load1<E_DT>(e, base[i] + ct) : 0.f;
    top[i] = magnitude(ft[i]);
  }
#pragma unroll 2
  for (int c = lane * 8; c < c8; c += 512) {
    float f[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) load8<E_DT>(e, base[i] + c, f[i]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) top[i] = max(top[i], magnitude(f[i][k]));
  }
#pragma unroll
  for (int i = 0; i < R; ++i) top[i] = wave_top(top[i]);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = wave + i * kFewWaves;
    if (t >= rows) break;
    const bool codes = row_has_codes(top[i]);
    const RowScale rs = row_factors(__uint_as_float(top[i]));
    const CodeRow out(reinterpret_cast<int8_t*>(lds + t * stride), K, true);
    if (lane == 0) sq[t] = row_scale(top[i]);
#pragma unroll 2
    for (int c = lane * 8; c < c8; c += 512) {
      float f[8];
      load8<E_DT>(e, base[i] + c, f);
      const u32x2_t w = codes ? quantize8(f, rs) : u32x2_t{0, 0};
      __builtin_memcpy(out.at(c), &w, 8);
    }
    if (ct < K) *out.at(ct) = static_cast<int8_t>(codes ? quantize(ft[i], rs) : 0);
    if (lane < out.shift) out.dst[out.whole + lane] = 0;
    for (int c = chunks + lane; c < (chunks + 3) / 4 * 4; c += 64) lds[t * stride + c] = u32x4_t{0, 0, 0, 0};
  }
}

// SHIFT: rows of W that start at any byte.  A load from an address that is no
// multiple of 4 takes the memory pipeline several times as long, so the 5
// words around each chunk are read and shifted into place.
// ks: wavefronts that share a group of 16 rows, taking every ks-th run of 64
// columns: all kFewWaves where rows are longer than one wavefront's loads in
// flight and groups too few to fill the chip (2 x 3840 x 219 17.3 -> 7.0 us, 8 x
// 4096 x 8192 24.3 -> 19.8), else 1 (1 x 1024 x 16384 8.1 us, shared 18.5).
template <typename OutT, int E_DT, int NB, bool SHIFT>
__global__ void __launch_bounds__(64 * kFewWaves)
__attribute__((amdgpu_waves_per_eu(NB == 1 && !SHIFT ? 4 : 2, NB == 1 && !SHIFT ? 4 : 2)))
project_i8_few_kernel(ProjectI8Args a, const void* __restrict__ e, int ks) {
  extern __shared__ u32x4_t lds[];
  __shared__ float sq[16 * NB];
  __shared__ i32x4_t part[kFewWaves][NB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = a.K, chunks = (K + 15) / 16, steps = (chunks + 3) / 4;
  const int n_tok = static_cast<int>(a.n_tok), stride = few_stride(K) / 16;   // in chunks
  const int r = lane & 15, h = lane >> 4;
  const int64_t groups = (a.n_out + 15) / 16, all = static_cast<int64_t>(gridDim.x) * (kFewWaves / ks);
  int64_t g = ks == 1 ? static_cast<int64_t>(blockIdx.x) * kFewWaves + wave : blockIdx.x;
  const int first = ks == 1 ? 0 : wave;

  u32x4_t w[16];
  uint32_t wx[SHIFT ? 16 : 1];   // the word behind each of them
  const int8_t* const w_end = a.w + a.n_out * K;
  // Bytes by which the chunk at p lies past a multiple of 4, or 0 where its
  // five words are not all W's own (at W's ends): it is then read as it lies.
  auto shift_of = [&](const int8_t* p) {
    const int s4 = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
    return p - s4 < a.w || p - s4 + 20 > w_end ? 0 : s4;
  };
  auto chunk_of = [&](int64_t grp, int step) {
    return a.w + min(grp * 16 + r, a.n_out - 1) * K + min((step * 4 + h) * 16, K - 16);
  };
  auto load = [&](int64_t grp, int s0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int8_t* p = chunk_of(grp, s0 + i * ks);
      if constexpr (SHIFT) {
        const int s4 = shift_of(p);
        __builtin_memcpy(&w[i], p - s4, 16);
        __builtin_memcpy(&wx[i], s4 != 0 ? p - s4 + 16 : p, 4);
      } else {
        __builtin_memcpy(&w[i], p, 16);
      }
    }
  };
  auto operand = [&](int64_t grp, int s0, int i) {
    if constexpr (SHIFT) {
      const uint32_t s4 = static_cast<uint32_t>(shift_of(chunk_of(grp, s0 + i * ks)));
      return i32x4_t{static_cast<int>(__builtin_amdgcn_alignbyte(w[i][1], w[i][0], s4)),
                     static_cast<int>(__builtin_amdgcn_alignbyte(w[i][2], w[i][1], s4)),
                     static_cast<int>(__builtin_amdgcn_alignbyte(w[i][3], w[i][2], s4)),
                     static_cast<int>(__builtin_amdgcn_alignbyte(wx[i], w[i][3], s4))};
    } else {
      return __builtin_bit_cast(i32x4_t, w[i]);
    }
  };
  if (g < groups) load(g, first);

  // codes into LDS, in the layout of a chunked row with the tail right-aligned
  if constexpr (E_DT == ENGRAM_I8) {
    for (int i = threadIdx.x; i < n_tok * steps * 4; i += 64 * kFewWaves) {
      const int t = i / (steps * 4), c = i % (steps * 4);
      const int8_t* row = a.q + t * a.ldq;
      u32x4_t v{0, 0, 0, 0};
      if (c < chunks) v = a.tailed ? *reinterpret_cast<const u32x4_t*>(row + c * 16) : load_chunk(row, c, K);
      lds[t * stride + c] = v;
    }
    if (threadIdx.x < 16 * NB) sq[threadIdx.x] = a.q_scale[min(static_cast<int>(threadIdx.x), n_tok - 1)];
  } else if (n_tok <= kFewWaves) {
    quantize_into<E_DT, 1>(e, n_tok, K, lds, stride, sq);
  } else {
    quantize_into<E_DT, 2>(e, n_tok, K, lds, stride, sq);
  }
  __syncthreads();

  for (; g < groups; g += all) {
    const int64_t o = g * 16 + h * 4;   // acc[b][k]: output o + k of token 16 b + r
    float so[4];                        // read before the next group's rows: loads return in order
#pragma unroll
    for (int k = 0; k < 4; ++k) so[k] = a.w_scale[min(o + k, a.n_out - 1)];
    i32x4_t acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = i32x4_t{0, 0, 0, 0};
    for (int s0 = first; s0 < steps; s0 += 16 * ks) {
      if (s0 > first) load(g, s0);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (s0 + i * ks < steps) {
          const i32x4_t wi = operand(g, s0, i);
#pragma unroll
          for (int b = 0; b < NB; ++b)   // tokens past the last read the first one's codes; not stored
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                wi,
                __builtin_bit_cast(i32x4_t, lds[(b * 16 + r < n_tok ? b * 16 + r : 0) * stride + (s0 + i * ks) * 4 + h]), acc[b], 0, 0, 0);
        }
      }
    }
    if (g + all < groups) load(g + all, first);
    if (ks > 1) {   // the workgroup's wavefronts share the group: their sums join in the first one
#pragma unroll
      for (int b = 0; b < NB; ++b) part[wave][b][lane] = acc[b];
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll 1
          for (int k = 1; k < kFewWaves; ++k) acc[b] += part[k][b][lane];
      }
      __syncthreads();
      if (wave != 0) continue;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b * 16 + r >= n_tok) continue;
      const float st = sq[b * 16 + r];
      OutT x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = to_out<OutT>(static_cast<float>(acc[b][k]) * st * so[k]);
      OutT* dst = static_cast<OutT*>(a.out) + static_cast<int64_t>(b * 16 + r) * a.n_out + o;
      if (o + 4 <= a.n_out) {
        __builtin_memcpy(dst, x, sizeof(x));
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (o + k < a.n_out) dst[k] = x[k];
      }
    }
  }
}

template <typename OutT, int E_DT, int NB, bool SHIFT>
hipError_t launch_few(const ProjectI8Args& a, const void* e, hipStream_t s) {
  auto* const fn = project_i8_few_kernel<OutT, E_DT, NB, SHIFT>;
  const int bytes = static_cast<int>(a.n_tok) * few_stride(a.K);
  static std::atomic<uint64_t> attr_set{0};   // > 64 KiB of dynamic LDS, raised once per device
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if ((attr_set.load() & bit) == 0) {
    err = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kFewLds);
    if (err != hipSuccess) return err;
    attr_set.fetch_or(bit);
  }
  const int64_t groups = (a.n_out + 15) / 16;
  const int64_t most = NB == 1 && !SHIFT && bytes <= kFewLds / 2 ? 512 : 256;   // workgroups that are on the chip together
  const bool shared = a.K > 1024 && groups <= kFewShared;
  const int64_t blocks = std::min(most, shared ? groups : (groups + kFewWaves - 1) / kFewWaves);
  launch_k(fn, dim3(static_cast<unsigned>(blocks)), dim3(64 * kFewWaves), bytes, s, a, e, shared ? kFewWaves : 1);
  return launch_error();
}

template <typename OutT, int E_DT, int NB>
hipError_t launch_few_shift(const ProjectI8Args& a, const void* e, hipStream_t s) {
  return a.K % 4 == 0 ? launch_few<OutT, E_DT, NB, false>(a, e, s) : launch_few<OutT, E_DT, NB, true>(a, e, s);
}

template <typename OutT, int E_DT>
hipError_t launch_few_blocks(const ProjectI8Args& a, const void* e, hipStream_t s) {
  if constexpr (E_DT == ENGRAM_I8) {
    if (a.n_tok > 16) return launch_few_shift<OutT, E_DT, 2>(a, e, s);
  }
  return launch_few_shift<OutT, E_DT, 1>(a, e, s);
}

template <typename OutT, int TF, int TT, int WF, int WT, bool GATE = false>
hipError_t launch_tile(const ProjectI8Args& a, hipStream_t s) {
  constexpr int kLds = 2 * (TF + TT) * 128 + 2 * (TF + TT) * 4 + (GATE ? WF * TT * 16 : 0);
  static_assert(kLds * (8 / (WF * WT)) <= 160 << 10, "one workgroup of 8 wavefronts, or two of 4, on a CU");
  auto* const fn = project_i8_tile_kernel<OutT, TF, TT, WF, WT, GATE>;
  static std::atomic<uint64_t> attr_set{0};   // > 64 KiB of dynamic LDS, raised once per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if ((attr_set.load() & bit) == 0) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit);
  }
  const int64_t tf = (a.n_out + TF - 1) / TF, tt = (a.n_tok + TT - 1) / TT;
  if (tf * tt > (1 << 30)) return hipErrorInvalidValue;
  // one workgroup of 8 wavefronts per CU, or two of 4
  const int grid = static_cast<int>(std::min<int64_t>(256 * 8 / (WF * WT), (tf * tt + 7) / 8 * 8));
  launch_k(fn, dim3(grid), dim3(64 * WF * WT), kLds, s, a, static_cast<int>(tf), static_cast<int>(tt));
  return launch_error();
}

// Which kernel a product of aligned operands takes.
enum class Form { kRing, kTile128, kTile256 };

Form product_form(int64_t n_tok, int64_t n_out, int64_t K) {
  if (((n_out + 63) / 64) * ((n_tok + 63) / 64) <= 256 * ring_places(K)) return Form::kRing;
  // a large tile for every CU
  return ((n_out + 255) / 256) * ((n_tok + 255) / 256) >= 256 ? Form::kTile256 : Form::kTile128;
}

template <typename OutT>
hipError_t launch_tiles(const ProjectI8Args& a, hipStream_t s) {
  switch (product_form(a.n_tok, a.n_out, a.K)) {
    case Form::kRing: return launch_ring<OutT>(a, s);
    case Form::kTile256: return launch_tile<OutT, 256, 256, 4, 2>(a, s);
    default: return launch_tile<OutT, 128, 128, 2, 2>(a, s);
  }
}

// The GATE forms' sums come in runs of 64 columns (ring), 128 or 256; the conv
// takes at most kConvMaxStats of them per row.
Form gate_form(int64_t n_tok, int64_t n_out, int64_t K, int d) {
  const Form f = product_form(n_tok, n_out, K);
  return f == Form::kRing && 2 * d / 64 > kConvMaxStats ? Form::kTile128 : f;
}

}  // namespace

// Copied rows past 512 columns begin on whole 128-byte lines, like the slices
// that the products read of them (2000 x 4112 x 2000 33 us, 2000 x 4224 x 2000
// 27); shorter ones would grow by more than they gain (300 x 77 x 128000 moves
// 60% more).
int64_t i8_row_stride(int64_t cols) {
  const int64_t whole = cols > 512 ? 128 : 16;
  return cols % 16 == 0 ? cols : (cols + whole - 1) / whole * whole;
}

namespace {

AlignJob align_job(const int8_t* x, int8_t* y, int64_t rows, int64_t K) {
  const int64_t per = 256 * kAlignItems;
  return AlignJob{x, reinterpret_cast<u32x4_t*>(y), rows, (rows * (i8_row_stride(K) / 16) + per - 1) / per};
}

// Workgroups of 256 threads that a launch can have: it has fewer than 2^32
// work-items (launch_k).
constexpr int64_t kMostGroups = (1 << 24) - 1;

// More rows than a launch has workgroups for go in pieces; W's come with the first.
template <int DT, int N>
hipError_t launch_quantize_n(QuantizeArgs a, AlignJob w, hipStream_t s) {
  constexpr int64_t per = N > 0 ? 4 : 1;   // rows of a workgroup
  const int chunks = static_cast<int>(i8_row_stride(a.cols) / 16);
  if (w.groups >= kMostGroups) return hipErrorInvalidConfiguration;
  for (int64_t left = a.rows; left > 0;) {
    const int64_t n = std::min(left, (kMostGroups - w.groups) * per);
    const dim3 grid(static_cast<unsigned>(w.groups + (n + per - 1) / per));
    a.rows = n;
    prof_stage("quantize_i8_kernel");
    if (w.groups > 0) launch_k((quantize_rows_kernel<DT, N, true>), grid, dim3(256), 0, s, a, w, chunks);
    else launch_k((quantize_rows_kernel<DT, N, false>), grid, dim3(256), 0, s, a, w, chunks);
    const hipError_t e = launch_error();
    if (e != hipSuccess) return e;
    a.x = static_cast<const char*>(a.x) + n * a.cols * (DT == ENGRAM_BF16 ? 2 : 4);
    a.q += n * a.ldq;
    a.scale += n;
    w = AlignJob{};
    left -= n;
  }
  return hipSuccess;
}

template <int DT>
hipError_t launch_quantize_dt(const QuantizeArgs& a, const AlignJob& w, hipStream_t s) {
  // the fewest registers that hold a row
  if (a.cols < 512 + 8) return launch_quantize_n<DT, 1>(a, w, s);
  if (a.cols < 1024 + 8) return launch_quantize_n<DT, 2>(a, w, s);
  if (a.cols < 2048 + 8) return launch_quantize_n<DT, 4>(a, w, s);
  if (a.cols < 4096 + 8) return launch_quantize_n<DT, 8>(a, w, s);
  return launch_quantize_n<DT, 0>(a, w, s);
}

}  // namespace

hipError_t launch_quantize_i8(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* q, int64_t ldq, bool tail, float* scale,
                              const int8_t* w, int64_t w_rows, int8_t* w_out, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const QuantizeArgs a{x, rows, q, ldq, scale, static_cast<int>(cols), tail ? 1 : 0};
  const AlignJob job = w_out != nullptr ? align_job(w, w_out, w_rows, cols) : AlignJob{};
  return dtype == ENGRAM_BF16 ? launch_quantize_dt<ENGRAM_BF16>(a, job, s) : launch_quantize_dt<ENGRAM_F32>(a, job, s);
}

namespace {

bool project_i8_few(int64_t n_tok, int64_t K) {
  return n_tok <= 32 && K >= 16 && n_tok * few_stride(static_cast<int>(K)) <= kFewLds;
}

}  // namespace

bool project_i8_quantizes(int64_t n_tok, int64_t K) { return n_tok <= 16 && n_tok * K <= 32768 && project_i8_few(n_tok, K); }

bool project_i8_aligns(int64_t n_tok, int64_t K) { return K >= 16 && K % 16 != 0 && !project_i8_few(n_tok, K); }

hipError_t launch_align_i8(const int8_t* w, int64_t w_rows, int8_t* w_out, const int8_t* q, int64_t q_rows, int8_t* q_out, int64_t K,
                           hipStream_t s) {
  const AlignJob a = align_job(w, w_out, w_rows, K), b = align_job(q, q_out, q_rows, K);
  if (a.groups + b.groups > kMostGroups) return hipErrorInvalidConfiguration;   // (copies of 2^38 bytes)
  launch_k(align_rows_kernel, dim3(static_cast<unsigned>(a.groups + b.groups)), dim3(256), 0, s, a, b, static_cast<int>(K),
           static_cast<int>(i8_row_stride(K) / 16));
  return launch_error();
}

namespace {

template <typename OutT>
hipError_t launch_product(ProjectI8Args a, const void* e, int e_dtype, hipStream_t s) {
  if (e_dtype == ENGRAM_BF16) return launch_few_blocks<OutT, ENGRAM_BF16>(a, e, s);
  if (e_dtype == ENGRAM_F32) return launch_few_blocks<OutT, ENGRAM_F32>(a, e, s);
  if (project_i8_few(a.n_tok, a.K)) return launch_few_blocks<OutT, ENGRAM_I8>(a, nullptr, s);
  if (a.K < 16) {
    // one thread an output, so tokens go in pieces of at most 2^31 outputs
    const int64_t n_tok = a.n_tok, piece = std::max<int64_t>((int64_t{1} << 31) / a.n_out, 1);
    for (int64_t t = 0; t < n_tok; t += piece) {
      a.n_tok = std::min(piece, n_tok - t);
      prof_stage("project_i8_kernel");
      launch_k(project_i8_short_kernel<OutT>, dim3(static_cast<unsigned>((a.n_tok * a.n_out + 255) / 256)), dim3(256), 0, s, a);
      const hipError_t err = launch_error();
      if (err != hipSuccess) return err;
      a.q += piece * a.ldq;
      a.q_scale += piece;
      a.out = static_cast<OutT*>(a.out) + piece * a.n_out;
    }
    return hipSuccess;
  }
  // whole chunks from here on: the rows are the product's own layout
  a.K = static_cast<int>(i8_row_stride(a.K));
  return launch_tiles<OutT>(a, s);
}

}  // namespace

hipError_t launch_project_i8(const void* e, int e_dtype, int64_t ldq, bool tailed, const float* q_scale, const int8_t* w,
                             const float* w_scale, int64_t n_tok, int64_t K, int64_t n_out, int out_dtype, void* out,
                             hipStream_t s) {
  if (n_tok == 0) return hipSuccess;
  const ProjectI8Args a{static_cast<const int8_t*>(e), q_scale, w, w_scale, out, n_tok, ldq, n_out, static_cast<int>(K), tailed ? 1 : 0,
                        nullptr, nullptr, 0, 0, 0, StateAdvance{}};
  return out_dtype == ENGRAM_BF16 ? launch_product<uint16_t>(a, e, e_dtype, s) : launch_product<float>(a, e, e_dtype, s);
}

bool project_i8_gate_advances(int64_t n_tok, int64_t K, int d, int M) {
  return gate_form(n_tok, static_cast<int64_t>(1 + M) * d, K, d) == Form::kRing;
}

int project_i8_gate_columns(int64_t n_tok, int64_t K, int d, int M) {
  switch (gate_form(n_tok, static_cast<int64_t>(1 + M) * d, K, d)) {
    case Form::kRing: return 64;
    case Form::kTile256: return d % 256 == 0 ? 256 : 128;
    default: return 128;
  }
}

hipError_t launch_project_i8_gate(const int8_t* q, const float* q_scale, const int8_t* w, const float* w_scale, int64_t n_tok, int64_t K,
                                  int d, int M, const void* H, float* v, float4* stats, const StateAdvance& adv, hipStream_t s) {
  if (n_tok == 0) return hipSuccess;
  if (K % 16 != 0 || d % 128 != 0 || d > 4096) return hipErrorInvalidValue;
  if (adv.adv_B > 0 && !project_i8_gate_advances(n_tok, K, d, M)) return hipErrorInvalidValue;
  const int64_t n_out = static_cast<int64_t>(1 + M) * d;
  const ProjectI8Args a{q, q_scale, w, w_scale, v, n_tok, K, n_out, static_cast<int>(K), 0, static_cast<const uint16_t*>(H), stats, d, M,
                        static_cast<int>(n_out / project_i8_gate_columns(n_tok, K, d, M)), adv};
  switch (gate_form(n_tok, n_out, K, d)) {
    case Form::kRing: return launch_ring<float, true>(a, s);
    case Form::kTile256: return launch_tile<float, 256, 256, 4, 2, true>(a, s);
    default: return launch_tile<float, 128, 128, 2, 2, true>(a, s);
  }
}

}  // namespace engram
