// Step 5 ("DeepSeek Engram series guide": v_t = W_V e_t, k_t = W_K e_t) for
// many requests at once, each with a low-rank adapter of its own beside the
// shared W:
//   out_t = W e_t + s_a B_a (A_a e_t),   a = the adapter of token t's request
//
// Two launches.  The first leaves h_t = s_a A_a e_t for every token that has
// an adapter; the second is the product with W, which adds B_a h_t to its
// sums before they are rounded once and stored.  Tokens stay where they are:
// a block of 32 tokens goes over the adapters that occur in it, with the rows
// h of the other tokens read as zeros, so one adapter costs a few matrix
// instructions and one read of its rows of B however its tokens are spread.
//
// bf16 layers keep h as the sum of two bf16 numbers (off by 2^-17 of h, beside
// the 2^-8 of an output in bf16): one alone would be off by 2^-9, too much for
// float32 outputs; A and B enter unrounded.  float32 layers run on
// the float32 matrix instructions throughout.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device_util.h"
#include "engram_internal.h"

namespace engram {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kChunk = 64;   // columns of a step of the fragment loops

// 16 bytes of a row are a lane's share of a step: 8 bf16 columns (one
// v_mfma_f32_32x32x16_bf16) or 4 float32 ones (four v_mfma_f32_32x32x2_f32).
template <int DT>
struct Frag {
  static constexpr int kSize = DT == ENGRAM_BF16 ? 2 : 4;
  static constexpr int kVals = 16 / kSize;
  static constexpr int kSteps = kChunk / 2 / kVals;   // of a chunk: lanes 0-31 take its first half, 32-63 its second
};

template <int DT>
__device__ __forceinline__ f32x16_t multiply(u32x4_t a, u32x4_t b, f32x16_t acc) {
  if constexpr (DT == ENGRAM_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
  } else {
    const f32x4_t x = __builtin_bit_cast(f32x4_t, a), y = __builtin_bit_cast(f32x4_t, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], acc, 0, 0, 0);
    return acc;
  }
}

// Element i of an array of the layer's type.
template <int DT>
__device__ __forceinline__ const char* element(const void* p, int64_t i) { return static_cast<const char*>(p) + i * Frag<DT>::kSize; }

__device__ __forceinline__ u32x4_t load16(const char* p) { return *reinterpret_cast<const u32x4_t*>(p); }

struct AdaptArgs {
  const void* e;          // [n_tok][K]
  const void* w;          // [n_out][K]
  const void* a;          // [adapters][rank][K]
  const void* b;          // [adapters][n_out][rank]
  const float* scale;     // [adapters] or null
  const int32_t* which;   // [ceil(n_tok / per)]
  void* h;                // bf16: [n_tok][2][padded rank], float32: [n_tok][rank]
  void* out;              // [n_tok][n_out]
  int64_t n_tok;
  uint32_t per;
  int32_t K;
  int32_t n_out;
  int32_t rank;
  int32_t adapters;
  uint32_t first;         // workgroup of this launch
};

// A launch has fewer than 2^32 work-items (launch_k): workgroups, of up to 1024
// threads, are launched so many at a time.
constexpr int64_t kMostGroups = 1 << 21;

// Columns of a row of h: whole matrix steps.
__device__ __host__ __forceinline__ int h_columns(int dt, int rank) { return dt == ENGRAM_BF16 ? 2 * ((rank + 15) / 16 * 16) : rank; }

// Token t's adapter, -1 for none.
__device__ __forceinline__ int adapter_of(const AdaptArgs& a, int64_t t) {
  if (t >= a.n_tok) return -1;
  const int id = a.which[a.per == 1 ? static_cast<uint32_t>(t) : static_cast<uint32_t>(t) / a.per];
  return static_cast<uint32_t>(id) < static_cast<uint32_t>(a.adapters) ? id : -1;
}

// f(adapter, its place among them) of the adapters that occur among a wavefront's ids.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F f) {
  uint64_t left = __ballot(id >= 0);
  for (int j = 0; left != 0; ++j) {
    const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    left &= ~__ballot(id == one);
    f(one, j);
  }
}

// ---- h ----
// The rows of A of all adapters in a block of 32 tokens, one adapter after
// another, are taken 32 a workgroup (small ranks share one, large ones take
// several), each with all of the block's tokens; what is stored is each token's
// products with its own adapter.  NW wavefronts take every NW-th 64 columns.  A
// chain of loads where tokens are few (256 tokens of 64 adapters of rank 16, 1024
// columns: 7 us), the operands' way from the L2 where they are many (4096: 31 us;
// with a workgroup for every adapter, whatever its rank, 46).  A block's tokens meet
// all of its adapters' rows, one share of the products is kept: 32763 tokens of 64
// adapters take 197 us at rank 16 and 739 at rank 64 with an adapter a token, 16 and
// 36 with one for every 256.
template <int DT, int NW>
__global__ void __launch_bounds__(NW * 64)
adapter_rows_kernel(AdaptArgs a) {
  using Fr = Frag<DT>;
  __shared__ f32x4_t part[NW][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 31, lh = lane >> 5;
  const int64_t t = static_cast<int64_t>(a.first + blockIdx.x) * 32 + lr;
  const int id = adapter_of(a, t);
  const int v = static_cast<int>(blockIdx.y) * 32 + lr, which = v / a.rank, r = v - which * a.rank;   // this lane's row
  int mine = -1;
  each_adapter(id, [&](int one, int j) { mine = j == which ? one : mine; });
  if (!__any(mine >= 0)) return;   // fewer rows in this block
  const bool row = mine >= 0;
  const char* e = element<DT>(a.e, min(t, a.n_tok - 1) * a.K + lh * (kChunk / 2));
  const char* ap = element<DT>(a.a, (static_cast<int64_t>(row ? mine : 0) * a.rank + r) * a.K + lh * (kChunk / 2));
  f32x16_t acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int c = wave * kChunk; c < a.K; c += NW * kChunk) {
    u32x4_t fa[Fr::kSteps], fe[Fr::kSteps];
#pragma unroll
    for (int s = 0; s < Fr::kSteps; ++s) {
      fa[s] = load16(ap + static_cast<int64_t>(c) * Fr::kSize + s * 16);
      fe[s] = load16(e + static_cast<int64_t>(c) * Fr::kSize + s * 16);
    }
#pragma unroll
    for (int s = 0; s < Fr::kSteps; ++s) acc = multiply<DT>(row ? fa[s] : u32x4_t{0, 0, 0, 0}, fe[s], acc);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) part[wave][g][lane] = f32x4_t{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
  __syncthreads();
  // rows 8 wave + 4 lh .. + 3 of these 32, of the lane's token (of one adapter: a rank is a multiple of 8)
  if (wave >= 4) return;
  const int owner = __shfl(mine, wave * 8 + lh * 4, 64), column = __shfl(r, wave * 8 + lh * 4, 64);
  if (owner < 0 || owner != id) return;
  f32x4_t x = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) x += part[w][wave][lane];
  x *= a.scale != nullptr ? a.scale[owner] : 1.0f;
  const int hc = h_columns(DT, a.rank);
  if constexpr (DT == ENGRAM_BF16) {
    uint16_t* h = static_cast<uint16_t*>(a.h) + t * hc + column;
    uint32_t hi[2], lo[2];
    // The first part stops at bf16's largest number: what is larger goes on in the second one, an infinity or a NaN too.
    constexpr float kMost = 0x1.fep127f;
    auto first_part = [](float y) { return __builtin_amdgcn_fmed3f(y, -kMost, kMost); };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hi[i] = pack_bf16x2(first_part(x[2 * i]), first_part(x[2 * i + 1]));
      lo[i] = pack_bf16x2(x[2 * i] - __uint_as_float(hi[i] << 16), x[2 * i + 1] - __uint_as_float(hi[i] & 0xffff0000u));
    }
    *reinterpret_cast<uint2*>(h) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(h + hc / 2) = make_uint2(lo[0], lo[1]);
  } else {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.h) + t * hc + column) = x;
  }
}

// Adds B_a h_t to the sums of a block of 32 outputs (from f0 on) x one of 32
// tokens: every `of`-th of the adapters in it, from `first` on.  id: of the
// lane's token t.  A lane's sums are its own token's: where the block holds other
// tokens they keep what they had, so that an infinity or a NaN in one request's
// adapter stays with it.
template <int DT>
__device__ __forceinline__ void add_adapters(const AdaptArgs& a, int id, int64_t t, int64_t f0, int first, int of, f32x16_t& acc) {
  constexpr int kStep = 2 * Frag<DT>::kVals;   // columns of B of a step
  const int lr = threadIdx.x & 31, lh = (threadIdx.x & 63) >> 5, hc = h_columns(DT, a.rank);
  const char* h = static_cast<const char*>(a.h) + min(t, a.n_tok - 1) * hc * Frag<DT>::kSize + lh * 16;
  each_adapter(id, [&](int one, int j) {
    if (j % of != first) return;
    const char* b = element<DT>(a.b, (static_cast<int64_t>(one) * a.n_out + f0 + lr) * a.rank) + lh * 16;
    f32x16_t sum = acc;
    for (int r = 0; r < a.rank; r += kStep) {
      const bool in = r + lh * Frag<DT>::kVals < a.rank;   // (a rank of 8, 24, ..: the last step's second half has no columns)
      const int at = r * Frag<DT>::kSize;
      const u32x4_t zero = {0, 0, 0, 0};
      u32x4_t fb = load16(b + (in ? at : 0)), h0 = load16(h + at), h1 = zero;
      if constexpr (DT == ENGRAM_BF16) h1 = load16(h + at + hc);
      if (!in) fb = h0 = h1 = zero;
      sum = multiply<DT>(fb, h0, sum);
      if constexpr (DT == ENGRAM_BF16) sum = multiply<DT>(fb, h1, sum);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = id == one ? sum[i] : acc[i];
  });
}

// ---- few tokens ----
// A block of 32 tokens x 32 outputs a workgroup.  Its NW wavefronts share the
// columns (every NW-th 64) and the adapters, operands straight from memory into
// registers; their sums meet in LDS.  One token, 1024 x 2048 in bf16: 4.8 us, a
// chain of loads.
template <int DT, int NW, typename OutT>
__global__ void __launch_bounds__(NW * 64)
adapt_small_kernel(AdaptArgs a, int tiles_f) {
  using Fr = Frag<DT>;
  __shared__ f32x4_t part[NW][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 31, lh = lane >> 5;
  const unsigned block = a.first + blockIdx.x;
  const int64_t f0 = static_cast<int64_t>(block % tiles_f) * 32, t = static_cast<int64_t>(block / tiles_f) * 32 + lr;
  const char* w = element<DT>(a.w, (f0 + lr) * a.K + lh * (kChunk / 2));
  const char* e = element<DT>(a.e, min(t, a.n_tok - 1) * a.K + lh * (kChunk / 2));
  const int id = adapter_of(a, t);
  f32x16_t acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int c = wave * kChunk; c < a.K; c += NW * kChunk) {
    u32x4_t fw[Fr::kSteps], fe[Fr::kSteps];
#pragma unroll
    for (int s = 0; s < Fr::kSteps; ++s) {
      fw[s] = load16(w + static_cast<int64_t>(c) * Fr::kSize + s * 16);
      fe[s] = load16(e + static_cast<int64_t>(c) * Fr::kSize + s * 16);
    }
#pragma unroll
    for (int s = 0; s < Fr::kSteps; ++s) acc = multiply<DT>(fw[s], fe[s], acc);
  }
  add_adapters<DT>(a, id, t, f0, wave, NW, acc);
#pragma unroll
  for (int g = 0; g < 4; ++g) part[wave][g][lane] = f32x4_t{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
  __syncthreads();
  if (wave >= 4 || t >= a.n_tok) return;
  f32x4_t x = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) x += part[w][wave][lane];
  OutT* out = static_cast<OutT*>(a.out) + t * a.n_out + f0 + wave * 8 + lh * 4;
  if constexpr (sizeof(OutT) == 2) *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  else *reinterpret_cast<f32x4_t*>(out) = x;
}

// ---- more tokens ----
// A tile of TF outputs x TT tokens a workgroup, WF x WT wavefronts; slices of
// 128 bytes of both operands' rows go from memory straight into LDS, RING - 1 in
// flight while one is multiplied.  A slice's row is 128 bytes, its 16-byte
// chunk c at c ^ ((row >> 1) & 7), so that the rows a fragment read touches
// spread over the banks.
//
// The adapters are more slices of the same loop: behind the columns of W come
// kColumns columns of B of every adapter that occurs among a wavefront's tokens, four
// to a slice, kPer = 4 / WT for each row of wavefronts, multiplied with the
// tokens' rows of h from registers.  Read from memory by the wavefronts
// themselves, one adapter after another, they took 25 of 34 us at 256 tokens of
// 64 adapters (1024 x 5120); in slices that one row of wavefronts filled after
// the other, 31 of 41.  Bound by the LDS reads of the operands: 32763 x 1024 x 5120
// with 16 adapters, bf16 outputs, 420 us (median of 60 calls in three series, 380 to
// 526 as the clock goes; the library's product without adapters, in turn with it, 285
// and 273 to 394), float32 8192 x 1024 x 5120 658 (the matrix cores: 131 TFLOP/s).
// Every adapter that occurs among a wavefront's tokens costs as many matrix
// instructions as if all of them had it, so spread ones cost by their number and
// rank: 32763 x 1024 x 2048 with 64 adapters, an adapter a token and one for every 256,
// rank 16 444 and 166 us, rank 64 1736 and 195; float32, 4096 tokens, rank 64, 787 and
// 158.  Two workgroups of 128 x 128 share a CU, which
// needs no more than 256 registers a lane: with 268, as the compiler chose by
// itself, bf16 outputs took 44 us instead of 32 at 2048 tokens x 5120.
constexpr int kXcds = 8, kBand = 8;

// Waits until at most `younger` slices of LOADS instructions are in flight.
template <int LOADS, int MOST>
__device__ __forceinline__ void wait_slices(int younger) {
  static_assert(LOADS * MOST < 64, "the counter's range");
  if constexpr (MOST > 0) {
    if (younger >= MOST) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS * MOST) : "memory");
      return;
    }
    wait_slices<LOADS, MOST - 1>(younger);
  } else {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

template <int DT, int TF, int TT, int WF, int WT, int RING, typename OutT>
__global__ void __launch_bounds__(WF * WT * 64, 2)
adapt_tile_kernel(AdaptArgs a, int tiles_f, int tiles_t) {
  constexpr int NT = WF * WT * 64, FB = TF / WF / 32, TB = TT / WT / 32;
  constexpr int kSize = Frag<DT>::kSize, kVals = Frag<DT>::kVals, kColumns = 2 * kVals;   // kColumns of B: a part of a slice
  constexpr int kRowsAtOnce = NT / 8, kLoadsW = TF / kRowsAtOnce, kLoadsE = TT / kRowsAtOnce, kBuffer = (TF + TT) * 8;
  extern __shared__ u32x4_t lds[];   // [RING][TF + TT rows][8 chunks]; afterwards each wavefront's outputs
  constexpr int kPer = 4 / WT, kTokens = TT / WT;
  static_assert(TB <= 2 && WT * kPer == 4, "a lane of the wavefront for each of its tokens, four adapters a slice");
  __shared__ int adapters[WT][kTokens], counts[WT];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 31, lh = lane >> 5;
  const int wf = wave % WF, wt = wave / WF;
  // Workgroup i runs on XCD i % 8: each XCD walks tiles of its own, band by
  // band of token tiles, outputs outside, so that a band's rows stay in its L2
  // while W streams past.
  const int per_xcd = gridDim.x / kXcds, tile = a.first + (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
  if (tile >= tiles_f * tiles_t) return;
  const int band = tile / (tiles_f * kBand), in_band = tile - band * tiles_f * kBand, bt = min(kBand, tiles_t - band * kBand);
  const int64_t f0 = static_cast<int64_t>(in_band / bt) * TF, t0 = (static_cast<int64_t>(band) * kBand + in_band % bt) * TT;
  const int K = a.K, ksteps = K * kSize / 128;
  const int r0 = tid >> 3, ch = (tid & 7) ^ ((r0 >> 1) & 7);
  // rows past the end read zeros
  const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(element<DT>(a.w, f0 * K)), 0,
                                                    static_cast<int>(min(int64_t{TF}, a.n_out - f0)) * K * kSize, 0x00020000);
  const auto re = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(element<DT>(a.e, t0 * K)), 0,
                                                    static_cast<int>(min(int64_t{TT}, a.n_tok - t0)) * K * kSize, 0x00020000);
  auto issue = [&](int kt) {
    u32x4_t* dst = lds + (kt % RING) * kBuffer + wave * 64;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (__attribute__((address_space(3))) void*)(dst + i * NT), 16,
                                               ((r0 + i * kRowsAtOnce) * K + ch * kVals) * kSize, kt * 128, 0, 0);
#pragma unroll
    for (int i = 0; i < kLoadsE; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (__attribute__((address_space(3))) void*)(dst + TF * 8 + i * NT), 16,
                                               ((r0 + i * kRowsAtOnce) * K + ch * kVals) * kSize, kt * 128, 0, 0);
  };
  const int64_t tw0 = t0 + wt * (TT / WT);
  int id[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) id[b] = adapter_of(a, tw0 + b * 32 + lr);
#pragma unroll
  for (int p = 0; p < RING - 1; ++p)
    if (p < ksteps) issue(p);
  // the adapters among each row of wavefronts' tokens, in the order of their first ones
  const int token = TB == 2 && lh == 1 ? id[TB - 1] : TB == 1 && lh == 1 ? -1 : id[0];   // a lane's own of them
  bool opens = token >= 0;
  if (!__all(token == __builtin_amdgcn_readfirstlane(token)))
#pragma unroll 4
    for (int l = 0; l < kTokens - 1; ++l) {
      const int earlier = __builtin_amdgcn_readlane(token, l);   // (every lane active)
      opens &= (l >= lane) | (earlier != token);
    }
  else
    opens &= lane == 0;
  const uint64_t openers = __ballot(opens);
  const int own = __popcll(openers);
  if (wf == 0) {
    if (opens) adapters[wt][__popcll(openers & ((uint64_t{1} << lane) - 1))] = token;
    if (lane == 0) counts[wt] = own;
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  int most = 0;
#pragma unroll
  for (int g = 0; g < WT; ++g) most = max(most, counts[g]);
  // The slices: kColumns columns of B after kColumns columns, each of kPer adapters of every row of wavefronts after kPer.
  const int turns = (most + kPer - 1) / kPer, slices = ksteps + turns * ((a.rank + kColumns - 1) / kColumns);
  // This lane loads a half of one entry a slice (chunk ch), the `load_j`-th adapter of its row, columns load_r .. + kVals - 1.
  // Where there is none something valid is loaded and not used.  An entry's place is found a slice ahead.
  const int row_of = (ch >> 1) / kPer, in_row = counts[row_of];
  int load_j = (ch >> 1) % kPer, load_r = (ch & 1) * kVals;
  auto entry = [&]() {
    const bool has = load_j < in_row && load_r < a.rank;
    const int64_t from = has ? static_cast<int64_t>(adapters[row_of][load_j]) * a.n_out : 0;
    const char* src = element<DT>(a.b, from * a.rank + (has ? load_r : 0));
    load_j += kPer;
    if (load_j >= turns * kPer) {
      load_j -= turns * kPer;
      load_r += kColumns;
    }
    return src;
  };
  int rows[kLoadsW];   // the rows of B that this lane loads
#pragma unroll
  for (int l = 0; l < kLoadsW; ++l) {
    const int64_t o = f0 + r0 + l * kRowsAtOnce;
    rows[l] = static_cast<int>(o < a.n_out ? o : 0);
  }
  const char* from = slices > ksteps ? entry() : nullptr;
  auto issue_adapters = [&](int kt) {
    u32x4_t* dst = lds + (kt % RING) * kBuffer + wave * 64;
#pragma unroll
    for (int l = 0; l < kLoadsW; ++l)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)element<DT>(from, static_cast<int64_t>(rows[l]) * a.rank),
                                       (__attribute__((address_space(3))) void*)(dst + l * NT), 16, 0, 0);
#pragma unroll
    for (int l = 0; l < kLoadsE; ++l)   // (no rows: a slice has its number of loads all the same)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (__attribute__((address_space(3))) void*)(dst + TF * 8 + l * NT), 16, 0x7fff0000, 0, 0, 0);
    from = entry();
  };
#pragma unroll
  for (int p = 0; p < RING - 1; ++p)
    if (p >= ksteps && p < slices) issue_adapters(p);
  f32x16_t acc[TB][FB];
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int f = 0; f < FB; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[b][f][i] = 0.f;
  // (the wait: slice kt is there, and slice kt - 1, whose buffer is filled next, has been read)
  auto begin = [&](int kt) {
    wait_slices<kLoadsW + kLoadsE, RING - 2>(slices - 1 - kt);
    const int next = kt + RING - 1;
    if (next < ksteps) issue(next);
    else if (next < slices) issue_adapters(next);
  };
  for (int kt = 0; kt < ksteps; ++kt) {
    begin(kt);
    const u32x4_t* ws = lds + (kt % RING) * kBuffer + (wf * (TF / WF)) * 8;
    const u32x4_t* es = lds + (kt % RING) * kBuffer + (TF + wt * (TT / WT)) * 8;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int kc = (s * 2 + lh) ^ ((lr >> 1) & 7);
      u32x4_t fw[FB], fe[TB];
#pragma unroll
      for (int f = 0; f < FB; ++f) fw[f] = ws[(f * 32 + lr) * 8 + kc];
#pragma unroll
      for (int b = 0; b < TB; ++b) fe[b] = es[(b * 32 + lr) * 8 + kc];
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int f = 0; f < FB; ++f) acc[b][f] = multiply<DT>(fw[f], fe[b], acc[b][f]);
    }
  }
  const u32x4_t zero = {0, 0, 0, 0};
  const int hc = h_columns(DT, a.rank);
  auto both = [&](u32x4_t b, u32x4_t first, u32x4_t second, f32x16_t sums) {   // a block's sums and B with both parts of h
    sums = multiply<DT>(b, first, sums);
    if constexpr (DT == ENGRAM_BF16) sums = multiply<DT>(b, second, sums);
    return sums;
  };
  u32x4_t h0[TB], h1[TB];   // (float32: h0 alone)
  int j = 0, r = -kColumns;   // this wavefront's next adapter, its columns
  bool in = false;
  for (int kt = ksteps; kt < slices; ++kt) {
    begin(kt);
    if (j == 0) {
      r += kColumns;
      in = r + lh * kVals < a.rank;   // (a rank of 8, 24, ..: the last columns' second half is none)
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const char* h = static_cast<const char*>(a.h) + (min(tw0 + b * 32 + lr, a.n_tok - 1) * hc + r + lh * kVals) * kSize;
        h0[b] = load16(h);
        h1[b] = DT == ENGRAM_BF16 ? load16(h + hc) : zero;
        if (!in) h0[b] = h1[b] = zero;
      }
    }
    const u32x4_t* ws = lds + (kt % RING) * kBuffer + (wf * (TF / WF)) * 8;
    int one[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) one[p] = j + p < own ? adapters[wt][j + p] : -2;
    j += kPer;
    if (j >= turns * kPer) j = 0;
    bool mine[TB][kPer], any[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      bool some = false;
#pragma unroll
      for (int p = 0; p < kPer; ++p) some |= mine[b][p] = id[b] == one[p];
      any[b] = __any(some);
    }
#pragma unroll
    for (int f = 0; f < FB; ++f) {
      u32x4_t fw[kPer];
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        fw[p] = ws[(f * 32 + lr) * 8 + (((wt * kPer + p) * 2 + lh) ^ ((lr >> 1) & 7))];
        if (!in) fw[p] = zero;
      }
      uint32_t top = 0;   // an exponent of ones carries into the sign's place
      constexpr uint32_t kExponent = DT == ENGRAM_BF16 ? 0x7f807f80u : 0x7f800000u, kOne = DT == ENGRAM_BF16 ? 0x00800080u : 0x00800000u;
#pragma unroll
      for (int p = 0; p < kPer; ++p)
#pragma unroll
        for (int x = 0; x < 4; ++x) top |= (fw[p][x] & kExponent) + kOne;
      const bool odd = __any((top & (~kExponent & (kExponent + kOne))) != 0);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if (!odd) {        // the other tokens' rows of h as zeros
#pragma unroll
          for (int p = 0; p < kPer; ++p)
            acc[b][f] = both(fw[p], mine[b][p] ? h0[b] : zero, mine[b][p] ? h1[b] : zero, acc[b][f]);
        } else if (any[b]) {
          // an infinity or a NaN in B: a lane's sums are its own token's, it takes its adapter's product and no other's,
          // so that one request's bad adapter stays with it
#pragma unroll
          for (int p = 0; p < kPer; ++p) {
            const f32x16_t sum = both(fw[p], h0[b], h1[b], acc[b][f]);
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[b][f][x] = mine[b][p] ? sum[x] : acc[b][f][x];
          }
        }
      }
    }
  }
  const int64_t fw0 = f0 + wf * (TF / WF);
  // outputs: a block of 32 tokens at a time through the wavefront's own LDS, whole rows of it to memory
  __syncthreads();
  constexpr int kRow = FB * 32 * static_cast<int>(sizeof(OutT)) + 16;   // bytes, 16 more than a row's: the rows' banks differ
  constexpr int kRuns = FB * 32 * static_cast<int>(sizeof(OutT)) / 16;  // 16-byte runs of a row
  constexpr int kEach = 16 / static_cast<int>(sizeof(OutT));
  char* mem = reinterpret_cast<char*>(lds) + wave * 32 * kRow;
#pragma unroll
  for (int b = 0; b < TB; ++b) {
#pragma unroll
    for (int f = 0; f < FB; ++f)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        char* to = mem + lr * kRow + (f * 32 + g * 8 + lh * 4) * static_cast<int>(sizeof(OutT));
        const f32x16_t& x = acc[b][f];
        if constexpr (sizeof(OutT) == 2)
          *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(x[4 * g], x[4 * g + 1]), pack_bf16x2(x[4 * g + 2], x[4 * g + 3]));
        else
          *reinterpret_cast<f32x4_t*>(to) = f32x4_t{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wavefront's block is in LDS
#pragma unroll
    for (int i = 0; i < 32 * kRuns / 64; ++i) {
      const int run = i * 64 + lane, row = run / kRuns, c = run % kRuns;
      const int64_t t = tw0 + b * 32 + row, o = fw0 + c * kEach;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mem + row * kRow + c * 16);
      if (t < a.n_tok && o < a.n_out) *reinterpret_cast<u32x4_t*>(static_cast<OutT*>(a.out) + t * a.n_out + o) = v;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // and read, before the next block's writes
  }
}

// launch(arguments, number of workgroups) for all of them, each launch a stage.
template <typename F>
hipError_t launch_groups(AdaptArgs a, int64_t groups, const char* stage, F launch) {
  if (groups > INT32_MAX) return hipErrorInvalidConfiguration;
  for (int64_t first = 0; first < groups; first += kMostGroups) {
    prof_stage(stage);
    a.first = static_cast<uint32_t>(first);
    launch(a, std::min(kMostGroups, groups - first));
    const hipError_t e = launch_error();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int TF, int TT, int WF, int WT, int RING, typename OutT>
hipError_t launch_tile(const AdaptArgs& a, hipStream_t s) {
  constexpr int kOut = WF * WT * 32 * (TF / WF * static_cast<int>(sizeof(OutT)) + 16);
  constexpr int kLds = std::max(RING * (TF + TT) * 128, kOut);
  auto* const fn = adapt_tile_kernel<DT, TF, TT, WF, WT, RING, OutT>;
  static std::atomic<uint64_t> attr_set{0};   // > 64 KiB of dynamic LDS, raised once per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if ((attr_set.load(std::memory_order_acquire) & bit) == 0) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_release);
  }
  const int tiles_f = static_cast<int>((int64_t{a.n_out} + TF - 1) / TF), tiles_t = static_cast<int>((a.n_tok + TT - 1) / TT);
  return launch_groups(a, static_cast<int64_t>(tiles_f) * tiles_t, "project_adapted_kernel", [&](const AdaptArgs& b, int64_t groups) {
    launch_k(fn, dim3(static_cast<unsigned>((groups + kXcds - 1) / kXcds * kXcds)), dim3(WF * WT * 64), kLds, s, b, tiles_f, tiles_t);
  });
}

template <int DT, int NW, typename OutT>
hipError_t launch_small(const AdaptArgs& a, hipStream_t s) {
  const int tiles_f = a.n_out / 32;
  return launch_groups(a, (a.n_tok + 31) / 32 * tiles_f, "project_adapted_kernel", [&](const AdaptArgs& b, int64_t groups) {
    launch_k((adapt_small_kernel<DT, NW, OutT>), dim3(static_cast<unsigned>(groups)), dim3(NW * 64), 0, s, b, tiles_f);
  });
}

template <typename OutT>
hipError_t launch_product(const AdaptArgs& a, int dtype, hipStream_t s) {
  const int64_t t = a.n_tok, o = a.n_out;
  // The adapters that 64 tokens may meet.  Each one's B is more columns for a tile, so many favour small tiles.
  const int64_t spread = std::min<int64_t>({a.adapters, 64, (62 + a.per) / a.per + 1});
  auto tiles = [&](int64_t side) { return (t + side - 1) / side * ((o + side - 1) / side); };
  // workgroups of a tile by turns on the GPU's 256 CUs
  auto rounds = [&](int64_t side) { return (tiles(side) + 255) / 256; };
  if (dtype == ENGRAM_F32) {
    if constexpr (sizeof(OutT) == 4) {
      // Too few tiles of 64: 256 x 1024 x 1024 23 us so and 25 in tiles (64 adapters: 27 and 47), 64 x 1024 x 5120 36 and 25.
      if (tiles(32) <= 256) return launch_small<ENGRAM_F32, 8, float>(a, s);
      // A tile of 128 takes as long as three of 64: 512 x 1024 x 5120 66 us in tiles of 64, 74 of 128; 1024 x 1024 x 2048 44
      // and 73, x 5120 108 and 134; 4096 x 1024 x 2048 163 and 136.
      if (rounds(64) < 3 * rounds(128)) return launch_tile<ENGRAM_F32, 64, 64, 2, 2, 4, float>(a, s);
      return launch_tile<ENGRAM_F32, 128, 128, 2, 2, 2, float>(a, s);
    }
    return hipErrorInvalidValue;
  }
  const bool many = spread > 8;
  // At 32 x 1024 x 20480 15 us so and 18 in tiles of 64; 64 adapters: 256 x 1024 x 2048 13 and 16.5, 128 x 1024 x 5120 18.4
  // and 17.1; 4 adapters: 256 x 1024 x 1024 6 and 9, x 2048 10.1 and 9.4.
  if (t <= 32 || tiles(32) <= (many ? 512 : 256)) return launch_small<ENGRAM_BF16, 16, OutT>(a, s);
  // While the tiles of 64 all have their place on the chip: 1024 x 1024 x 2048 12 us (128: 16.5), 512 x 1024 x 5120 18 (15);
  // 64 adapters: 512 x 1024 x 5120 34 (43), 2048 x 1024 x 5120 94 (90).
  if (tiles(64) <= (many ? 1024 : 512)) return launch_tile<ENGRAM_BF16, 64, 64, 2, 2, 4, OutT>(a, s);
  // Tiles of 256 where the last turn is mostly filled: 8192 x 1024 x 2048 37 us (128: 43), 32763 x 1024 x 5120 346 (409), 5120 x
  // 1024 x 5120 68 (71), but 3584 x 1024 x 5120 61 (51); 64 adapters: 371 (268) at 8192 x 1024 x 5120.
  if (many || tiles(256) * 4 < rounds(256) * 256 * 3) return launch_tile<ENGRAM_BF16, 128, 128, 2, 2, 2, OutT>(a, s);
  return launch_tile<ENGRAM_BF16, 256, 256, 2, 4, 2, OutT>(a, s);
}

}  // namespace

size_t adapt_workspace(int64_t n_tok, int dtype, int rank) {
  return static_cast<size_t>(n_tok) * h_columns(dtype, rank) * (dtype == ENGRAM_BF16 ? 2 : 4);
}

hipError_t launch_project_adapted(const void* e, const void* w, int64_t n_tok, int64_t d_mem, int64_t n_out, int dtype, const void* lora_a,
                                  const void* lora_b, const float* scale, int32_t rank, int32_t adapters, const int32_t* which, int64_t per,
                                  int out_dtype, void* out, void* ws, hipStream_t s) {
  if (n_tok == 0) return hipSuccess;
  per = std::min(per, n_tok);
  const AdaptArgs a{e, w, lora_a, lora_b, scale, which, ws, out, n_tok, static_cast<uint32_t>(per), static_cast<int32_t>(d_mem),
                    static_cast<int32_t>(n_out), rank, adapters, 0};
  if (adapters > 0) {
    // a block of 32 tokens meets at most so many requests, each with one adapter
    const int64_t most = std::min<int64_t>({32, adapters, (30 + per) / per + 1});
    const unsigned rows = static_cast<unsigned>((most * rank + 31) / 32);
    // few workgroups: more wavefronts for the columns of each (bf16, 256 tokens of 16 adapters: 5.4 us with 16, 6.4 with 4;
    // 2048: 18 and 14; float32, one wavefront's share longer: 64 tokens 10 with 8, 12.6 with 4)
    const bool few = n_tok <= 512;
    const hipError_t r = launch_groups(a, (n_tok + 31) / 32, "adapter_rows_kernel", [&](const AdaptArgs& b, int64_t groups) {
      const dim3 grid(static_cast<unsigned>(groups), rows);
      if (dtype == ENGRAM_F32) launch_k(few ? adapter_rows_kernel<ENGRAM_F32, 8> : adapter_rows_kernel<ENGRAM_F32, 4>, grid, dim3(few ? 512 : 256), 0, s, b);
      else launch_k(few ? adapter_rows_kernel<ENGRAM_BF16, 16> : adapter_rows_kernel<ENGRAM_BF16, 4>, grid, dim3(few ? 1024 : 256), 0, s, b);
    });
    if (r != hipSuccess) return r;
  }
  return out_dtype == ENGRAM_BF16 ? launch_product<uint16_t>(a, dtype, s) : launch_product<float>(a, dtype, s);
}

}  // namespace engram
