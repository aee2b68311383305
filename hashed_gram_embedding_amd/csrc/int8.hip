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
#include "device_util.h"
#include "engram_internal.h"

namespace engram {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// ---- quantisation of rows ----

__device__ __forceinline__ float load_f32(const void* x, int64_t i, int dtype) {
  return dtype == ENGRAM_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
}

// rne(127 x / top) of exact arithmetic, for |x| <= top.  x * (127 / top) in
// float is off by less than 2^-15; only where that could change the rounding
// (or 127 / top overflows: top below 2^-120) is the quotient formed in
// double, whose error of 2^-53 cannot: 127 x / top is a ratio of numbers of
// 31 and 24 bits, so it is a tie or at least 2^-26 away from one.
__device__ __forceinline__ int quantize(float x, float top, float inv) {
  const float y = x * inv;
  float r = rintf(y);
  if (!(fabsf(y - r) < 0.5f - 1.0f / 8192.0f)) r = static_cast<float>(rint(static_cast<double>(x) * 127.0 / static_cast<double>(top)));
  return static_cast<int>(r);
}

// One row per group of THREADS lanes.  Codes go to q [rows][ldq].  With
// `tail` the last, incomplete run of 16 columns is stored right-aligned in
// its 16 bytes (zeros before it): the product reads W's last 16 columns there
// (load_chunk) and the zeros leave out those already counted.  A row of zeros
// has scale 0; one holding an infinity or a NaN has codes 0 and scale NaN, so
// its products are NaN.
template <int THREADS>
__global__ void __launch_bounds__(256)
quantize_kernel(const void* __restrict__ x, int dtype, int64_t rows, int cols, int8_t* __restrict__ q, int64_t ldq,
                int tail, float* __restrict__ scale) {
  __shared__ uint32_t part[4];
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / THREADS;
  const int t = threadIdx.x % THREADS;
  if (row >= rows) return;   // whole groups leave together
  const int64_t base = row * cols;
  // largest magnitude by its bits: an infinity and a NaN order above every
  // finite value
  uint32_t top = 0;
  for (int c = t; c < cols; c += THREADS) top = max(top, __float_as_uint(load_f32(x, base + c, dtype)) & 0x7fffffffu);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, 64)));
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  const bool finite = top < 0x7f800000u;
  const float ft = __uint_as_float(top);
  const float inv = 127.0f / ft;
  if (t == 0) scale[row] = finite ? ft / 127.0f : __uint_as_float(0x7fc00000u);
  const int whole = tail ? cols / 16 * 16 : cols;
  const int shift = tail && whole < cols ? 16 - (cols - whole) : 0;
  int8_t* dst = q + row * ldq;
  for (int c = t; c < cols; c += THREADS) {
    const float v = load_f32(x, base + c, dtype);
    const int code = top != 0 && finite ? quantize(v, ft, inv) : 0;
    dst[c < whole ? c : c + shift] = static_cast<int8_t>(code);
  }
  if (t < shift) dst[whole + t] = 0;
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
};

// 16 columns of a row of K bytes, chunk c, from any alignment.  A last chunk
// that is not whole reads the row's last 16 bytes instead (rows of fewer than
// 16 are read byte by byte, right-aligned); the other operand holds zeros for
// the columns that are then read twice.
__device__ __forceinline__ u32x4_t load_chunk(const int8_t* row, int c, int K) {
  u32x4_t v{0, 0, 0, 0};
  if (K >= 16) {
    __builtin_memcpy(&v, row + min(c * 16, K - 16), 16);
  } else {
    for (int i = 0; i < K; ++i) {
      const int b = 16 - K + i;
      v[b >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[i])) << (8 * (b & 3));
    }
  }
  return v;
}

// The same of a token row, with the columns counted before cleared.
__device__ __forceinline__ u32x4_t load_chunk_once(const int8_t* row, int c, int K) {
  u32x4_t v = load_chunk(row, c, K);
  const int twice = c * 16 + 16 - K;   // leading bytes that an earlier chunk holds
  if (twice > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(max(twice - 4 * i, 0), 4);
      v[i] = n == 4 ? 0u : v[i] & (0xffffffffu << (8 * n));
    }
  }
  return v;
}

template <typename OutT>
__device__ __forceinline__ OutT to_out(float f) {
  if constexpr (sizeof(OutT) == 2) return f32_to_bf16(f);
  else return f;
}

// General product: any K and alignment.  64 tokens x 64 outputs per workgroup
// of four wavefronts, 32 x 32 each on v_mfma_i32_32x32x32_i8; 64 columns a
// step through registers into LDS.
template <typename OutT>
__global__ void __launch_bounds__(256)
project_i8_kernel(ProjectI8Args a) {
  __shared__ u32x4_t Ws[64 * 4], Qs[64 * 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles_n = static_cast<int>((a.n_out + 63) / 64);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % tiles_n) * 64, t0 = static_cast<int64_t>(blockIdx.x / tiles_n) * 64;
  const int chunks = (a.K + 15) / 16;
  const int r = tid >> 2, cc = tid & 3;
  const int8_t* wrow = a.w + min(n0 + r, a.n_out - 1) * a.K;
  const int8_t* qrow = a.q + min(t0 + r, a.n_tok - 1) * a.ldq;
  i32x16_t acc{};
  for (int c0 = 0; c0 < chunks; c0 += 4) {
    const int c = c0 + cc;
    u32x4_t vw{0, 0, 0, 0}, vq{0, 0, 0, 0};
    if (c < chunks) {
      vw = load_chunk(wrow, c, a.K);
      vq = a.tailed ? *reinterpret_cast<const u32x4_t*>(qrow + c * 16) : load_chunk_once(qrow, c, a.K);
    }
    __syncthreads();
    Ws[r * 4 + (cc ^ (r & 3))] = vw;
    Qs[r * 4 + (cc ^ (r & 3))] = vq;
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int kc = ks * 2 + (lane >> 5);
      const int rw = (wave & 1) * 32 + (lane & 31), rq = (wave >> 1) * 32 + (lane & 31);
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, Ws[rw * 4 + (kc ^ (rw & 3))]),
                                                  __builtin_bit_cast(i32x4_t, Qs[rq * 4 + (kc ^ (rq & 3))]), acc, 0, 0, 0);
    }
  }
  const int64_t tok = t0 + (wave >> 1) * 32 + (lane & 31);
  if (tok >= a.n_tok) return;
  const float st = a.q_scale[tok];
  OutT* out = static_cast<OutT*>(a.out) + tok * a.n_out;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t o = n0 + (wave & 1) * 32 + (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3);
    if (o < a.n_out) out[o] = to_out<OutT>(static_cast<float>(acc[i]) * st * a.w_scale[o]);
  }
}

}  // namespace

int64_t i8_row_stride(int64_t cols) { return (cols + 15) / 16 * 16; }

hipError_t launch_quantize_i8(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* q, int64_t ldq, bool tail,
                              float* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int c = static_cast<int>(cols);
  if (cols <= 2048)
    launch_k(quantize_kernel<64>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s, x, dtype, rows, c, q, ldq,
             tail ? 1 : 0, scale);
  else
    launch_k(quantize_kernel<256>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, x, dtype, rows, c, q, ldq,
             tail ? 1 : 0, scale);
  return hipGetLastError();
}

hipError_t launch_project_i8(const int8_t* q, int64_t ldq, bool tailed, const float* q_scale, const int8_t* w,
                             const float* w_scale, int64_t n_tok, int64_t K, int64_t n_out, int out_dtype, void* out,
                             hipStream_t s) {
  if (n_tok == 0) return hipSuccess;
  const ProjectI8Args a{q, q_scale, w, w_scale, out, n_tok, ldq, n_out, static_cast<int>(K), tailed ? 1 : 0};
  const int64_t tiles = ((n_out + 63) / 64) * ((n_tok + 63) / 64);
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  if (out_dtype == ENGRAM_BF16) launch_k(project_i8_kernel<uint16_t>, grid, dim3(256), 0, s, a);
  else launch_k(project_i8_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace engram
