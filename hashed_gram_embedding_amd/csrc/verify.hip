// Token probabilities and the verification of drafted tokens: the end of a
// speculative decode step whose layers ran over the drafted chunk.
#include "device_util.h"
#include "engram_internal.h"

namespace engram {
namespace {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float load_f32(const void* x, int64_t i, int dtype) {
  return dtype == ENGRAM_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
  return x;
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// ---- probabilities ----
// One workgroup per row: largest logit, sum of exponentials, probabilities.
// p_v = e^((l_v - max) / T) / sum; at T <= 0 the lowest index of the largest
// logit has probability 1.  A row of -inf alone has probabilities 0; one with
// a NaN has NaN throughout, and so has one with +inf at T > 0.
__global__ void __launch_bounds__(256)
probs_kernel(const void* __restrict__ logits, int dtype, int64_t V, int64_t ld, const float* __restrict__ temperature,
             int64_t per, float* __restrict__ probs) {
  __shared__ float red[4];
  __shared__ int64_t first[4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t in = row * ld;
  float* out = probs + row * V;
  const float temp = temperature != nullptr ? temperature[row / per] : 1.0f;
  float mx = -__builtin_inff();
  bool nan = false;
  for (int64_t v = tid; v < V; v += 256) {
    const float l = load_f32(logits, in + v, dtype);
    nan |= l != l;
    mx = fmaxf(mx, l);
  }
  nan = __syncthreads_or(nan);
  mx = wave_max(mx);
  if ((tid & 63) == 0) red[tid >> 6] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  if (nan || mx == -__builtin_inff() || (mx == __builtin_inff() && temp > 0.f)) {
    const float fill = !nan && mx < 0.f ? 0.f : __builtin_nanf("");
    for (int64_t v = tid; v < V; v += 256) out[v] = fill;
    return;
  }
  if (!(temp > 0.f)) {
    int64_t at = V;
    for (int64_t v = tid; v < V && at == V; v += 256)
      if (load_f32(logits, in + v, dtype) == mx) at = v;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) at = min(at, static_cast<int64_t>(__shfl_xor(static_cast<long long>(at), off, 64)));
    if ((tid & 63) == 0) first[tid >> 6] = at;
    __syncthreads();
    at = min(min(first[0], first[1]), min(first[2], first[3]));
    for (int64_t v = tid; v < V; v += 256) out[v] = v == at ? 1.f : 0.f;
    return;
  }
  const float k = kLog2e / temp;
  float sum = 0.f;
  for (int64_t v = tid; v < V; v += 256) sum += __builtin_amdgcn_exp2f((load_f32(logits, in + v, dtype) - mx) * k);
  sum = wave_sum(sum);
  if ((tid & 63) == 0) red[tid >> 6] = sum;
  __syncthreads();
  sum = (red[0] + red[1]) + (red[2] + red[3]);
  const float inv = 1.0f / sum;
  for (int64_t v = tid; v < V; v += 256) out[v] = __builtin_amdgcn_exp2f((load_f32(logits, in + v, dtype) - mx) * k) * inv;
}

// ---- verification ----
// A draft x_i is accepted while u_i q_i(x_i) < p_i(x_i) (both sides exact in
// double: 24-bit factors).  The next token comes from the row r of the first
// refusal, r = max(p - q, 0), or from p itself behind the last accepted draft
// (and where p - q leaves nothing): the lowest index whose cumulative sum
// passes u * total.  Sums are in double: a border between two tokens then
// moves by about 2^-50 of the total rather than 2^-22.

struct VerifyArgs {
  const void* target;      // [S][G+1][V]
  const void* draft;       // [S][G][V] or null: each draft had probability 1
  const int32_t* drafted;  // [S][G]
  const int32_t* n_draft;  // [S] or null: G each
  const float* u_accept;   // [S][G]
  const float* u_sample;   // [S]
  int32_t* tokens;         // [S][G+1]
  int32_t* n_accepted;     // [S]
  double2* part;           // [S][chunks]: sums of max(p - q, 0) and of p
  int64_t V;
  int G;
  int dtype;
  int chunks;
};

constexpr int kPerThread = 16;
constexpr int kChunk = 256 * kPerThread;

// Accepted drafts of sequence s, and whether one was refused.  Every
// wavefront of the workgroup computes it: lane i looks at draft i.
__device__ __forceinline__ int accepted(const VerifyArgs& a, int64_t s, bool* refused) {
  const int lane = threadIdx.x & 63;
  const int n = a.n_draft != nullptr ? min(max(a.n_draft[s], 0), a.G) : a.G;
  bool ok = true;
  if (lane < n) {
    const int32_t x = a.drafted[s * a.G + lane];
    ok = x >= 0 && x < a.V;
    if (ok) {
      const double p = load_f32(a.target, (s * (a.G + 1) + lane) * a.V + x, a.dtype);
      const double q = a.draft != nullptr ? load_f32(a.draft, (s * a.G + lane) * a.V + x, a.dtype) : 1.0f;
      ok = static_cast<double>(a.u_accept[s * a.G + lane]) * q < p;
    }
  }
  const uint64_t bad = __ballot(lane < n && !ok);
  *refused = bad != 0;
  return bad != 0 ? __builtin_ctzll(bad) : n;
}

// max(p_v - q_v, 0) and p_v of one entry; a NaN counts as nothing.
struct Rest {
  const void* p;
  const void* q;    // null: none, or a draft without probabilities
  int64_t p0, q0;   // first entry of the row
  int64_t drop;     // token with draft probability 1, or -1
  int dtype;
  __device__ __forceinline__ double2 at(int64_t v) const {
    const double pv = load_f32(p, p0 + v, dtype);
    double d = pv;
    if (q != nullptr) d -= static_cast<double>(load_f32(q, q0 + v, dtype));
    if (v == drop) d = 0.0;
    return make_double2(d > 0.0 ? d : 0.0, pv > 0.0 ? pv : 0.0);
  }
};

__device__ __forceinline__ Rest rest_of(const VerifyArgs& a, int64_t s, int acc, bool refused) {
  Rest r{a.target, refused ? a.draft : nullptr, (s * (a.G + 1) + acc) * a.V, (s * a.G + acc) * a.V, -1, a.dtype};
  if (refused && a.draft == nullptr) r.drop = a.drafted[s * a.G + acc];
  return r;
}

__global__ void __launch_bounds__(256)
verify_sums_kernel(VerifyArgs a) {
  __shared__ double2 red[4];
  const int64_t s = blockIdx.y;
  const int tid = threadIdx.x;
  bool refused;
  const int acc = accepted(a, s, &refused);
  const Rest r = rest_of(a, s, acc, refused);
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kChunk;
  double rest = 0.0, row = 0.0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t v = v0 + i * 256 + tid;
    if (v < a.V) {
      const double2 d = r.at(v);
      rest += d.x;
      row += d.y;
    }
  }
  rest = wave_sum64(rest);
  row = wave_sum64(row);
  if ((tid & 63) == 0) red[tid >> 6] = make_double2(rest, row);
  __syncthreads();
  if (tid == 0)
    a.part[s * a.chunks + blockIdx.x] = make_double2((red[0].x + red[1].x) + (red[2].x + red[3].x),
                                                     (red[0].y + red[1].y) + (red[2].y + red[3].y));
}

// Inclusive sum over the lanes of a wavefront.
__device__ __forceinline__ double wave_scan64(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(256)
verify_pick_kernel(VerifyArgs a) {
  __shared__ double wsum[4];
  __shared__ int found[4], last[4];
  __shared__ int chunk_s;
  __shared__ double left_s;
  __shared__ int use_row_s;
  const int64_t s = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  bool refused;
  const int acc = accepted(a, s, &refused);
  const Rest r = rest_of(a, s, acc, refused);
  if (tid == 0) {
    const double2* part = a.part + s * a.chunks;
    double rest = 0.0, row = 0.0;
    for (int c = 0; c < a.chunks; ++c) {
      rest += part[c].x;
      row += part[c].y;
    }
    const bool use_row = !(rest > 0.0);
    const double total = use_row ? row : rest;
    const double want = static_cast<double>(a.u_sample[s]) * total;
    int chunk = -1, end = -1;
    double before = 0.0, left = 0.0;
    if (total > 0.0 && total < __builtin_inf()) {
      for (int c = 0; c < a.chunks && chunk < 0; ++c) {
        const double x = use_row ? part[c].y : part[c].x;
        if (before + x > want) {
          chunk = c;
          left = before;
        } else {
          before += x;
        }
        if (x > 0.0) end = c;
      }
      if (chunk < 0) {   // u not below 1: the last token that has any probability
        chunk = end;
        left = __builtin_inf();
      }
    }
    chunk_s = chunk;
    left_s = left;
    use_row_s = use_row;
    wsum[0] = want;
  }
  __syncthreads();
  const int chunk = chunk_s;
  const double want = wsum[0], left = left_s;
  const bool use_row = use_row_s != 0;
  __syncthreads();
  int32_t token = -1;
  if (chunk >= 0) {
    const int64_t v0 = static_cast<int64_t>(chunk) * kChunk + tid * kPerThread;
    double x[kPerThread], sum = 0.0;
    int end = -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      x[i] = 0.0;
      if (v0 + i < a.V) {
        const double2 d = r.at(v0 + i);
        x[i] = use_row ? d.y : d.x;
      }
      if (x[i] > 0.0) end = tid * kPerThread + i;
      sum += x[i];
    }
    const double scan = wave_scan64(sum);
    if (lane == 63) wsum[wave] = scan;
    __syncthreads();
    double run = left + (scan - sum);
    for (int w = 0; w < wave; ++w) run += wsum[w];
    int at = kChunk;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      run += x[i];
      if (at == kChunk && x[i] > 0.0 && run > want && left < __builtin_inf()) at = tid * kPerThread + i;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      at = min(at, __shfl_xor(at, off, 64));
      end = max(end, __shfl_xor(end, off, 64));
    }
    if (lane == 0) {
      found[wave] = at;
      last[wave] = end;
    }
    __syncthreads();
    at = min(min(found[0], found[1]), min(found[2], found[3]));
    end = max(max(last[0], last[1]), max(last[2], last[3]));
    // the chunk's sum was formed in another order: by a last bit it may not
    // reach what it reached there
    token = static_cast<int32_t>(static_cast<int64_t>(chunk) * kChunk + (at < kChunk ? at : end));
  }
  if (tid == 0) a.n_accepted[s] = acc;
  for (int i = tid; i <= a.G; i += 256) a.tokens[s * (a.G + 1) + i] = i < acc ? a.drafted[s * a.G + i] : (i == acc ? token : -1);
}

}  // namespace

size_t probs_workspace(int64_t, int64_t) { return 0; }

hipError_t launch_token_probs(const void* logits, int dtype, int64_t rows, int64_t V, int64_t ld, const float* temperature,
                              int64_t per, float* probs, void*, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  launch_k(probs_kernel, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, logits, dtype, V, ld, temperature, per, probs);
  return hipGetLastError();
}

size_t verify_workspace(int64_t S, int64_t V) { return static_cast<size_t>(S) * ((V + kChunk - 1) / kChunk) * sizeof(double2); }

hipError_t launch_verify(const void* target, const void* draft, int dtype, const int32_t* drafted, const int32_t* n_draft,
                         const float* u_accept, const float* u_sample, int64_t S, int32_t G, int64_t V, int32_t* tokens,
                         int32_t* n_accepted, void* ws, hipStream_t s) {
  if (S == 0) return hipSuccess;
  const int chunks = static_cast<int>((V + kChunk - 1) / kChunk);
  const VerifyArgs a{target, draft, drafted, n_draft, u_accept, u_sample, tokens, n_accepted, static_cast<double2*>(ws),
                     V, G, dtype, chunks};
  launch_k(verify_sums_kernel, dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(S)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_k(verify_pick_kernel, dim3(static_cast<unsigned>(S)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace engram
