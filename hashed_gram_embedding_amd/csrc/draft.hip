// The decode state after a drafted chunk: engram_forward_draft leaves the
// state as it was, and this takes in the tokens that were kept.
#include "device_util.h"
#include "engram_internal.h"
#include "hash_device.h"

namespace engram {
namespace {

constexpr int kThreads = 1024;

// One workgroup per sequence: pos and ids change when everyone has read them.
// With k kept tokens the ring's slots hold the conv inputs u_t = gamma_t v_t of
// the last min(k, span) of them, the position p = pos + t in slot p % span (as
// after k steps of one token); ids become the last N-1 compressed ids of (ids,
// kept tokens); pos grows by k.  The launch lasts as long as the sequence that
// keeps most: 256 sequences of 8 tokens, d = 1024, 4 branches 4.4 us where each
// keeps one, 8.4 where each keeps all, 7.9 where they keep 1 to 8.
__global__ void __launch_bounds__(kThreads)
commit_draft_kernel(const float* __restrict__ v, int64_t v_stride, const float* __restrict__ gamma, int64_t T,
                    GateConvArgs g, StateArgs st, const int32_t* __restrict__ tokens, const int32_t* __restrict__ proj,
                    int32_t max_n, int32_t vocab, const int32_t* __restrict__ n_accepted, uint32_t* err) {
  const int64_t b = blockIdx.x;
  const int M = g.branches, d = g.d, span = (g.kernel_w - 1) * g.dilation;
  const int64_t kept = min(max(static_cast<int64_t>(n_accepted[b]) + 1, int64_t{0}), T);
  const int64_t pos0 = st.pos[b];
  if (kept == 0) return;
  const int L = static_cast<int>(min(kept, static_cast<int64_t>(span)));
  const int c4 = d / 4;
  const int64_t t0 = kept - L;   // the last L kept tokens
  for (int idx = threadIdx.x; idx < L * c4; idx += kThreads) {
    const int p = idx / c4, cq = idx - p * c4;
    const int64_t row = b * T + t0 + p;
    const float4 x = *reinterpret_cast<const float4*>(v + row * v_stride + cq * 4);
    const int slot = static_cast<int>((pos0 + t0 + p) % span);
    float* dst = st.conv + (b * M * span + slot) * static_cast<int64_t>(d) + cq * 4;
    for (int m = 0; m < M; ++m) {
      const float gm = gamma[row * M + m];
      *reinterpret_cast<float4*>(dst + static_cast<int64_t>(m) * span * d) = make_float4(x.x * gm, x.y * gm, x.z * gm, x.w * gm);
    }
  }
  if (threadIdx.x == 0) {
    const int hl = max_n - 1;
    int32_t next[ENGRAM_MAX_ORDER];
#pragma unroll
    for (int i = 0; i < ENGRAM_MAX_ORDER - 1; ++i) {
      if (i < hl) {
        const int64_t idx = kept + i;   // in (old ids, chunk ids)
        next[i] = idx < hl ? st.ids[b * hl + idx] : proj[token_in_vocab(tokens[b * T + idx - hl], vocab, err)];
      }
    }
#pragma unroll
    for (int i = 0; i < ENGRAM_MAX_ORDER - 1; ++i)
      if (i < hl) st.ids[b * hl + i] = next[i];
  }
  __syncthreads();
  if (threadIdx.x == 0) st.pos[b] = static_cast<int32_t>(pos0 + kept);
}

}  // namespace

hipError_t launch_commit_draft(const float* v, int64_t v_stride, const float* gamma, int64_t B, int64_t T,
                               const GateConvArgs& g, const StateArgs& st, const int32_t* tokens, const int32_t* proj,
                               int32_t max_n, int32_t vocab, const int32_t* n_accepted, uint32_t* err, hipStream_t s) {
  if (B == 0 || T == 0) return hipSuccess;
  launch_k(commit_draft_kernel, dim3(static_cast<unsigned>(B)), dim3(kThreads), 0, s, v, v_stride, gamma, T, g, st, tokens, proj,
           max_n, vocab, n_accepted, err);
  return launch_error();
}

}  // namespace engram
