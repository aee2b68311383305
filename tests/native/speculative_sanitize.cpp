// Host-side exercise of the speculative decode entry points for the address
// and undefined-behaviour sanitizers: sizing calls over the ends of their
// ranges, and calls that the host checks must reject (no GPU is touched).
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>
#include <vector>

#include "engram.h"

static int failures = 0;
#define EXPECT(c)                                                           \
  do {                                                                      \
    if (!(c)) {                                                             \
      std::printf("FAILED line %d: %s (%s)\n", __LINE__, #c, engram_last_error()); \
      ++failures;                                                           \
    }                                                                       \
  } while (0)

static void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }

int main() {
  constexpr int64_t kMax = std::numeric_limits<int64_t>::max(), kMin = std::numeric_limits<int64_t>::min();
  constexpr int64_t kInt = std::numeric_limits<int32_t>::max();
  const std::initializer_list<int64_t> ends = {kMin, -1, 0, 1, 15, 16, 17, 32, 33, 4096, 65535, 65536, 131071, 131072, kInt, kInt + 1, kMax};
  for (int64_t a : ends)
    for (int64_t b : ends) {
      if (a < 1 || b < 1 || a > kInt || b > kInt) EXPECT(engram_token_probs_workspace(a, b) == 0);
      else engram_token_probs_workspace(a, b);
      if (a < 1 || b < 1 || a > 65535 || b > kInt) EXPECT(engram_verify_drafts_workspace(a, b) == 0);
      else EXPECT(engram_verify_drafts_workspace(a, b) <= size_t(65535) * 64 * 8);
      for (int64_t c : ends)
        for (engram_dtype dt : {ENGRAM_F32, ENGRAM_BF16, ENGRAM_I8}) {
          const size_t n = engram_project_i8_workspace(a, b, c, dt);
          if (a < 1 || b < 1 || c < 1 || a > kInt || b > 131071 || c > kInt) EXPECT(n == 0);
        }
    }

  // a layer of fake device pointers (never dereferenced)
  std::vector<uint64_t> mult(2 * 2 * 3, 1);
  uint32_t prime[4] = {1009, 1013, 1019, 1021};
  engram_hash_params hp{static_cast<const int32_t*>(fake(0x1000)), 1000, 3, 2, mult.data(), prime};
  int64_t off[4] = {0, 1009, 2022, 3041}, nrows[4] = {1009, 1013, 1019, 1021};
  engram_tables tab{};
  tab.n_tables = 4; tab.dim = 16; tab.dtype = ENGRAM_F32; tab.rows = fake(0x10000);
  tab.row_offset = off; tab.n_rows = nrows; tab.total_rows = 4062;
  engram_layer L{};
  L.hash = hp; L.tables = tab; L.w = fake(0x30000);
  const engram_i8_weights w8{static_cast<const int8_t*>(fake(0x50000)), static_cast<const float*>(fake(0x60000))};
  for (engram_dtype dt : {ENGRAM_F32, ENGRAM_BF16})
    for (int d : {1, 64, 128, 192, 256, 4096, 8192})
      for (int dim : {0, 1, 16, 128, 256, 512, 1 << 30}) {
        L.tables.dim = dim;
        L.gc = engram_gate_conv_params{d, 4, 4, 3, 1e-6f, dt, static_cast<const float*>(fake(0x20000))};
        for (int64_t b : ends)
          for (int64_t t : {int64_t{-1}, int64_t{0}, int64_t{1}, int64_t{9}, kInt, kInt + 1, kMax}) {
            const size_t i8 = engram_forward_i8_workspace(b, t, &L), dr = engram_forward_draft_workspace(b, t, &L, nullptr),
                         d8 = engram_forward_draft_workspace(b, t, &L, &w8);
            if (b < 0 || b > 65535 || t < 0 || t > kInt || dim < 1) EXPECT(i8 == 0 && dr == 0 && d8 == 0);
          }
        const int64_t stride = engram_draft_stride(&L);
        EXPECT(stride == d || stride == int64_t{5} * d);
      }
  EXPECT(engram_draft_stride(nullptr) == 0 && engram_forward_i8_workspace(1, 1, nullptr) == 0);
  L.tables.dim = 16;
  L.gc = engram_gate_conv_params{64, 1, 4, 3, 1e-6f, ENGRAM_F32, static_cast<const float*>(fake(0x20000))};

  // refused calls
  void* p = fake(0x40000);
  int32_t* ip = static_cast<int32_t*>(p);
  float* fp = static_cast<float*>(p);
  int8_t* bp = static_cast<int8_t*>(p);
  EXPECT(engram_quantize_i8(p, ENGRAM_I8, 1, 1, bp, fp, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_quantize_i8(p, ENGRAM_F32, -1, 1, bp, fp, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_quantize_i8(p, ENGRAM_F32, kMax, kMax, bp, fp, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_project_i8(p, ENGRAM_I8, fp, bp, fp, kMax, 16, 16, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_project_i8(p, ENGRAM_I8, fp, bp, fp, 400, 17, 16, ENGRAM_F32, p, p, 1, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_token_probs(p, ENGRAM_F32, 1, kMax, kMax, nullptr, 1, fp, nullptr, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_token_probs(p, ENGRAM_F32, 1, 40000, 40000, nullptr, kMax, fp, nullptr, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_verify_drafts(p, nullptr, ENGRAM_F32, ip, nullptr, fp, fp, 1, 65, 10, ip, ip, nullptr, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_verify_drafts(p, nullptr, ENGRAM_F32, ip, nullptr, fp, fp, 1, 4, 90000, ip, ip, nullptr, 0, nullptr) == ENGRAM_EINVAL);
  engram_decode_state st{ip, fp, ip};
  engram_draft dr{fp, 64, fp};
  EXPECT(engram_forward_i8(ip, p, 1, 1, &L, nullptr, nullptr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_forward_i8(ip, p, 1, 1, &L, &w8, nullptr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_forward_i8(ip, p, kMax, kMax, &L, &w8, nullptr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_forward_draft(ip, p, 1, 1, &L, nullptr, nullptr, &dr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_forward_draft(ip, p, 1, 1, &L, nullptr, &st, nullptr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_forward_draft(ip, p, 1, 1, &L, nullptr, &st, &dr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);   // stride 128
  EXPECT(engram_commit_draft(ip, 1, 1, &L, &dr, nullptr, &st, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_commit_draft(ip, kMax, 1, &L, &dr, ip, &st, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_commit_draft(ip, 0, 1, &L, &dr, ip, &st, nullptr) == ENGRAM_OK);
  if (failures == 0) std::printf("all passed\n");
  return failures == 0 ? 0 : 1;
}
