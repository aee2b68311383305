// Host-side exercise of the entry points around the layer for the address and
// undefined-behaviour sanitizers: sizing calls over the ends of their ranges,
// and calls that the host checks must reject (no GPU is touched).
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
  const std::initializer_list<int64_t> ends = {kMin, -1, 0, 1, 7, 8, 64, 4096, 16384, 16385, 65535, 65536, 1 << 28, (1 << 28) + 1, kInt, kInt + 1, kMax};
  for (int64_t a : ends)
    for (int64_t b : ends) {
      const size_t g = engram_embed_backward_workspace(a, b);
      EXPECT((g == 0) == (a < 1 || a > (1 << 28) || b < 1 || b > 65536));
      for (engram_dtype dt : {ENGRAM_F32, ENGRAM_BF16, ENGRAM_I8}) {
        const int32_t rank = static_cast<int32_t>(b < -1000 ? -1000 : b > 1000 ? 1000 : b);
        const size_t n = engram_project_adapted_workspace(a, dt, rank);
        EXPECT((n == 0) == (a < 1 || a > kInt || rank < 8 || rank > 128 || dt == ENGRAM_I8));
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
  engram_adapters ad{3, 8, fake(0x50000), fake(0x60000), nullptr};
  for (engram_dtype dt : {ENGRAM_F32, ENGRAM_BF16})
    for (int d : {1, 64, 4096, 65536, 1 << 30})
      for (int m : {0, 1, 64, 65})
        for (int dim : {0, 1, 16, 1 << 30})
          for (int rank : {0, 8, 128, 136}) {
            L.tables.dim = dim;
            ad.rank = rank;
            L.gc = engram_gate_conv_params{d, m, 4, 3, 1e-6f, dt, static_cast<const float*>(fake(0x20000))};
            for (int64_t b : ends)
              for (int64_t t : {int64_t{-1}, int64_t{0}, int64_t{1}, int64_t{9}, kInt, kInt + 1, kMax}) {
                const size_t n = engram_forward_adapted_workspace(b, t, &L, &ad);
                if (b < 0 || b > 65535 || t < 0 || t > kInt || dim < 1 || m < 1 || m > 64 || rank < 8 || rank > 128) EXPECT(n == 0);
              }
          }
  L.tables.dim = 16;
  ad.rank = 8;
  L.gc = engram_gate_conv_params{64, 1, 4, 3, 1e-6f, ENGRAM_F32, static_cast<const float*>(fake(0x20000))};

  // refused calls
  void* p = fake(0x40000);
  int32_t* ip = static_cast<int32_t*>(p);
  float* fp = static_cast<float*>(p);
  EXPECT(engram_embed(ip, kMax, p, ENGRAM_F32, 10, 16, 1.f, 1, ENGRAM_F32, p, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_embed(ip, 4, p, ENGRAM_F32, kMax, kMax, 1.f, 1, ENGRAM_F32, p, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_embed(ip, 4, p, ENGRAM_F32, 10, kMin, 1.f, 1, ENGRAM_F32, p, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_embed(ip, 0, nullptr, ENGRAM_F32, 10, 16, 1.f, 1, ENGRAM_F32, nullptr, nullptr) == ENGRAM_OK);
  EXPECT(engram_embed_backward(ip, kMax, p, ENGRAM_F32, 10, 16, 1.f, 1, 0, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_embed_backward(ip, 4, p, ENGRAM_F32, 10, 16, 1.f, 1, 0, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_embed_backward(ip, 0, nullptr, ENGRAM_F32, 10, 16, 1.f, 1, 1, ENGRAM_F32, p, nullptr, 0, nullptr) == ENGRAM_OK);
  EXPECT(engram_project_adapted(p, p, kMax, 64, 64, ENGRAM_F32, &ad, ip, 1, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_project_adapted(p, p, 4, 64, 64, ENGRAM_F32, &ad, ip, kMax, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_project_adapted(p, p, 4, 64, 64, ENGRAM_F32, nullptr, ip, 1, ENGRAM_F32, p, p, 0, nullptr) == ENGRAM_EINVAL);
  engram_decode_state st{ip, fp, ip};
  EXPECT(engram_forward_adapted(ip, p, 1, 1, &L, &ad, ip, &st, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EINVAL);
  EXPECT(engram_forward_adapted(ip, p, 65535, kInt, &L, &ad, ip, &st, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_forward_adapted(ip, p, kMax, kMax, &L, &ad, ip, nullptr, nullptr, nullptr, p, 0, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_sample_tokens(p, ENGRAM_F32, kMax, 10, 10, nullptr, nullptr, nullptr, nullptr, 1, fp, ip, fp, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_sample_tokens(p, ENGRAM_F32, 1, kMax, kMax, nullptr, nullptr, nullptr, nullptr, kMax, fp, ip, fp, nullptr) == ENGRAM_EUNSUPPORTED);
  EXPECT(engram_sample_tokens(p, ENGRAM_F32, 1, 10, kMin, nullptr, nullptr, nullptr, nullptr, 1, fp, ip, fp, nullptr) == ENGRAM_EINVAL);
  if (failures == 0) std::printf("all passed\n");
  return failures == 0 ? 0 : 1;
}
