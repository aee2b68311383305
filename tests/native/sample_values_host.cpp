// Host build of the rule that picks a bf16 row's table of weights
// (sample_values.h), for every exponent that a row's largest logit can have; run
// by tests/test_around_host.py.
#include <cstdio>

#include "sample_values.h"

int main() {
  using namespace engram;
  int failures = 0;
  for (uint32_t exponent = 0; exponent < 255; ++exponent) {
    const int64_t first = first_value(exponent, false), end = first + kValues;   // bits of magnitudes, 128 an exponent
    const int64_t last = exponent < 133 ? 133 : exponent;
    bool ok = first == (last - kExponents + 1) * 128 && end == (last + 1) * 128;
    // the largest logit's own magnitudes are in it unless they are below all of it; no infinity and no NaN is
    ok = ok && (exponent < 133 - kExponents + 1 || (first <= exponent * 128 && exponent * 128 + 127 < end)) && end <= 0x7f80;
    // rows below 128 in magnitude share one table
    ok = ok && (first_value(exponent, false) == kFirstBase) == (exponent < 127 + 7);
    if (!ok) {
      std::printf("FAILED exponent %u: values from %lld\n", exponent, static_cast<long long>(first));
      ++failures;
    }
  }
  if (first_value(0, true) != 0) {
    std::printf("FAILED zeros\n");
    ++failures;
  }
  if (failures == 0) std::printf("all passed\n");
  return failures != 0;
}
