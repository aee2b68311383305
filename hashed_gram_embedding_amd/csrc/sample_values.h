// Which logits a bf16 row's table of weights holds (plain C++: the device code
// and a host test use it).
#pragma once

#include <cstdint>

namespace engram {

// bf16 logits take few values: a table holds those of kExponents powers of two,
// of both signs, 128 a power.
constexpr int kExponents = 15, kValues = kExponents << 7;

// Bits of the smallest magnitude in the table of a row whose largest logit has
// this biased exponent: the powers up to that logit's, and no fewer than those
// up to [64, 128), the table of a row whose logits lie near zero or below it.
// zeros: of a row of little but zeros, whose table begins with them.
constexpr uint32_t first_value(uint32_t exponent, bool zeros) {
  const uint32_t last = exponent > 127 + 6 ? exponent : 127 + 6;
  return zeros ? 0 : (last + 1) * 128 - kValues;
}

constexpr uint32_t kFirstBase = first_value(0, false);   // of rows whose largest logit is below 128 in magnitude

}  // namespace engram
