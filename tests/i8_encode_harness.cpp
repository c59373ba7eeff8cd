// CPU harness for the int8 row codec (csrc/i8_codec.h, host + device source): the scale of a row's largest
// magnitude, and the codes of its values, eight and four at a time as the kernels pack them.  Test infrastructure;
// built by tests/test_i8_codec.py with hipcc --cuda-host-only (no GPU code).
#include <stdint.h>

#include "i8_codec.h"

extern "C" float i8_row_scale(uint32_t amax_bits) { return moe::i8_scale(amax_bits); }
template <bool BF16>
static void codes(float scale, const float* v, uint32_t n4, uint32_t* out) {
  const moe::Scale s(scale);
  uint32_t i = 0;
  for (; i + 2 <= n4; i += 2) moe::i8_pack<2, BF16>(v + 4 * i, s, out + i);
  for (; i < n4; ++i) moe::i8_pack<1, BF16>(v + 4 * i, s, out + i);
}
extern "C" void i8_row_codes(float scale, const float* v, uint32_t n4, uint32_t* out) {
  codes<false>(scale, v, n4, out);
}
extern "C" void i8_row_codes_bf16(float scale, const float* v, uint32_t n4, uint32_t* out) {
  codes<true>(scale, v, n4, out);
}
