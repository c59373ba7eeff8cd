// CPU harness for the int8 row codec (csrc/i8_codec.h, host + device source): the scale of a row's largest
// magnitude, and the codes of its values, four at a time as the kernels pack them.  Test infrastructure;
// built by tests/test_i8_codec.py with hipcc --cuda-host-only (no GPU code).
#include <stdint.h>

#include "i8_codec.h"

extern "C" float i8_row_scale(uint32_t amax_bits) { return moe::i8_scale(amax_bits); }
extern "C" void i8_row_codes(float scale, const float* v, uint32_t n4, uint32_t* out) {
  const moe::Scale s(scale);
  for (uint32_t i = 0; i < n4; ++i) out[i] = moe::i8_pack4(v + 4 * i, s);
}
