// e4m3.cuh -- e4m3 codes to bf16, exactly: the code's bits s eeee mmm placed as
// the bf16 s 0000eeee mmm0000 are the value * 2^-120 (a subnormal code becomes a
// subnormal bf16), so one product by 2^120, or by 2^120 times a power-of-two
// scale, gives the value.
#pragma once
#include <cstdint>

namespace attn {

constexpr uint32_t kExpNaN = 255u;  // exponent byte of a row that held an infinity or a NaN

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The codes in bytes 1 and 3 of x.
__device__ __forceinline__ uint32_t e4m3_hi_bits(uint32_t x) { return ((x >> 4) & 0x07F007F0u) | (x & 0x80008000u); }

// The product that takes a code's bits to code * 2^(exp - 127): by m = 2^(exp - 7),
// which bf16 holds up to exp 134, and above that by `more` as well (1 below).
// exp 255 gives NaN, exp 0 (a row that is not there) gives zero.
struct E4m3Factor {
  uint32_t m, more;
};
__device__ __forceinline__ E4m3Factor e4m3_factor(uint32_t e) {
  const uint32_t k = e > 134u ? 134u : e;
  // 2^(k - 7): biased exponent k + 120; 0 for k = 0
  const uint32_t m = e == kExpNaN ? 0x7FFFu : (k == 0u ? 0u : (k + 120u) << 7);
  const uint32_t more = (127u + (e - k)) << 7;
  return E4m3Factor{m | (m << 16), e == kExpNaN ? 0x7FFF7FFFu : more | (more << 16)};
}

}  // namespace attn
