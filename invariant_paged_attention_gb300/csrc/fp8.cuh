// The number formats of the 8-bit paged cache: e4m3 codes and one e8m0
// (power-of-two) scale per (key, kv head) row.
//
//   e = the smallest integer >= kMinRowExp with amax(row) <= 448 * 2^e
//   code_d = e4m3(x_d * 2^-e)  (nearest even)      scale byte = e + 127
//   value_d = code_d * 2^e
//
// A power of two costs a floating code no accuracy (scaling by it is exact),
// takes one byte a row, and makes the value exact in bf16: a code has 4
// significant bits, and with e >= -120 its last place (2^(e-9)) is at least
// bf16's smallest subnormal.  (At the top, elements above 248 * 2^120 round to
// the code 256 under e = 120: 2^128, in bf16 an infinity.)  A row's codes and scale depend on that row
// alone, so what a cache holds never depends on batch, page or chunk.
#pragma once

#include <cstdint>

namespace bia {

constexpr int kMinRowExp = -120;
constexpr uint32_t kBf16Inf = 0x7f80u; // |x| bits of an infinity; above it NaN

// Row exponent from the largest finite magnitude (>= 0): 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int ex = static_cast<int>(b >> 23) - 127; // subnormals and zero: below the clamp
  const int e = (b & 0x7fffffu) <= 0x600000u ? ex - 8 : ex - 7;
  return max(e, kMinRowExp);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// Value of an e8m0 byte: 2^(b - 127); 255 is NaN, 0 the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23;
  return __uint_as_float(bits);
}
// Two fp32 -> two e4m3 codes (nearest even, saturating; NaN stays NaN), first
// argument in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes -> two fp32, exactly.
__device__ __forceinline__ void e4m3x2_values(uint32_t codes, float &lo, float &hi) {
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %2;\n\t"
      "mov.b32 {a, b}, h;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "h"(static_cast<uint16_t>(codes)));
}

// ---------------------------------------------------------------- cache policy
// Codes are read once and scales by every head's CTA and, in a randomly paged
// cache, line by line for many keys in turn: the codes' lines leave L2 first.
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_evict_last() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// Loads of scale bytes that bring their whole 128-byte line into L2.
__device__ __forceinline__ uint32_t ld_scale_u8(const uint8_t *p, uint64_t policy) {
  uint16_t v;
  asm("{\n\t.reg .u32 t;\n\t"
      "ld.global.nc.L1::no_allocate.L2::cache_hint.L2::128B.u8 t, [%1], %2;\n\t"
      "cvt.u16.u32 %0, t;\n\t}"
      : "=h"(v) : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ uint32_t ld_scale_u16(const uint8_t *p, uint64_t policy) {
  uint16_t v;
  asm("ld.global.nc.L1::no_allocate.L2::cache_hint.L2::128B.u16 %0, [%1], %2;"
      : "=h"(v) : "l"(p), "l"(policy));
  return v;
}
// 16-byte global->shared copy with a cache policy; zero-fills when !valid.
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void *src, bool valid,
                                                uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(valid ? 16 : 0), "l"(policy)
               : "memory");
}

// ---------------------------------------------------------------- tensor cores
// D[tmem] (+)= A[smem] * B[smem]^T of e4m3 codes (K = 32 a step), one elected
// thread.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t"
               "setp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1),
// e4m3 A and B (bits 7-9, 10-12 = 0), MN-major A / B (bits 15 / 16), N/8 at
// bits 17-22, M/16 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor without swizzle (layout type 0): 8 x 16-byte core
// matrices, `lbo` / `sbo` bytes apart.
__device__ __forceinline__ uint64_t desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46);
}

} // namespace bia
