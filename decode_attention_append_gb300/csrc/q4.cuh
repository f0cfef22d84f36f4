// The 4-bit KV cache: number formats and page layout, shared by the kernels
// that write it (append), read it back (dequant) and attend over it.
//
// A cache value is  e2m1 * e4m3 * 2^e:  a 4-bit float (sign, two exponent bits,
// one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), the scale of its block of 16
// dims of one token and head, and the head's exponent (kv_exp; 0 without one).
// e2m1 has 2 significant bits and e4m3 has 4, so e2m1 * e4m3 is exact in fp16
// (at most 6 * 448 = 2688, at least 2^-10) and in bf16; nothing is rounded when
// a value is read.
//
// One (page, head) holds a K slice and a V slice of kSlice(d) = 9 d bytes side
// by side:
//   16 token rows of d/2 bytes (dim 2i low nibble, dim 2i + 1 high nibble), then
//   d scale bytes: K [16 tokens][d/16 blocks], V [d/16 blocks][16 tokens]
//   (each the order in which its product reads them).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace daa {

constexpr int kQ4Block = 16;  // dims of one scale
constexpr int kQ4Page = 16;   // tokens of a page
constexpr int kQ4MaxExp = 32;  // |kv_exp| is cut to this, so powers of two stay normal

__host__ __device__ constexpr int q4_slice_bytes(int d) { return 9 * d; }

// Loads of what the kernel ahead may have written.  These kernels are launched
// programmatically and start before that one has ended, so its results are no
// constants of theirs: not ld.global.nc (__ldg), and volatile, to stay behind the wait.
__device__ __forceinline__ int32_t ld_word(const void* p) {
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_byte(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Eight e2m1 codes (one 32-bit word, lowest nibble first) -> four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two e4m3 bytes -> an fp16 pair (low byte in the low half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// An fp16 pair -> e4m3 bytes, nearest, ties to even, cut at 448 (low half in the low byte).
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

// 1 / x, off by 2^-23 (relative) at most.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight fp16 values -> e2m1 codes, nearest, ties to even, cut at 6 (first lowest).
__device__ __forceinline__ uint32_t f16x8_to_e2m1x8(const uint32_t (&h)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}

// Two floats -> fp16 pair, nearest (lo in the low half); infinities stay.
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A head's exponent, cut to [-kQ4MaxExp, kQ4MaxExp], and two to its power.
__device__ __forceinline__ int q4_exp(int e) { return min(max(e, -kQ4MaxExp), kQ4MaxExp); }
__device__ __forceinline__ float q4_pow2(int e) { return __int_as_float((q4_exp(e) + 127) << 23); }

}  // namespace daa
