// kv4.cuh -- the paged cache of keys and values in 4 bits: its layout, and the
// arithmetic of its codes.
//
// A cache is uint8 [pages][HK][page bytes]; a page of P tokens (P = 16, 32, 64 or
// 128) holds of one key/value head, one after the other,
//   key codes     P x D/2    E2M1, value 2i of a row in the low half of byte i
//   key scales    P x D/16   E4M3, one for 16 values
//   value codes   P x D/2
//   value scales  P x D/16
// so that a page of a head is one run of 9 D P / 8 bytes, which a bulk copy takes
// whole, and a token's codes are whole rows that a write or a move can take alone.
//
// A value is code * scale * g (g the call's k_scale or v_scale).  E2M1 has two
// significant bits and E4M3 four, so code * scale has six and is exact in FP16 and
// BF16 alike: |code * scale| <= 2688 and, where not zero, >= 2^-10.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace fp8bq {
namespace {

constexpr float kE2m1Max = 6.0f;
constexpr float kE4m3Least = 0x1p-9f;  // the smallest scale that is not zero
constexpr uint32_t kE4m3Nan = 0x7Fu;

// 8 codes -> 4 x 2 FP16 values, code 2i in the low half of o[i]
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// two E4M3 bytes (low 16 bits) -> FP16 pair, the low byte in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// one half of an FP16 pair in both halves
__device__ __forceinline__ uint32_t both_low(uint32_t v) { return __byte_perm(v, v, 0x1010); }
__device__ __forceinline__ uint32_t both_high(uint32_t v) { return __byte_perm(v, v, 0x3232); }

}  // namespace

// byte offsets of a page's parts
struct Kv4Page {
  int code_bytes, scale_bytes;  // of one token's keys (or values)
  int k_scales, v_codes, v_scales, bytes;
};
__host__ __device__ inline Kv4Page kv4_page(int page, int D) {
  Kv4Page p;
  p.code_bytes = D / 2, p.scale_bytes = D / 16;
  p.k_scales = page * p.code_bytes;
  p.v_codes = p.k_scales + page * p.scale_bytes;
  p.v_scales = p.v_codes + page * p.code_bytes;
  p.bytes = p.v_scales + page * p.scale_bytes;
  return p;
}

}  // namespace fp8bq
