// E4M3 codes of bf16 values under a scale s, amax / 448 up to its rounding to fp32: what the fp8 quantizers, by row and by
// block of 128, share.
#pragma once

#include "qpl_device.h"

namespace qpl {

__device__ __forceinline__ uint32_t vec_absmax(const u32x4& v, uint32_t m) {
  return absmax_acc(absmax_acc(absmax_acc(absmax_acc(m, v.x), v.y), v.z), v.w);
}

// Codes of a bf16 pair in a row whose scale is 0 (every element is +-0): the sign only.
__device__ __forceinline__ uint32_t fp8_pair_zero(uint32_t p) { return ((p >> 8) & 0x80u) | ((p >> 16) & 0x8000u); }

// Row quantizer state: the scale s and r = RN(1/s) for the division.
struct RowDiv {
  float s, r;
  bool zero, tiny;
};

__device__ __forceinline__ RowDiv scale_div(float s) {
  RowDiv d;
  d.s = s;
  d.zero = !(d.s > 0.0f);
  d.tiny = !div_rn_ok(d.s);
  d.r = 1.0f / d.s;
  return d;
}

// By row: the correctly rounded quotient.
__device__ __forceinline__ RowDiv row_div(float amax) { return scale_div(amax / 448.0f); }

// By block: the product with fp32(1 / 448), 0.375 * 2^-23 of itself above it before its rounding.  torch divides a
// tensor on the GPU by a number like that, so codes made here are those that a program in torch makes there: a value
// of bf16 over s often lies on the border between two codes, and one step of s decides for either.
__device__ __forceinline__ RowDiv block_div(float amax) { return scale_div(amax * (1.0f / 448.0f)); }

// |x| <= amax, so |x / s| stays at 448 up to rounding: no overflow, and no clamp
// needed before the converter.
__device__ __forceinline__ float qdiv(float x, const RowDiv& d) {
  return d.tiny ? x / d.s : div_rn_finite(x, d.s, d.r);
}

// E4M3 codes of two bf16 pairs: pair a in bits 15:0, pair b in bits 31:16 (the
// converter's word select fills the halves; no clamp, see qdiv).
__device__ __forceinline__ uint32_t fp8_word(uint32_t a, uint32_t b, const RowDiv& d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(qdiv(bf16_lo(a), d), qdiv(bf16_hi(a), d), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(qdiv(bf16_lo(b), d), qdiv(bf16_hi(b), d), lo, true);
}

__device__ __forceinline__ u32x2 fp8_vec(u32x4 v, const RowDiv& d) {
  u32x2 o;
  if (d.zero) {
    o.x = fp8_pair_zero(v.x) | (fp8_pair_zero(v.y) << 16);
    o.y = fp8_pair_zero(v.z) | (fp8_pair_zero(v.w) << 16);
    return o;
  }
  o.x = fp8_word(v.x, v.y, d);
  o.y = fp8_word(v.z, v.w, d);
  return o;
}

}  // namespace qpl
