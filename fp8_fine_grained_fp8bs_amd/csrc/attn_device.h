// attn_device.h -- number conversions and constants of the attention kernels (gfx950).
#pragma once

#include "attn_sched.h"

namespace fp8bs {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kNoKeys = -1e30f;       // reference of a row that has seen no key yet
constexpr float kHeadroom = 15.0f;      // log2 of the largest p' before the reference moves
constexpr float kMostWeight = 0x1p15f;  // the same, as a sum of weights
constexpr float kTop = 8.0f;            // log2 of the largest p' after a move
constexpr float kMinVScale = 0x1p-100f;
// Keys of a block with a smaller value scale than this (a block of zeros has none) go
// into the denominator as p / 2^m, by an exponential of their own: by way of p' / v they
// would be lost where p' falls below FP32's least (beside scales of 2^34 and more), and
// leave its range at 2^115 a key.  The reference then also keeps p / 2^m below 2^97, so
// that the sums of 2^30 keys stay in range.
constexpr float kTinyV = 0x1p-32f, kTinyLog = -32.0f;
constexpr float kDenHeadroom = 97.0f, kDenTop = 96.0f;   // log2, as kHeadroom and kTop
constexpr float kMostDen = 0x1p102f;    // the headroom, as a sum of 32 keys
constexpr float kMinKScale = 0x1p-120f; // of a key block's factor, so that it keeps a masked score's -infinity

// Eight codes (two dwords) to eight BF16 / FP16 values, exact.
__device__ __forceinline__ bf16x8 bf16_of_codes(uint32_t a, uint32_t b) {
  const u32x4 w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true))};
  return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ f16x8 f16_of_codes(uint32_t a, uint32_t b) {
  const u32x4 w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true))};
  return __builtin_bit_cast(f16x8, w);
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), f16x2));
}

// A 4x4 byte transpose: r[i] holds byte i of a, b, c, d.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t r[4]) {
  const uint32_t x = __builtin_amdgcn_perm(b, a, 0x05010400u), y = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t z = __builtin_amdgcn_perm(d, c, 0x05010400u), w = __builtin_amdgcn_perm(d, c, 0x07030602u);
  r[0] = __builtin_amdgcn_perm(z, x, 0x05040100u);
  r[1] = __builtin_amdgcn_perm(z, x, 0x07060302u);
  r[2] = __builtin_amdgcn_perm(w, y, 0x05040100u);
  r[3] = __builtin_amdgcn_perm(w, y, 0x07060302u);
}

}  // namespace fp8bs
