// Device helpers of the column quantisers: where the grouped layout's blocks
// come from, and a column block's maximum and scale.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
  return __builtin_bit_cast(uint32_t, r);
}

// Grouped column mode: the wave's 32 output rows r0 .. r0+31 (a block of
// the padded token axis) -> first source row and number of real rows.  The
// group is the last g with P_g <= r0, found by counting (one ballot per 64
// groups, all offsets loaded at once, lane l of word k holding offsets[64k+l]);
// offsets are clamped into [0, T], so
// bad offsets give wrong blocks but only rows inside [0, T) are read.
constexpr int GCOL_MAX_GROUPS = 512;

// A wave-uniform lane's copy of a 64-bit register.
__device__ __forceinline__ int64_t readlane64(int64_t v, int l) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), l);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ void gcol_block(const int64_t* __restrict__ offsets, int64_t G,
                                           int64_t T, int64_t r0, int lane, int64_t& src,
                                           int& nreal) {
  int64_t o[GCOL_MAX_GROUPS / 64];
#pragma unroll
  for (int k = 0; k < GCOL_MAX_GROUPS / 64; k++) {
    const int64_t gg = 64 * k + lane;
    o[k] = gg <= G ? offsets[gg] : T;
  }
  int cnt = 0;
#pragma unroll
  for (int k = 0; k < GCOL_MAX_GROUPS / 64; k++) {
    const int64_t gg = 64 * k + lane;
    const int64_t oc = o[k] < 0 ? 0 : (o[k] > T ? T : o[k]);
    cnt += __popcll(__ballot(gg < G && 128 * (oc / 128 + gg) <= r0));
  }
  src = 0;
  nreal = 0;
  if (cnt == 0) return;
  const int64_t g = cnt - 1;
  // offsets[g] and offsets[g + 1] from the lanes that loaded them (g is
  // uniform); only offsets[512] lies past the loaded words
  int64_t lo = 0, hi = 0;
#pragma unroll
  for (int k = 0; k < GCOL_MAX_GROUPS / 64; k++) {
    if ((g >> 6) == k) lo = readlane64(o[k], (int)(g & 63));
    if (((g + 1) >> 6) == k) hi = readlane64(o[k], (int)((g + 1) & 63));
  }
  if (g + 1 == GCOL_MAX_GROUPS) hi = offsets[g + 1];
  lo = lo < 0 ? 0 : (lo > T ? T : lo);
  hi = hi < lo ? lo : (hi > T ? T : hi);
  const int64_t first = 128 * (lo / 128 + g);
  if (r0 < first) return;                       // only with decreasing offsets
  const int64_t j = (r0 - first) >> 5;          // block of the group's range
  const int64_t left = (hi - lo) - 32 * j;
  src = lo + 32 * j;
  nreal = left <= 0 ? 0 : (left >= 32 ? 32 : (int)left);
}

// Column maxima of a wave whose lane l = 8 g + h holds rows of the same columns
// as lanes h, h + 8, ..., h + 56, two columns' magnitudes to a word: each step
// halves the words a lane is left with, so that a word is reduced in one place.
// 8 words: lane g ends with the maximum of word g; 4: of word g / 2.
__device__ __forceinline__ uint32_t max_swap32(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return pk_max(r[0], r[1]);  // lanes below 32: a of both halves, above: b
}
__device__ __forceinline__ uint32_t max_swap16(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  return pk_max(r[0], r[1]);  // even rows of 16 lanes: a of both rows, odd ones: b
}
__device__ __forceinline__ uint32_t ror8(uint32_t v) {  // lane ^ 8 of the row of 16
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t column_max8(const uint32_t w[8], int lane) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; i++) x[i] = max_swap32(w[i], w[i + 4]);
  const uint32_t y0 = max_swap16(x[0], x[2]), y1 = max_swap16(x[1], x[3]);
  const bool odd = (lane & 8) != 0;
  return pk_max(odd ? y1 : y0, ror8(odd ? y0 : y1));
}
__device__ __forceinline__ uint32_t column_max4(const uint32_t w[4]) {
  const uint32_t y = max_swap16(max_swap32(w[0], w[2]), max_swap32(w[1], w[3]));
  return pk_max(y, ror8(y));
}

// Two columns' scales from their maxima (BF16 magnitudes in the halves of a
// word), each as the BF16 bits of 2^(byte - 127): byte << 7, or 0x0040 for byte
// 0.  The mantissa's carry is the rceil rule: E - off + [m > top] is the
// exponent of amax + 127 - top less off.  A non-finite block gives 0x7F80.
template <int EL>
__device__ __forceinline__ uint32_t pair_scale(uint32_t amax) {
  constexpr unsigned short top = EL == ELEM_E2M1 ? 64 : 96;
  constexpr unsigned short off = EL == ELEM_E5M2 ? 15 : EL == ELEM_E2M1 ? 2 : 8;  // 127 less
  const u16x2 a = __builtin_bit_cast(u16x2, amax);
  const u16x2 one = (u16x2){1, 1};
  u16x2 b = __builtin_elementwise_sub_sat((u16x2)((a + (unsigned short)(127 - top)) >> 7), (u16x2){off, off});
  b = __builtin_elementwise_max((u16x2)(b << 7), (u16x2){0x40, 0x40});
  // 1 where the magnitude is Inf or NaN
  const u16x2 bad = __builtin_elementwise_min(__builtin_elementwise_sub_sat(a, (u16x2){0x7F7F, 0x7F7F}), one);
  b = __builtin_elementwise_max(b, (u16x2)(bad * (unsigned short)0x7F80));
  return __builtin_bit_cast(uint32_t, b);
}

}  // namespace mx
