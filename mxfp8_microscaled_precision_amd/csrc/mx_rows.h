// Vector access to rows of any length: four logits or eight BF16 elements at
// once wherever they lie (global memory takes vector accesses at any address
// of the element's alignment), and the last few of a row one by one.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

typedef float f32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One and four elements as FP32.
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf_lo(*p); }
__device__ __forceinline__ void load4(const float* p, float v[4]) {
  const f32x4_at4 a = *(const f32x4_at4*)p;
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float v[4]) {
  const u32x2_at2 a = *(const u32x2_at2*)p;
  v[0] = bf_lo(a.x), v[1] = bf_hi(a.x), v[2] = bf_lo(a.y), v[3] = bf_hi(a.y);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)cvt_pk_bf16(v, v); }
__device__ __forceinline__ void store4(float* p, const float v[4]) {
  *(f32x4_at4*)p = (f32x4_at4){v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float v[4]) {
  *(u32x2_at2*)p = (u32x2_at2){cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
}

// BF16 elements c .. c + 7 of a row of H, as packed pairs.  WHOLE: all eight
// are in the row; otherwise at least one is, and the rest read as 0.
template <bool WHOLE>
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t* row, int64_t c, int64_t H) {
  if (WHOLE) return __builtin_nontemporal_load((const u32x4_at2*)(row + c));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (c + i < H) w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return (u32x4){w[0], w[1], w[2], w[3]};
}
// STREAM: past the caches.
template <bool WHOLE, bool STREAM>
__device__ __forceinline__ void store_bf16x8(uint16_t* row, int64_t c, int64_t H, u32x4 v) {
  if (WHOLE) {
    if (STREAM) __builtin_nontemporal_store(v, (u32x4_at2*)(row + c));
    else *(u32x4_at2*)(row + c) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (c + i < H) row[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ void unpack8(u32x4 v, float f[8]) {
  f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}
__device__ __forceinline__ u32x4 pack8(const float f[8]) {
  return (u32x4){cvt_pk_bf16(f[0], f[1]), cvt_pk_bf16(f[2], f[3]), cvt_pk_bf16(f[4], f[5]),
                 cvt_pk_bf16(f[6], f[7])};
}

}  // namespace mx
