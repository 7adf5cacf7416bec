// Shared by the kernels for products with 4-bit MX weights (internal).
#pragma once
#include "gemm_common.h"
#include "mx_rows.h"

namespace mx {

typedef float v4f __attribute__((ext_vector_type(4)));

// dma16 and dma4 with a scalar offset added.  Whether the buffer's range check
// counts it makes no difference here: it moves along a row that lies in the
// buffer, and an offset past the buffer stays past it.
__device__ __forceinline__ void dma16_at(const lds_u8* lds, uint32_t voffset, u32x4 rsrc, uint32_t soffset) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  soffset = __builtin_amdgcn_readfirstlane(soffset);
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(m0), "v"(voffset), "s"(rsrc), "s"(soffset)
               : "memory");
}
__device__ __forceinline__ void dma4_at(const lds_u8* lds, uint32_t voffset, u32x4 rsrc, uint32_t soffset) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  soffset = __builtin_amdgcn_readfirstlane(soffset);
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(m0), "v"(voffset), "s"(rsrc), "s"(soffset)
               : "memory");
}

// A wave's result, FN x FM accumulators of 32x32 that begin at row m0 and column
// n0, in BF16 for any N: lanes l and l + 32 trade groups so that a lane holds
// eight consecutive columns (gemm_common.h).
template <int FN, int FM>
__device__ __forceinline__ void store_bf16(const v16f (&acc)[FN][FM], uint16_t* __restrict__ c, int64_t N,
                                           int64_t m0, int64_t m_end, int64_t n0, int lane) {
  const int g = lane >> 5, i = lane & 31;
  // opaque, or a caller's loop over tiles has the addresses hoisted over its K
  // loop; and one accumulator at a time, or all are copied first
  asm volatile("" : "+v"(m0), "+v"(n0));
#pragma unroll
  for (int fn = 0; fn < FN; fn++)
#pragma unroll
    for (int fm = 0; fm < FM; fm++) {
      __builtin_amdgcn_sched_barrier(0);
      const v16f& v = acc[fn][fm];
      uint32_t p[4][2];
#pragma unroll
      for (int r4 = 0; r4 < 4; r4++) {
        p[r4][0] = cvt_pk_bf16(v[4 * r4 + 0], v[4 * r4 + 1]);
        p[r4][1] = cvt_pk_bf16(v[4 * r4 + 2], v[4 * r4 + 3]);
      }
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int d = 0; d < 2; d++) {
          const auto s = __builtin_amdgcn_permlane32_swap(p[2 * h][d], p[2 * h + 1][d], false, false);
          p[2 * h][d] = s[0];
          p[2 * h + 1][d] = s[1];
        }
      const int64_t m = m0 + 32 * fm + i;
      if (m >= m_end) continue;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int64_t n = n0 + 32 * fn + 16 * h + 8 * g;
        const uint32_t w[4] = {p[2 * h][0], p[2 * h][1], p[2 * h + 1][0], p[2 * h + 1][1]};
        uint16_t* dst = c + m * N + n;
        if (n + 8 <= N) {
          *(u32x4_at2*)dst = (u32x4_at2){w[0], w[1], w[2], w[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (n + e < N) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
}

// The kernels with small tiles and many stages (gemm4_deep.hip); ws:
// gemm4_deep_workspace bytes, written and read by the call.
size_t gemm4_deep_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm4_deep(int a_elem, int64_t M, int64_t N, int64_t K, const void* a,
                             const void* sa, const void* b, const void* sb, void* c, void* ws,
                             hipStream_t stream);
hipError_t launch_grouped_gemm4_deep(int a_elem, int64_t G, const int64_t* offsets, int64_t T,
                                     int64_t N, int64_t K, const void* a, const void* sa,
                                     const void* b, const void* sb, void* c, hipStream_t stream);

}  // namespace mx
