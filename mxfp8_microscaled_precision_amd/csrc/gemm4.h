// Shared by the kernels for products with 4-bit MX weights (internal).
#pragma once
#include "gemm_common.h"

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
