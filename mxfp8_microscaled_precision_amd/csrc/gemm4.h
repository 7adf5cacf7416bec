// Shared by the kernels for products with 4-bit MX weights (internal).
#pragma once
#include "gemm_common.h"

namespace mx {

typedef float v4f __attribute__((ext_vector_type(4)));
// global memory takes these at any address
typedef uint16_t u16_at1 __attribute__((aligned(1)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

// The kernels for few rows (gemm4_few.hip).
hipError_t launch_gemm4_few(int a_elem, int64_t M, int64_t N, int64_t K, const void* a,
                            const void* sa, const void* b, const void* sb, void* c,
                            hipStream_t stream);
hipError_t launch_grouped_gemm4_few(int a_elem, int64_t G, const int64_t* offsets, int64_t T,
                                    int64_t N, int64_t K, const void* a, const void* sa,
                                    const void* b, const void* sb, void* c, hipStream_t stream);

}  // namespace mx
