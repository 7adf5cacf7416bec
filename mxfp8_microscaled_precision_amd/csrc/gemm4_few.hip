// Products of few rows with 4-bit MX weights for gfx950 (a decoding step's
// tokens): C = A * B^T as in gemm4.hip, which has the lane layouts.
#include "gemm4.h"

namespace mx {

// ---------------------------------------------------------------------------
// Few rows: the weight streams from memory straight into MFMA operands.
// ---------------------------------------------------------------------------
// A workgroup of 8 waves computes 16 MF rows x 16 NF columns; its waves take
// the 256-element chunks of K in turn and their sums are added in LDS in the
// order of the waves.  A lane's share of a chunk of a 4-bit row is 32
// consecutive bytes, blocks 2 g and 2 g + 1: MFMA j takes block 2 g + j as
// hardware block g, and a row's four lanes read one whole line.
constexpr int SK_WAVES = 8;
constexpr int SK_THREADS = 64 * SK_WAVES;

// One lane's operands of a chunk for one fragment of 16 rows.
template <int F>
struct SkFrag {
  v4i lo[2], hi[2];  // hi: 8-bit operands only
  uint32_t sc;       // scale bytes of MFMA 0 and 1

  // p, s: the lane's row; c: chunk; full: the whole chunk lies in K
  __device__ __forceinline__ void load(const uint8_t* __restrict__ p, const uint8_t* __restrict__ s,
                                       int64_t c, int64_t K, int g, bool full) {
    const int64_t nkb = K >> 5;
    if (full) {
      sc = *(const u16_at1*)(s + 8 * c + 2 * g);
    } else {
      sc = 0x7F7Fu;
      for (int j = 0; j < 2; j++)
        if (8 * c + 2 * g + j < nkb)
          sc = (sc & ~(0xFFu << (8 * j))) | ((uint32_t)s[8 * c + 2 * g + j] << (8 * j));
    }
#pragma unroll
    for (int j = 0; j < 2; j++) {
      if (F == ELEM_E2M1) {
        const int b = 2 * g + j;
        lo[j] = full || 8 * c + b < nkb ? *(const v4i*)(p + 128 * c + 16 * b) : (v4i){0, 0, 0, 0};
      } else {
        const int b = 2 * (g >> 1) + j;
        const uint8_t* at = p + 256 * c + 32 * b + 16 * (g & 1);
        lo[j] = full || 8 * c + b < nkb ? *(const v4i*)at : (v4i){0, 0, 0, 0};
        hi[j] = full || 8 * c + b + 4 < nkb ? *(const v4i*)(at + 128) : (v4i){0, 0, 0, 0};
      }
    }
  }
  __device__ __forceinline__ v8i operand(int j) const {
    if (F == ELEM_E2M1) return (v8i){lo[j].x, lo[j].y, lo[j].z, lo[j].w, 0, 0, 0, 0};
    return (v8i){lo[j].x, lo[j].y, lo[j].z, lo[j].w, hi[j].x, hi[j].y, hi[j].z, hi[j].w};
  }
};

template <int FA, int MF, int NF>
struct SkChunk {
  SkFrag<FA> a[MF];
  SkFrag<ELEM_E2M1> b[NF];
};

// Rows m0 .. m_end - 1 (at most 16 MF of them) x columns n0 .. of C.
template <int FA, int MF, int NF>
__device__ __forceinline__ void skinny_tile(const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                                            const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                                            uint16_t* __restrict__ c, int64_t m0, int64_t m_end,
                                            int64_t n0, int64_t N, int64_t K, v4f* red) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i = lane & 15;
  const int64_t pitch_a = FA == ELEM_E2M1 ? K >> 1 : K, pitch_b = K >> 1, nkb = K >> 5;
  const uint8_t *pa[MF], *psa[MF], *pb[NF], *psb[NF];
  // rows past the end repeat the last one; their results are not stored
#pragma unroll
  for (int f = 0; f < MF; f++) {
    int64_t m = m0 + 16 * f + i;
    m = m < m_end ? m : m_end - 1;
    pa[f] = a + m * pitch_a;
    psa[f] = sa + m * nkb;
  }
#pragma unroll
  for (int f = 0; f < NF; f++) {
    int64_t n = n0 + 16 * f + i;
    n = n < N ? n : N - 1;
    pb[f] = b + n * pitch_b;
    psb[f] = sb + n * nkb;
  }
  v4f acc[NF][MF];
#pragma unroll
  for (int x = 0; x < NF; x++)
#pragma unroll
    for (int y = 0; y < MF; y++) acc[x][y] = (v4f){0, 0, 0, 0};
  auto load = [&](SkChunk<FA, MF, NF>& t, int64_t ch, bool full) {
#pragma unroll
    for (int f = 0; f < NF; f++) t.b[f].load(pb[f], psb[f], ch, K, g, full);
#pragma unroll
    for (int f = 0; f < MF; f++) t.a[f].load(pa[f], psa[f], ch, K, g, full);
  };
  auto mma = [&](const SkChunk<FA, MF, NF>& t) {
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int x = 0; x < NF; x++)
#pragma unroll
        for (int y = 0; y < MF; y++) {
          if (j == 0)
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                t.b[x].operand(0), t.a[y].operand(0), acc[x][y], ELEM_E2M1, FA, 0, (int)t.b[x].sc, 0,
                (int)t.a[y].sc);
          else
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                t.b[x].operand(1), t.a[y].operand(1), acc[x][y], ELEM_E2M1, FA, 1, (int)t.b[x].sc, 1,
                (int)t.a[y].sc);
        }
  };
  const int64_t whole = K >> 8;  // whole chunks
  SkChunk<FA, MF, NF> t0, t1;
  int64_t ch = wave;
  if (ch < whole) load(t0, ch, true);
  for (; ch < whole; ch += 2 * SK_WAVES) {
    const bool two = ch + SK_WAVES < whole;
    if (two) load(t1, ch + SK_WAVES, true);
    mma(t0);
    if (!two) break;
    if (ch + 2 * SK_WAVES < whole) load(t0, ch + 2 * SK_WAVES, true);
    mma(t1);
  }
  if ((K & 255) != 0 && wave == (int)(whole % SK_WAVES)) {
    load(t0, whole, false);
    mma(t0);
  }
  // lane l, element e of a fragment: column 4 (l / 16) + e, row l % 16
#pragma unroll
  for (int x = 0; x < NF; x++)
#pragma unroll
    for (int y = 0; y < MF; y++) red[((wave * NF + x) * MF + y) * 64 + lane] = acc[x][y];
  __syncthreads();
  for (int t = threadIdx.x; t < NF * MF * 64; t += SK_THREADS) {
    v4f v = red[t];
#pragma unroll
    for (int w = 1; w < SK_WAVES; w++) v += red[w * NF * MF * 64 + t];
    const int l = t & 63, f = t >> 6;
    const int64_t m = m0 + 16 * (f % MF) + (l & 15);
    const int64_t n = n0 + 16 * (f / MF) + 4 * (l >> 4);
    if (m >= m_end) continue;
    uint16_t* dst = c + m * N + n;
    const uint32_t w[2] = {cvt_pk_bf16(v.x, v.y), cvt_pk_bf16(v.z, v.w)};
    if ((N & 3) == 0 && n < N) {
      *(u32x2*)dst = (u32x2){w[0], w[1]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (n + e < N) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
  __syncthreads();  // `red` may be written again
}

template <int FA, int MF, int NF>
__global__ void __launch_bounds__(SK_THREADS)
gemm4_skinny_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                    const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                    uint16_t* __restrict__ c, int64_t M, int64_t N, int64_t K) {
  __shared__ v4f red[SK_WAVES * NF * MF * 64];
  for (int64_t m0 = (int64_t)blockIdx.y * 16 * MF; m0 < M; m0 += (int64_t)gridDim.y * 16 * MF)
    skinny_tile<FA, MF, NF>(a, sa, b, sb, c, m0, m0 + 16 * MF < M ? m0 + 16 * MF : M,
                            (int64_t)blockIdx.x * 16 * NF, N, K, red);
}

template <int FA, int MF, int NF>
__global__ void __launch_bounds__(SK_THREADS)
grouped4_skinny_kernel(const int64_t* __restrict__ offsets, int64_t T,
                       const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                       const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                       uint16_t* __restrict__ c, int64_t N, int64_t K) {
  __shared__ v4f red[SK_WAVES * NF * MF * 64];
  const int64_t g = blockIdx.y;
  // clamped, so that bad offsets read and write rows of [0, T) only
  int64_t lo = offsets[g], hi = offsets[g + 1];
  lo = lo < 0 ? 0 : (lo > T ? T : lo);
  hi = hi < lo ? lo : (hi > T ? T : hi);
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * MF)
    skinny_tile<FA, MF, NF>(a, sa, b + g * N * (K >> 1), sb + g * N * (K >> 5), c, m0,
                            m0 + 16 * MF < hi ? m0 + 16 * MF : hi, (int64_t)blockIdx.x * 16 * NF, N, K,
                            red);
}

template <int FA>
static void launch_few(int64_t M, int64_t N, int64_t K, const uint8_t* a, const uint8_t* sa,
                       const uint8_t* b, const uint8_t* sb, uint16_t* c, hipStream_t stream) {
  const unsigned gx = (unsigned)((N + 31) / 32);
#define MX_FEW(MF_)                                                                               \
  hipLaunchKernelGGL((gemm4_skinny_kernel<FA, MF_, 2>), dim3(gx, (unsigned)((M + 16 * MF_ - 1) / (16 * MF_))), \
                     dim3(SK_THREADS), 0, stream, a, sa, b, sb, c, M, N, K)
  if (M <= 16) MX_FEW(1);
  else if (M <= 32) MX_FEW(2);
  else MX_FEW(4);
#undef MX_FEW
}

hipError_t launch_gemm4_few(int a_elem, int64_t M, int64_t N, int64_t K, const void* a,
                            const void* sa, const void* b, const void* sb, void* c,
                            hipStream_t stream) {
  const uint8_t *A = (const uint8_t*)a, *SA = (const uint8_t*)sa, *B = (const uint8_t*)b,
                *SB = (const uint8_t*)sb;
  uint16_t* C = (uint16_t*)c;
  if (a_elem == ELEM_E4M3) launch_few<ELEM_E4M3>(M, N, K, A, SA, B, SB, C, stream);
  else if (a_elem == ELEM_E5M2) launch_few<ELEM_E5M2>(M, N, K, A, SA, B, SB, C, stream);
  else if (a_elem == ELEM_E2M1) launch_few<ELEM_E2M1>(M, N, K, A, SA, B, SB, C, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_grouped_gemm4_few(int a_elem, int64_t G, const int64_t* offsets, int64_t T,
                                    int64_t N, int64_t K, const void* a, const void* sa,
                                    const void* b, const void* sb, void* c, hipStream_t stream) {
  const dim3 grid((unsigned)((N + 31) / 32), (unsigned)G);
#define MX_GFEW(FA_, MF_)                                                                         \
  hipLaunchKernelGGL((grouped4_skinny_kernel<FA_, MF_, 2>), grid, dim3(SK_THREADS), 0, stream, offsets, \
                     T, (const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb, \
                     (uint16_t*)c, N, K)
#define MX_GFEW_M(FA_)               \
  do {                               \
    if (T <= 16 * G) MX_GFEW(FA_, 1); \
    else MX_GFEW(FA_, 4);            \
  } while (0)
  if (a_elem == ELEM_E4M3) MX_GFEW_M(ELEM_E4M3);
  else if (a_elem == ELEM_E5M2) MX_GFEW_M(ELEM_E5M2);
  else if (a_elem == ELEM_E2M1) MX_GFEW_M(ELEM_E2M1);
  else return hipErrorInvalidValue;
#undef MX_GFEW_M
#undef MX_GFEW
  return hipGetLastError();
}

}  // namespace mx
