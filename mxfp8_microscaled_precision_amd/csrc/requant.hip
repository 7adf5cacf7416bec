// Column blocks of an 8-bit MX tensor that is held in row blocks, for gfx950: a
// forward product's operand, kept as the 8-bit checkpoint, becomes the operand
// of the weight gradient (dual-axis quantisation: torchtitan-npu MXFP8/HiF8
// tutorial, step-2 environment table, MXFP8_DUAL_AXIS_FORWARD; per expert group:
// MindSpeed RFC section 2.2).  Payload times scale, rounded to BF16 (exact but
// at the ends of BF16's range), is quantised again in blocks of 32 down the
// columns and written transposed; with groups the blocks restart at every
// group offset, in quant.hip's grouped layout.
//
// Bound by HBM and, next to it, by the vector unit: a byte in and a byte out an
// element leave little time for each, so the column maxima are reduced by
// halving (column_max8: 16 instructions for 16 columns instead of a butterfly
// of all), each scale is formed in one lane, and the lanes that need it read
// it back from LDS as a BF16 factor.  Measured at 131072 x 4096: 238 us dense
// and 247 in 64 groups (4.7 and 4.5 TB/s; 361 with a butterfly for every column
// and the scales formed by all lanes).  What is left of the gap to a copy's rate
// is the vector unit, busy 46% of the time, and the latency between the load,
// the exchange and the store of a tile.  Tiles dealt to the XCDs in contiguous
// parts: 238 us in groups, but 292 dense.
#include "mx_columns.h"
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int RQ_THREADS = 256;
constexpr int RQ_TILE = 128;

typedef __attribute__((address_space(3))) uint8_t lds8;
typedef __attribute__((address_space(3))) uint32_t lds32;
typedef __attribute__((address_space(3))) u32x4 lds128;

// A workgroup of four waves covers 128 rows x 128 columns; wave w takes rows 32
// w .. 32 w + 31, lane l = 8 g + h of it rows 4 g .. 4 g + 3 of columns 16 h ..
// 16 h + 15 as four 16-byte chunks: a load reads whole lines of eight rows.  A
// column block is the lanes h, h + 8, ..., h + 56.  The payload leaves through
// LDS in whole lines, 16-byte chunk k of column c at k ^ (c / 16 & 7).
template <int SRC, int EL, bool GROUPED>
__global__ void __launch_bounds__(RQ_THREADS)
requant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t R, int64_t C,
               uint8_t* __restrict__ qt, uint8_t* __restrict__ st, int64_t G,
               const int64_t* __restrict__ offsets, int64_t T) {
  __shared__ __attribute__((aligned(16))) uint8_t lqt_[RQ_TILE * 128];  // payload, a column to a row
  __shared__ __attribute__((aligned(16))) uint8_t lsf_[4 * RQ_TILE * 2];  // scales as BF16: [wave][column]
  lds8 *lqt = (lds8*)lqt_, *lsf = (lds8*)lsf_;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 3, h = lane & 7;
  // column tiles fastest: the row tiles that share a line of the scales run
  // close together
  const int64_t lin = (int64_t)blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  const int64_t tr = lin / gridDim.y, tc = lin - tr * gridDim.y;
  const int64_t R0 = tr * RQ_TILE, C0 = tc * RQ_TILE;
  const int64_t r0 = R0 + 32 * wave, c = C0 + 16 * h;
  int64_t src = r0;
  int nreal = 32;  // rows 0 .. nreal - 1 of the block are tokens
  if (GROUPED) {
    src = 0;
    nreal = 0;
    if (r0 < R) gcol_block(offsets, G, T, r0, lane, src, nreal);
  } else if (r0 >= R) {
    nreal = 0;  // R is a multiple of 32: a wave's rows are wholly in or out
  }
  u32x4 w[4];
  uint32_t sb[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    w[i] = (u32x4){0, 0, 0, 0};
    sb[i] = 0;
    if (c < C && 4 * g + i < nreal) {
      const int64_t at = (src + 4 * g + i) * C + c;
      w[i] = __builtin_nontemporal_load((const u32x4*)(q + at));
      sb[i] = s[at >> 5];
    }
  }
  uint32_t v[4][8];  // row i, columns 2 k and 2 k + 1
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint4 lo = decode8_t<SRC>(make_uint2(w[i].x, w[i].y), sb[i]);
    const uint4 hi = decode8_t<SRC>(make_uint2(w[i].z, w[i].w), sb[i]);
    v[i][0] = lo.x, v[i][1] = lo.y, v[i][2] = lo.z, v[i][3] = lo.w;
    v[i][4] = hi.x, v[i][5] = hi.y, v[i][6] = hi.z, v[i][7] = hi.w;
  }
  uint32_t m[8];
#pragma unroll
  for (int k = 0; k < 8; k++)
    m[k] = pk_max(pk_max(v[0][k] & 0x7FFF7FFFu, v[1][k] & 0x7FFF7FFFu),
                  pk_max(v[2][k] & 0x7FFF7FFFu, v[3][k] & 0x7FFF7FFFu));
  // lane g forms the scales of columns 16 h + 2 g and + 1
  const uint32_t two = pair_scale<EL>(column_max8(m, lane));
  *(lds32*)(lsf + wave * 256 + 32 * h + 4 * g) = two;
  const bool bad = __any((two & 0xFFFFu) == 0x7F80u || (two >> 16) == 0x7F80u);
  // (a wave's own LDS operations complete in order)
  uint32_t f[8];
  {
    const u32x4 a = *(const lds128*)(lsf + wave * 256 + 32 * h);
    const u32x4 b = *(const lds128*)(lsf + wave * 256 + 32 * h + 16);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  // byte i of a column's dword is row 4 g + i; rows that hold no token stay 0
  const int left = nreal - 4 * g;
  const uint32_t real = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : 0xFFFFFFFFu >> (32 - 8 * left);
  const int chunk = 2 * wave + (g >> 2);
#pragma unroll
  for (int j = 0; j < 16; j++) {
    const int k = j >> 1;
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    const uint32_t p01 = __builtin_amdgcn_perm(v[1][k], v[0][k], sel);
    const uint32_t p23 = __builtin_amdgcn_perm(v[3][k], v[2][k], sel);
    const uint32_t fb = (j & 1) ? f[k] & 0xFFFF0000u : f[k] << 16;
    uint32_t out = cvt4_t<EL>(p01, p23, __uint_as_float(fb));
    if (bad && fb == 0x7F800000u) out = 0x7F7F7F7Fu;
    if (GROUPED) out &= real;
    *(lds32*)(lqt + (16 * h + j) * 128 + ((chunk ^ h) << 4) + 4 * (g & 3)) = out;
  }
  __syncthreads();

  const int t = threadIdx.x;
  const int64_t rows_here = (R - R0) < RQ_TILE ? (R - R0) : RQ_TILE;
  const int64_t cols_here = (C - C0) < RQ_TILE ? (C - C0) : RQ_TILE;
#pragma unroll
  for (int u = 0; u < 4; u++) {  // 8 lanes to a column's 128 bytes
    const int id = t + RQ_THREADS * u;
    const int col = id >> 3, k = id & 7;
    if (col < cols_here && 16 * k < rows_here)
      __builtin_nontemporal_store(*(const lds128*)(lqt + col * 128 + ((k ^ ((col >> 4) & 7)) << 4)),
                                  (u32x4*)(qt + (C0 + col) * R + R0 + 16 * k));
  }
  if (t < cols_here) {
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; b++)
      word |= (((uint32_t)lsf[b * 256 + 2 * t] >> 7) | ((uint32_t)lsf[b * 256 + 2 * t + 1] << 1)) << (8 * b);
    uint8_t* dst = st + (C0 + t) * (R >> 5) + (R0 >> 5);
    const int nb = (int)(rows_here >> 5);
    if (nb == 4 && ((uintptr_t)dst & 3) == 0) {
      *(uint32_t*)dst = word;
    } else {
      for (int b = 0; b < nb; b++) dst[b] = (uint8_t)(word >> (8 * b));
    }
  }
}

template <bool GROUPED>
static hipError_t launch_requant(int elem, int out_elem, const void* q, const void* s, int64_t R, int64_t C,
                                 void* qt, void* st, int64_t G, const int64_t* offsets, int64_t T,
                                 hipStream_t stream) {
  const dim3 grid((unsigned)((R + RQ_TILE - 1) / RQ_TILE), (unsigned)((C + RQ_TILE - 1) / RQ_TILE));
#define MX_REQUANT(SRC_, EL_)                                                                       \
  hipLaunchKernelGGL((requant_kernel<SRC_, EL_, GROUPED>), grid, dim3(RQ_THREADS), 0, stream,       \
                     (const uint8_t*)q, (const uint8_t*)s, R, C, (uint8_t*)qt, (uint8_t*)st, G, offsets, T)
  if (elem == ELEM_E4M3 && out_elem == ELEM_E4M3) MX_REQUANT(ELEM_E4M3, ELEM_E4M3);
  else if (elem == ELEM_E4M3 && out_elem == ELEM_E5M2) MX_REQUANT(ELEM_E4M3, ELEM_E5M2);
  else if (elem == ELEM_E5M2 && out_elem == ELEM_E4M3) MX_REQUANT(ELEM_E5M2, ELEM_E4M3);
  else if (elem == ELEM_E5M2 && out_elem == ELEM_E5M2) MX_REQUANT(ELEM_E5M2, ELEM_E5M2);
  else return hipErrorInvalidValue;
#undef MX_REQUANT
  return hipGetLastError();
}

hipError_t launch_requant_col(int elem, int out_elem, const void* q, const void* s, int64_t R,
                              int64_t C, void* qt, void* st, hipStream_t stream) {
  return launch_requant<false>(elem, out_elem, q, s, R, C, qt, st, 0, nullptr, 0, stream);
}

hipError_t launch_requant_grouped_col(int elem, int out_elem, const void* q, const void* s,
                                      int64_t T, int64_t C, int64_t G, const int64_t* offsets,
                                      int64_t cap, void* qt, void* st, hipStream_t stream) {
  if (G < 1 || G > GCOL_MAX_GROUPS) return hipErrorInvalidValue;
  return launch_requant<true>(elem, out_elem, q, s, cap, C, qt, st, G, offsets, T, stream);
}

}  // namespace mx
