// 4-bit MX quantisation for gfx950: BF16 -> E2M1 payload (two codes to a byte)
// + one E8M0 scale per 32 elements, and any MX tensor back to BF16.
//
// A block's scale exponent is the smallest e with amax <= 6 * 2^e, at least
// -127; every element is divided by 2^e and rounded to nearest even onto 0,
// 0.5, 1, 1.5, 2, 3, 4, 6 (v_cvt_scalef32_pk_fp4_bf16).  The pages name 4-bit
// MX for the routed experts' weights (torchtitan-npu MXFP8/HiF8 tutorial,
// step-2 environment table, ENABLE_MXFP4_QAT; practice page, w4a8-mx).
//
// All kernels are bound by HBM: x is read once, every output byte is written
// once.  Measured at 18432 x 7168: rows 52 us (6.4 TB/s), columns 67 (5.0), both
// 84 (4.8; its writes go four ways); back to BF16 51 us from E2M1 and 60 from
// E4M3 (6.5 and 6.7).
#include "mx_columns.h"
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int ROW4_THREADS = 256;
constexpr int ROW4_UNROLL = 4;

// Blocks along rows: as in the 8-bit quantiser the flat array is walked in
// 16-byte chunks, four consecutive lanes to a block; a lane writes 4 bytes.
__global__ void __launch_bounds__(ROW4_THREADS)
quant4_row_kernel(const uint4* __restrict__ x, uint32_t* __restrict__ q, uint8_t* __restrict__ s,
                  int64_t nchunks) {
  const int64_t span = (int64_t)ROW4_THREADS * ROW4_UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * span; base < nchunks; base += (int64_t)gridDim.x * span) {
    uint4 v[ROW4_UNROLL];
#pragma unroll
    for (int u = 0; u < ROW4_UNROLL; u++) {
      const int64_t c = base + u * ROW4_THREADS + threadIdx.x;
      v[u] = c < nchunks ? load_stream16(x + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < ROW4_UNROLL; u++) {
      const int64_t c = base + u * ROW4_THREADS + threadIdx.x;
      // quads are either wholly in range or wholly out (nchunks % 4 == 0)
      const uint32_t sb = scale_byte_t<ELEM_E2M1>(quad_max(chunk_absmax(v[u])));
      if (c < nchunks) {
        q[c] = cvt8_e2m1(v[u], sb);
        if ((threadIdx.x & 3) == 0) s[c >> 2] = (uint8_t)sb;
      }
    }
  }
}

// Blocks down columns, written transposed, and with DUAL the row blocks too,
// from one read.  A workgroup of 8 waves covers 256 rows x 64 NC columns, so
// that a column's payload of the tile is one 128-byte line; wave w takes rows
// 32 w .. 32 w + 31, 64 columns at a time: lane l = 8 g + h holds rows 4 g ..
// 4 g + 3 of columns 8 h .. 8 h + 7 as four 16-byte chunks.  A column block is
// then the lanes h, h + 8, ..., h + 56 and a row block a quad of lanes.  The
// payload leaves through LDS (16-byte chunk k of column c at k ^ (c / 8 & 7),
// free of bank conflicts) in whole lines.
constexpr int TILE4_THREADS = 512;
constexpr int TILE4_ROWS = 256;

typedef __attribute__((address_space(3))) uint8_t lds8;
typedef __attribute__((address_space(3))) uint16_t lds16;
typedef __attribute__((address_space(3))) uint32_t lds32;

template <bool DUAL, int NC>
__global__ void __launch_bounds__(TILE4_THREADS)
quant4_tile_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C, uint8_t* __restrict__ q,
                   uint8_t* __restrict__ s, uint8_t* __restrict__ qt, uint8_t* __restrict__ st) {
  constexpr int COLS = 64 * NC;
  __shared__ __attribute__((aligned(16))) uint8_t lqt_[COLS * 128];  // column payload
  __shared__ __attribute__((aligned(16))) uint8_t lsf_[8 * COLS * 2];  // column scales as BF16: [wave][column]
  __shared__ __attribute__((aligned(16))) uint8_t lq_[DUAL ? TILE4_ROWS * COLS / 2 : 16];
  __shared__ __attribute__((aligned(16))) uint8_t ls_[DUAL ? TILE4_ROWS * COLS / 32 : 16];
  lds8 *lqt = (lds8*)lqt_, *lsf = (lds8*)lsf_, *lq = (lds8*)lq_, *ls = (lds8*)ls_;
  {
    const int64_t z = blockIdx.z, n = R * C;
    x += z * n;
    qt += z * (n >> 1);
    st += z * (n >> 5);
    if (DUAL) {
      q += z * (n >> 1);
      s += z * (n >> 5);
    }
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 3, h = lane & 7;
  // column tiles fastest: neighbours along a row run together
  const int64_t lin = (int64_t)blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  const int64_t tr = lin / gridDim.y, tc = lin - tr * gridDim.y;
  const int64_t R0 = tr * TILE4_ROWS, C0 = tc * COLS;
  const int64_t r0 = R0 + 32 * wave;
  uint4 v[NC][4];
#pragma unroll
  for (int n = 0; n < NC; n++) {
    // R and C are multiples of 32: a wave's rows, and quads of columns, are
    // wholly in or wholly out
    const int64_t c = C0 + 64 * n + 8 * h;
    const bool live = r0 < R && c < C;
#pragma unroll
    for (int i = 0; i < 4; i++)
      v[n][i] = live ? load_stream16(x + (r0 + 4 * g + i) * C + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int n = 0; n < NC; n++) {
    if (DUAL) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t sb = scale_byte_t<ELEM_E2M1>(quad_max(chunk_absmax(v[n][i])));
        const int r = 32 * wave + 4 * g + i;
        *(lds32*)(lq + r * (COLS / 2) + 32 * n + 4 * h) = cvt8_e2m1(v[n][i], sb);
        if ((h & 3) == 0) ls[r * (COLS / 32) + 2 * n + (h >> 2)] = (uint8_t)sb;
      }
    }
    // column maxima, two columns to a word; lanes 2 k and 2 k + 1 of g form the
    // scales of columns 8 h + 2 k and + 1, and every lane reads all back
    const uint32_t M = 0x7FFF7FFFu;
    const uint32_t* w0 = (const uint32_t*)&v[n][0];
    const uint32_t* w1 = (const uint32_t*)&v[n][1];
    const uint32_t* w2 = (const uint32_t*)&v[n][2];
    const uint32_t* w3 = (const uint32_t*)&v[n][3];
    uint32_t m[4];
#pragma unroll
    for (int k = 0; k < 4; k++) m[k] = pk_max(pk_max(w0[k] & M, w1[k] & M), pk_max(w2[k] & M, w3[k] & M));
    const uint32_t two = pair_scale<ELEM_E2M1>(column_max4(m));
    lds8* own = lsf + (wave * NC + n) * 128 + 16 * h;
    *(lds32*)(own + 4 * (g >> 1)) = two;
    const bool bad = __any((two & 0xFFFFu) == 0x7F80u || (two >> 16) == 0x7F80u);
    const u32x4 f = *(const __attribute__((address_space(3))) u32x4*)own;
    const uint32_t fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int k = j >> 1;
      const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
      const uint32_t p01 = __builtin_amdgcn_perm(w1[k], w0[k], sel);
      const uint32_t p23 = __builtin_amdgcn_perm(w3[k], w2[k], sel);
      const uint32_t fb = (j & 1) ? fs[k] & 0xFFFF0000u : fs[k] << 16;
      const float sc = __uint_as_float(fb);
      uint32_t o = 0;
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, p01), sc, 0);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, p23), sc, 1);
      if (bad && fb == 0x7F800000u) o = 0x7777u;
      const int cc = 64 * n + 8 * h + j;
      *(lds16*)(lqt + cc * 128 + ((wave ^ h) << 4) + 2 * g) = (uint16_t)o;
    }
  }
  __syncthreads();

  const int t = threadIdx.x;
  const int64_t rows_here = (R - R0) < TILE4_ROWS ? (R - R0) : TILE4_ROWS;
  const int64_t cols_here = (C - C0) < COLS ? (C - C0) : COLS;
#pragma unroll
  for (int u = 0; u < NC; u++) {  // 8 lanes to a column's 128 bytes
    const int id = t + TILE4_THREADS * u;
    const int col = id >> 3, k = id & 7;
    if (col < cols_here && 32 * k < rows_here) {
      const u32x4 d = *(const __attribute__((address_space(3))) u32x4*)(
          lqt + col * 128 + ((k ^ ((col >> 3) & 7)) << 4));
      __builtin_nontemporal_store(d, (u32x4*)(qt + (C0 + col) * (R >> 1) + (R0 >> 1) + 16 * k));
    }
  }
  if (t < cols_here) {
    uint32_t word[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 8; b++)
      word[b >> 2] |= (((uint32_t)lsf[b * COLS * 2 + 2 * t] >> 7) | ((uint32_t)lsf[b * COLS * 2 + 2 * t + 1] << 1))
                      << (8 * (b & 3));
    uint8_t* dst = st + (C0 + t) * (R >> 5) + (R0 >> 5);
    const int nb = (int)(rows_here >> 5);
    if (nb == 8 && ((uintptr_t)dst & 7) == 0) {
      *(u32x2*)dst = (u32x2){word[0], word[1]};
    } else {
      for (int b = 0; b < nb; b++) dst[b] = (uint8_t)(word[b >> 2] >> (8 * (b & 3)));
    }
  }
  if (DUAL) {
    constexpr int PER = COLS / 32;  // 16-byte chunks, and scales, of a tile row
#pragma unroll
    for (int u = 0; u < TILE4_ROWS * PER / TILE4_THREADS; u++) {
      const int id = t + TILE4_THREADS * u;
      const int r = id / PER, k = id % PER;
      if (r < rows_here && 32 * k < cols_here)
        __builtin_nontemporal_store(
            *(const __attribute__((address_space(3))) u32x4*)(lq + r * (COLS / 2) + 16 * k),
            (u32x4*)(q + (R0 + r) * (C >> 1) + (C0 >> 1) + 16 * k));
    }
    if (t < rows_here) {
      uint8_t* dst = s + (R0 + t) * (C >> 5) + (C0 >> 5);
      const int nb = (int)(cols_here >> 5);
      for (int b = 0; b < nb; b++) dst[b] = ls[t * PER + b];
    }
  }
}

// MX payload back to BF16: a lane takes eight codes and writes 16 bytes.
template <int EL>
__global__ void __launch_bounds__(ROW4_THREADS)
dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, uint4* __restrict__ y,
               int64_t nchunks) {
  const int64_t span = (int64_t)ROW4_THREADS * ROW4_UNROLL;
  for (int64_t base = (int64_t)blockIdx.x * span; base < nchunks; base += (int64_t)gridDim.x * span) {
    uint2 w[ROW4_UNROLL];
    uint32_t sb[ROW4_UNROLL];
#pragma unroll
    for (int u = 0; u < ROW4_UNROLL; u++) {
      const int64_t c = base + u * ROW4_THREADS + threadIdx.x;
      w[u] = make_uint2(0, 0);
      sb[u] = 0;
      if (c < nchunks) {
        if (EL == ELEM_E2M1) {
          w[u].x = __builtin_nontemporal_load((const uint32_t*)q + c);
        } else {
          const u32x2 d = __builtin_nontemporal_load((const u32x2*)q + c);
          w[u] = make_uint2(d.x, d.y);
        }
        sb[u] = s[c >> 2];
      }
    }
#pragma unroll
    for (int u = 0; u < ROW4_UNROLL; u++) {
      const int64_t c = base + u * ROW4_THREADS + threadIdx.x;
      if (c < nchunks) {
        if constexpr (EL == ELEM_E2M1) y[c] = decode8_e2m1(w[u].x, sb[u]);
        else y[c] = decode8_t<EL>(w[u], sb[u]);
      }
    }
  }
}

static unsigned row_blocks(int64_t nchunks) {
  const int64_t span = (int64_t)ROW4_THREADS * ROW4_UNROLL;
  const int64_t blocks = (nchunks + span - 1) / span;
  return (unsigned)(blocks > 65536 ? 65536 : blocks < 1 ? 1 : blocks);
}

hipError_t launch_quant4(int mode, const void* x, int64_t batch, int64_t R, int64_t C, void* q,
                         void* s, void* qt, void* st, hipStream_t stream) {
  if (mode == 0) {
    const int64_t nchunks = batch * R * C / 8;
    hipLaunchKernelGGL(quant4_row_kernel, dim3(row_blocks(nchunks)), dim3(ROW4_THREADS), 0, stream,
                       (const uint4*)x, (uint32_t*)q, (uint8_t*)s, nchunks);
    return hipGetLastError();
  }
  const unsigned nr = (unsigned)((R + TILE4_ROWS - 1) / TILE4_ROWS);
  if (mode == 1)
    hipLaunchKernelGGL((quant4_tile_kernel<false, 1>), dim3(nr, (unsigned)((C + 63) / 64), (unsigned)batch),
                       dim3(TILE4_THREADS), 0, stream, (const uint16_t*)x, R, C, (uint8_t*)q,
                       (uint8_t*)s, (uint8_t*)qt, (uint8_t*)st);
  else if (mode == 2)
    hipLaunchKernelGGL((quant4_tile_kernel<true, 2>), dim3(nr, (unsigned)((C + 127) / 128), (unsigned)batch),
                       dim3(TILE4_THREADS), 0, stream, (const uint16_t*)x, R, C, (uint8_t*)q,
                       (uint8_t*)s, (uint8_t*)qt, (uint8_t*)st);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_dequant(int elem, const void* q, const void* s, int64_t n, void* y,
                          hipStream_t stream) {
  const int64_t nchunks = n / 8;
  const dim3 grid(row_blocks(nchunks)), block(ROW4_THREADS);
  if (elem == ELEM_E2M1)
    hipLaunchKernelGGL(dequant_kernel<ELEM_E2M1>, grid, block, 0, stream, (const uint8_t*)q,
                       (const uint8_t*)s, (uint4*)y, nchunks);
  else if (elem == ELEM_E5M2)
    hipLaunchKernelGGL(dequant_kernel<ELEM_E5M2>, grid, block, 0, stream, (const uint8_t*)q,
                       (const uint8_t*)s, (uint4*)y, nchunks);
  else
    hipLaunchKernelGGL(dequant_kernel<ELEM_E4M3>, grid, block, 0, stream, (const uint8_t*)q,
                       (const uint8_t*)s, (uint4*)y, nchunks);
  return hipGetLastError();
}

}  // namespace mx
