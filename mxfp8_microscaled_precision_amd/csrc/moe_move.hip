// Moving token rows into the expert order and back, around the MoE experts'
// products.  slots [T, k]: the row of choice (t, j) in the expert order, -1
// for no expert; rows from `used` = offsets[E] on belong to no choice.
//
//   dispatch          y[slot] = x[t]             (BF16, or 1x32-quantised)
//   combine           o[t] = r[t] + sum_j w_tj y[slot]
//   combine backward  dy[slot] = w_tj do[t],  dw_tj = <do[t], y[slot]>
//
// All are bound by HBM bandwidth.  Every kernel walks tokens: a token's row is
// read (or written) once and its k expert rows are written (or read) once,
// so no row number has to be inverted.  A slot outside [0, T k) is skipped:
// bad slots give wrong rows but never a bad access.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_SPAN = 512;          // elements of a row that a wave holds, 8 a lane

// Eight elements of a row as packed BF16 pairs.  VEC: lane l holds elements
// 8 l .. 8 l + 7 of the span (rows of a multiple of 8 elements on 16-byte
// alignment); otherwise elements l, l + 64, ..., l + 448, one at a time.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c0, int lane, int64_t H) {
  if (VEC) {
    const int64_t c = c0 + 8 * lane;
    return c < H ? load_stream16(row + c) : make_uint4(0, 0, 0, 0);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t c = c0 + 128 * i + lane, d = c + 64;
    const uint32_t lo = c < H ? row[c] : 0, hi = d < H ? row[d] : 0;
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* row, int64_t c0, int lane, int64_t H, uint4 v) {
  if (VEC) {
    const int64_t c = c0 + 8 * lane;
    if (c < H) *(uint4*)(row + c) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t c = c0 + 128 * i + lane, d = c + 64;
    if (c < H) row[c] = (uint16_t)w[i];
    if (d < H) row[d] = (uint16_t)(w[i] >> 16);
  }
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(uint4 v, float f[8]) {
  f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float f[8]) {
  return make_uint4(cvt_pk_bf16(f[0], f[1]), cvt_pk_bf16(f[2], f[3]), cvt_pk_bf16(f[4], f[5]),
                    cvt_pk_bf16(f[6], f[7]));
}

// Rows of the expert order that hold a choice.
__device__ __forceinline__ int64_t rows_used(const int64_t* offsets, int E, int64_t P) {
  const int64_t u = offsets[E];
  return u < 0 ? 0 : (u > P ? P : u);
}

struct MoveArgs {
  int64_t T, H, P;
  int k, E, spans;                // spans: MOVE_SPAN-wide pieces of a row
  const int64_t* offsets;
  const int32_t* slots;
};

// A wave's number in the grid, as a scalar.
__device__ __forceinline__ int64_t wave_id() {
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  return (int64_t)blockIdx.x * (MOVE_THREADS / 64) + w;
}

// One wave per (token, span); the rows past the used ones are zeroed by all
// waves in turn.
template <bool VEC>
__global__ void __launch_bounds__(MOVE_THREADS)
dispatch_kernel(MoveArgs a, const uint16_t* __restrict__ x, uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id(), n = a.T * a.spans;
  if (id < n) {
    const int64_t t = id / a.spans, c0 = (id - t * a.spans) * MOVE_SPAN;
    const uint4 v = load8<VEC>(x + t * a.H, c0, lane, a.H);
    for (int j = 0; j < a.k; j++) {
      const int64_t s = a.slots[t * a.k + j];
      if (s >= 0 && s < a.P) store8<VEC>(y + s * a.H, c0, lane, a.H, v);
    }
  }
  const int64_t waves = (int64_t)gridDim.x * (MOVE_THREADS / 64);
  for (int64_t r = rows_used(a.offsets, a.E, a.P) + id; r < a.P; r += waves)
    for (int64_t c0 = 0; c0 < a.H; c0 += MOVE_SPAN)
      store8<VEC>(y + r * a.H, c0, lane, a.H, make_uint4(0, 0, 0, 0));
}

// The same, quantised in 1x32 blocks: four lanes hold a block, which is
// quantised once and written to every row of its token.  H % 32 == 0; VEC as
// above (a block never straddles spans).
template <int EL>
__global__ void __launch_bounds__(MOVE_THREADS)
dispatch_quant_kernel(MoveArgs a, const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                      uint8_t* __restrict__ s) {
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id(), n = a.T * a.spans;
  const int64_t S = a.H / 32;
  if (id < n) {
    const int64_t t = id / a.spans, c = (id - t * a.spans) * MOVE_SPAN + 8 * lane;
    const bool live = c < a.H;                    // whole quads in or out
    const uint4 v = live ? load_stream16(x + t * a.H + c) : make_uint4(0, 0, 0, 0);
    const uint32_t sb = scale_byte_t<EL>(quad_max(chunk_absmax(v)));
    const uint2 o = cvt8_t<EL>(v, sb);
    for (int j = 0; j < a.k; j++) {
      const int64_t r = a.slots[t * a.k + j];
      if (r >= 0 && r < a.P && live) {
        *(uint2*)(q + r * a.H + c) = o;
        if ((lane & 3) == 0) s[r * S + (c >> 5)] = (uint8_t)sb;
      }
    }
  }
  const int64_t waves = (int64_t)gridDim.x * (MOVE_THREADS / 64);
  for (int64_t r = rows_used(a.offsets, a.E, a.P) + id; r < a.P; r += waves) {
    for (int64_t c = 8 * lane; c < a.H; c += MOVE_SPAN) *(uint2*)(q + r * a.H + c) = make_uint2(0, 0);
    for (int64_t c = lane; c < S; c += 64) s[r * S + c] = 0;
  }
}

// One wave per (token, span): the k rows' pieces are added in 32 bits, in
// the order of the choices, and rounded once.
template <bool VEC>
__global__ void __launch_bounds__(MOVE_THREADS)
combine_kernel(MoveArgs a, const uint16_t* __restrict__ y, const float* __restrict__ weights,
               const uint16_t* residual, uint16_t* out) {   // out may be residual
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id();
  if (id >= a.T * a.spans) return;
  const int64_t t = id / a.spans, c0 = (id - t * a.spans) * MOVE_SPAN;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int j = 0; j < a.k; j++) {
    const int64_t s = a.slots[t * a.k + j];
    if (s < 0 || s >= a.P) continue;
    const float w = weights ? weights[t * a.k + j] : 1.0f;
    float f[8];
    unpack8(load8<VEC>(y + s * a.H, c0, lane, a.H), f);
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] = fmaf(w, f[i], acc[i]);
  }
  if (residual) {
    float f[8];
    unpack8(load8<VEC>(residual + t * a.H, c0, lane, a.H), f);
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] += f[i];
  }
  store8<VEC>(out + t * a.H, c0, lane, a.H, pack8(acc));
}

constexpr int MOVE_MAX_K = 16;

// One workgroup per token; its waves take spans in turn, and the k products
// <do, y> are summed over lanes and then waves in a fixed order.
template <bool VEC, int KC>
__global__ void __launch_bounds__(MOVE_THREADS)
combine_backward_kernel(MoveArgs a, const uint16_t* __restrict__ dout,
                        const uint16_t* __restrict__ y, const float* __restrict__ weights,
                        uint16_t* __restrict__ dy, float* __restrict__ dweights) {
  __shared__ float part[MOVE_THREADS / 64][MOVE_MAX_K];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = blockIdx.x;
  float dot[KC];
#pragma unroll
  for (int j = 0; j < KC; j++) dot[j] = 0.0f;
  for (int64_t c0 = wave * MOVE_SPAN; c0 < a.H; c0 += MOVE_THREADS / 64 * MOVE_SPAN) {
    float d[8];
    unpack8(load8<VEC>(dout + t * a.H, c0, lane, a.H), d);
#pragma unroll
    for (int j = 0; j < KC; j++) {
      const int64_t s = j < a.k ? a.slots[t * a.k + j] : -1;
      if (s < 0 || s >= a.P) continue;
      const float w = weights[t * a.k + j];
      float f[8], g[8];
      unpack8(load8<VEC>(y + s * a.H, c0, lane, a.H), f);
#pragma unroll
      for (int i = 0; i < 8; i++) dot[j] = fmaf(d[i], f[i], dot[j]), g[i] = w * d[i];
      store8<VEC>(dy + s * a.H, c0, lane, a.H, pack8(g));
    }
  }
#pragma unroll
  for (int j = 0; j < KC; j++) {
    float v = dot[j];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    if (lane == 0) part[wave][j] = v;
  }
  __syncthreads();
  if ((int)threadIdx.x < a.k) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < MOVE_THREADS / 64; w++) v += part[w][threadIdx.x];
    const int64_t s = a.slots[t * a.k + threadIdx.x];
    dweights[t * a.k + threadIdx.x] = s >= 0 && s < a.P ? v : 0.0f;
  }
  const int64_t waves = (int64_t)gridDim.x * (MOVE_THREADS / 64);
  for (int64_t r = rows_used(a.offsets, a.E, a.P) + t * (MOVE_THREADS / 64) + wave; r < a.P; r += waves)
    for (int64_t c0 = 0; c0 < a.H; c0 += MOVE_SPAN)
      store8<VEC>(dy + r * a.H, c0, lane, a.H, make_uint4(0, 0, 0, 0));
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static MoveArgs move_args(int64_t T, int64_t H, int64_t k, int64_t E, const int64_t* offsets,
                          const int32_t* slots) {
  MoveArgs a;
  a.T = T, a.H = H, a.P = T * k, a.k = (int)k, a.E = (int)E;
  a.spans = (int)((H + MOVE_SPAN - 1) / MOVE_SPAN);
  a.offsets = offsets, a.slots = slots;
  return a;
}
static dim3 move_grid(const MoveArgs& a) {
  return dim3((unsigned)((a.T * a.spans + MOVE_THREADS / 64 - 1) / (MOVE_THREADS / 64)));
}
// Whole 16-byte pieces in every row of every operand.
static bool move_vec(int64_t H, uintptr_t ptrs) { return H % 8 == 0 && (ptrs & 15) == 0; }

hipError_t launch_dispatch(const void* x, int64_t T, int64_t H, int64_t k, int64_t E,
                           const int64_t* offsets, const int32_t* slots, void* y,
                           hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  if (move_vec(H, (uintptr_t)x | (uintptr_t)y))
    hipLaunchKernelGGL(dispatch_kernel<true>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint16_t*)y);
  else
    hipLaunchKernelGGL(dispatch_kernel<false>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint16_t*)y);
  return hipGetLastError();
}

hipError_t launch_dispatch_quant(int elem, const void* x, int64_t T, int64_t H, int64_t k, int64_t E,
                                 const int64_t* offsets, const int32_t* slots, void* q, void* s,
                                 hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  if (elem == ELEM_E5M2)
    hipLaunchKernelGGL(dispatch_quant_kernel<ELEM_E5M2>, move_grid(a), dim3(MOVE_THREADS), 0, stream,
                       a, (const uint16_t*)x, (uint8_t*)q, (uint8_t*)s);
  else
    hipLaunchKernelGGL(dispatch_quant_kernel<ELEM_E4M3>, move_grid(a), dim3(MOVE_THREADS), 0, stream,
                       a, (const uint16_t*)x, (uint8_t*)q, (uint8_t*)s);
  return hipGetLastError();
}

hipError_t launch_combine(const void* y, int64_t T, int64_t H, int64_t k, const int32_t* slots,
                          const float* weights, const void* residual, void* out,
                          hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, 0, nullptr, slots);
  if (move_vec(H, (uintptr_t)y | (uintptr_t)residual | (uintptr_t)out))
    hipLaunchKernelGGL(combine_kernel<true>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)y, weights, (const uint16_t*)residual, (uint16_t*)out);
  else
    hipLaunchKernelGGL(combine_kernel<false>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)y, weights, (const uint16_t*)residual, (uint16_t*)out);
  return hipGetLastError();
}

template <bool VEC, int KC>
static void launch_cb(const MoveArgs& a, const void* dout, const void* y, const float* weights,
                      void* dy, float* dweights, hipStream_t stream) {
  hipLaunchKernelGGL((combine_backward_kernel<VEC, KC>), dim3((unsigned)a.T), dim3(MOVE_THREADS), 0,
                     stream, a, (const uint16_t*)dout, (const uint16_t*)y, weights, (uint16_t*)dy,
                     dweights);
}

hipError_t launch_combine_backward(const void* dout, const void* y, int64_t T, int64_t H, int64_t k,
                                   int64_t E, const int64_t* offsets, const int32_t* slots,
                                   const float* weights, void* dy, float* dweights,
                                   hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  const bool vec = move_vec(H, (uintptr_t)dout | (uintptr_t)y | (uintptr_t)dy);
  if (k <= 8) {
    if (vec) launch_cb<true, 8>(a, dout, y, weights, dy, dweights, stream);
    else launch_cb<false, 8>(a, dout, y, weights, dy, dweights, stream);
  } else {
    if (vec) launch_cb<true, 16>(a, dout, y, weights, dy, dweights, stream);
    else launch_cb<false, 16>(a, dout, y, weights, dy, dweights, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
