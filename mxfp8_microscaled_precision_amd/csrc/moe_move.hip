// Moving token rows into the expert order and back, around the MoE experts'
// products.  slots [T, k]: the row of choice (t, j) in the expert order, -1
// for no expert; rows from `used` = offsets[E] on belong to no choice.
//
//   dispatch          y[slot] = x[t]             (BF16, or 1x32-quantised)
//   combine           o[t] = r[t] + sum_j w_tj y[slot]
//   combine backward  dy[slot] = w_tj do[t],  dw_tj = <do[t], y[slot]>
//
// All are bound by HBM bandwidth: 16384 tokens x 8 x 4096 take 245 us to
// dispatch (4.9 TB/s), 128 quantised (5.4), 207 to combine (5.8), 445 for its
// gradient (5.1); a 1 GiB copy runs at 5.1.  Every kernel walks tokens: a token's row is
// read (or written) once and its k expert rows are written (or read) once,
// so no row number has to be inverted.  A slot outside [0, T k) is skipped:
// bad slots give wrong rows but never a bad access.
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_SPAN = 512;          // elements of a row that a wave holds, 8 a lane

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

// Zero rows first, first + step, ... below P.
__device__ __forceinline__ void zero_rows(uint16_t* y, int64_t first, int64_t step, const MoveArgs& a,
                                          int lane) {
  const u32x4 zero = {0, 0, 0, 0};
  for (int64_t r = first; r < a.P; r += step)
    for (int64_t c = 8 * lane; c < a.H; c += MOVE_SPAN) {
      if (c + 8 <= a.H) store_bf16x8<true, false>(y + r * a.H, c, a.H, zero);
      else store_bf16x8<false, false>(y + r * a.H, c, a.H, zero);
    }
}

template <bool WHOLE, bool STREAM>
__device__ __forceinline__ void dispatch_span(const MoveArgs& a, int64_t t, int64_t c,
                                              const uint16_t* x, uint16_t* y) {
  const u32x4 v = load_bf16x8<WHOLE>(x + t * a.H, c, a.H);
  for (int j = 0; j < a.k; j++) {
    const int64_t s = a.slots[t * a.k + j];
    if (s >= 0 && s < a.P) store_bf16x8<WHOLE, STREAM>(y + s * a.H, c, a.H, v);
  }
}

// One wave per (token, span); the rows past the used ones are zeroed by all
// waves in turn.
template <bool STREAM>
__global__ void __launch_bounds__(MOVE_THREADS)
dispatch_kernel(MoveArgs a, const uint16_t* __restrict__ x, uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id(), n = a.T * a.spans;
  const int64_t used = rows_used(a.offsets, a.E, a.P);
  if (id < n) {
    const int64_t t = id / a.spans, c = (id - t * a.spans) * MOVE_SPAN + 8 * lane;
    if (c + 8 <= a.H) dispatch_span<true, STREAM>(a, t, c, x, y);
    else if (c < a.H) dispatch_span<false, STREAM>(a, t, c, x, y);
  }
  const int64_t waves = (int64_t)gridDim.x * (MOVE_THREADS / 64);
  zero_rows(y, used + id, waves, a, lane);
}

// The same, quantised in 1x32 blocks: four lanes hold a block, which is
// quantised once and written to every row of its token.  H % 32 == 0, so a
// block never straddles spans.  (16 elements a lane, with 16-byte payload and
// whole-word scale stores, measured 143 us against 132 at 16384 tokens x 8 x
// 4096, 76 against 81 at x 2 x 7168, the same below.)
template <int EL, bool STREAM>
__global__ void __launch_bounds__(MOVE_THREADS)
dispatch_quant_kernel(MoveArgs a, const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                      uint8_t* __restrict__ s) {
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id(), n = a.T * a.spans;
  const int64_t S = a.H / 32, used = rows_used(a.offsets, a.E, a.P);
  if (id < n) {
    const int64_t t = id / a.spans, c = (id - t * a.spans) * MOVE_SPAN + 8 * lane;
    const bool live = c < a.H;                    // whole quads in or out
    const uint4 v = live ? load_stream16(x + t * a.H + c) : make_uint4(0, 0, 0, 0);
    const uint32_t sb = scale_byte_t<EL>(quad_max(chunk_absmax(v)));
    const uint2 o = cvt8_t<EL>(v, sb);
    for (int j = 0; j < a.k; j++) {
      const int64_t r = a.slots[t * a.k + j];
      if (r >= 0 && r < a.P && live) {
        u32x2* dst = (u32x2*)(q + r * a.H + c);
        if (STREAM) __builtin_nontemporal_store((u32x2){o.x, o.y}, dst);
        else *dst = (u32x2){o.x, o.y};
        if ((lane & 3) == 0) s[r * S + (c >> 5)] = (uint8_t)sb;
      }
    }
  }
  const int64_t waves = (int64_t)gridDim.x * (MOVE_THREADS / 64);
  for (int64_t r = used + id; r < a.P; r += waves) {
    for (int64_t c = 8 * lane; c < a.H; c += MOVE_SPAN) *(uint2*)(q + r * a.H + c) = make_uint2(0, 0);
    for (int64_t c = lane; c < S; c += 64) s[r * S + c] = 0;
  }
}

template <bool WHOLE>
__device__ __forceinline__ void combine_span(const MoveArgs& a, int64_t t, int64_t c, const uint16_t* y,
                                             const float* weights, const uint16_t* residual,
                                             uint16_t* out) {
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  // eight rows in flight
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    u32x4 v[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int j = j0 + u;
      const int64_t s = j < a.k ? a.slots[t * a.k + j] : -1;
      const bool in = s >= 0 && s < a.P;
      v[u] = (u32x4){0, 0, 0, 0};
      w[u] = in && weights ? weights[t * a.k + j] : 1.0f;
      if (in) v[u] = load_bf16x8<WHOLE>(y + s * a.H, c, a.H);
    }
#pragma unroll
    for (int u = 0; u < 8; u++) {
      float f[8];
      unpack8(v[u], f);
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] = fmaf(w[u], f[i], acc[i]);
    }
  }
  if (residual) {
    float f[8];
    unpack8(load_bf16x8<WHOLE>(residual + t * a.H, c, a.H), f);
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] += f[i];
  }
  store_bf16x8<WHOLE, false>(out + t * a.H, c, a.H, pack8(acc));
}

// One wave per (token, span): the k rows' pieces are added in 32 bits, in
// the order of the choices, and rounded once.
__global__ void __launch_bounds__(MOVE_THREADS)
combine_kernel(MoveArgs a, const uint16_t* __restrict__ y, const float* __restrict__ weights,
               const uint16_t* residual, uint16_t* out) {   // out may be residual
  const int lane = threadIdx.x & 63;
  const int64_t id = wave_id();
  if (id >= a.T * a.spans) return;
  const int64_t t = id / a.spans, c = (id - t * a.spans) * MOVE_SPAN + 8 * lane;
  if (c + 8 <= a.H) combine_span<true>(a, t, c, y, weights, residual, out);
  else if (c < a.H) combine_span<false>(a, t, c, y, weights, residual, out);
}

template <bool WHOLE, int KC, bool STREAM>
__device__ __forceinline__ void combine_backward_span(const MoveArgs& a, int64_t t, int64_t c,
                                                      const uint16_t* dout, const uint16_t* y,
                                                      const float* weights, uint16_t* dy,
                                                      float dot[KC]) {
  float d[8];
  unpack8(load_bf16x8<WHOLE>(dout + t * a.H, c, a.H), d);
  // Eight rows to a batch.  Because dy is written in between, their slots come
  // by vector loads, and the wait for a slot also waits for the row asked for
  // before it: a wave has one or two rows in flight.  Many tokens hide that, few
  // do not (figures at the launcher).
#pragma unroll
  for (int j0 = 0; j0 < KC; j0 += 8) {
    if (j0 >= a.k) break;
    int64_t s[8];
    u32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int j = j0 + u;
      s[u] = j < a.k ? a.slots[t * a.k + j] : -1;
      if (s[u] >= a.P) s[u] = -1;
      v[u] = (u32x4){0, 0, 0, 0};
      if (s[u] >= 0) v[u] = load_bf16x8<WHOLE>(y + s[u] * a.H, c, a.H);
    }
#pragma unroll
    for (int u = 0; u < 8; u++) {
      if (s[u] < 0) continue;
      const float w = weights[t * a.k + j0 + u];
      float f[8], g[8];
      unpack8(v[u], f);
#pragma unroll
      for (int i = 0; i < 8; i++) dot[j0 + u] = fmaf(d[i], f[i], dot[j0 + u]), g[i] = w * d[i];
      store_bf16x8<WHOLE, STREAM>(dy + s[u] * a.H, c, a.H, pack8(g));
    }
  }
}

// Sums of N values over the 64 lanes: lane l gets the sum of value l % N.  A
// step halves what each lane holds while it has several values, exchanging the
// half it gives up (N - 1 exchanges), and adds the rest up (log2(64 / N) more).
template <int N>
__device__ __forceinline__ float lane_sums(float* v, int lane) {
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1) {
    const bool upper = (lane & n) != 0;
#pragma unroll
    for (int j = 0; j < n; j++) {
      const float give = upper ? v[j] : v[j + n];
      v[j] = (upper ? v[j + n] : v[j]) + __shfl_xor(give, n, 64);
    }
  }
  float s = v[0];
#pragma unroll
  for (int m = N; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
  return s;
}

// One workgroup per token, of a wave per span up to WAVES; its waves take spans
// in turn, and the k products <do, y> are summed over lanes and then waves in
// a fixed order.
template <int KC, bool STREAM, int WAVES>
__global__ void __launch_bounds__(64 * WAVES)
combine_backward_kernel(MoveArgs a, const uint16_t* __restrict__ dout,
                        const uint16_t* __restrict__ y, const float* __restrict__ weights,
                        uint16_t* __restrict__ dy, float* __restrict__ dweights) {
  __shared__ float part[WAVES][KC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = blockIdx.x;
  // what the end needs, asked for now: one token alone waits for every load
  const int64_t used = rows_used(a.offsets, a.E, a.P);
  const int64_t slot = (int)threadIdx.x < a.k ? a.slots[t * a.k + threadIdx.x] : -1;
  float dot[KC];
#pragma unroll
  for (int j = 0; j < KC; j++) dot[j] = 0.0f;
  const int waves = (int)(blockDim.x >> 6);
  for (int64_t c0 = wave * MOVE_SPAN; c0 < a.H; c0 += waves * MOVE_SPAN) {
    const int64_t c = c0 + 8 * lane;
    if (c + 8 <= a.H) combine_backward_span<true, KC, STREAM>(a, t, c, dout, y, weights, dy, dot);
    else if (c < a.H) combine_backward_span<false, KC, STREAM>(a, t, c, dout, y, weights, dy, dot);
  }
  const float sum = lane_sums<KC>(dot, lane);
  if (lane < KC) part[wave][lane] = sum;
  __syncthreads();
  if ((int)threadIdx.x < a.k) {
    float v = 0.0f;
    for (int w = 0; w < waves; w++) v += part[w][threadIdx.x];
    dweights[t * a.k + threadIdx.x] = slot >= 0 && slot < a.P ? v : 0.0f;
  }
  zero_rows(dy, used + t * waves + wave, (int64_t)gridDim.x * waves, a, lane);
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
// Expert rows in whole 128-byte lines may be written past the caches; rows
// that share a line with the next are merged in L2.
static bool whole_lines(int64_t row_bytes, const void* y) {
  return row_bytes % 128 == 0 && (uintptr_t)y % 128 == 0;
}
// BF16 rows are, from `least` bytes on.  Measured, plain against streaming
// stores: dispatch 133 / 122 us at 16384 tokens x 2 x 7168, 17.6 / 16.1 at 4096
// x 4 x 2048, 122 / 126 at 65536 x 8 x 512; combine's gradient 474 / 447 and
// 239 / 224 there, 55 / 65 at 8192 x 8 x 1000.
static bool stream_rows(int64_t row_bytes, const void* y, int64_t least) {
  return row_bytes >= least && whole_lines(row_bytes, y);
}
// A quantised payload is, from where the 256 MiB last-level cache stops holding
// it, whatever its rows' length (512 to 7168 bytes) and number of choices (1 to
// 12).  Measured, plain against streaming stores: with 8 choices and rows of
// 1024 bytes 29.2 / 32.2 us at 112 MiB, 47.4 / 54.3 at 200, 68.6 / 71.5 at 280,
// 124 / 113 at 448; of 4096 bytes 29.6 / 31.5, 46.6 / 53.3, 69.1 / 73.3, 118 /
// 112; with 4 choices 78.7 / 82.0 at 280, 101 / 94 at 320.  Below 64 MiB either
// is ahead by up to 10%.
constexpr int64_t QUANT_STREAM_BYTES = (int64_t)300 << 20;

hipError_t launch_dispatch(const void* x, int64_t T, int64_t H, int64_t k, int64_t E,
                           const int64_t* offsets, const int32_t* slots, void* y,
                           hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  if (stream_rows(2 * H, y, 4096))
    hipLaunchKernelGGL(dispatch_kernel<true>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint16_t*)y);
  else
    hipLaunchKernelGGL(dispatch_kernel<false>, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint16_t*)y);
  return hipGetLastError();
}

template <int EL>
static void launch_dq(const MoveArgs& a, const void* x, void* q, void* s, hipStream_t stream) {
  if (a.P * a.H >= QUANT_STREAM_BYTES && whole_lines(a.H, q))
    hipLaunchKernelGGL((dispatch_quant_kernel<EL, true>), move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint8_t*)q, (uint8_t*)s);
  else
    hipLaunchKernelGGL((dispatch_quant_kernel<EL, false>), move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                       (const uint16_t*)x, (uint8_t*)q, (uint8_t*)s);
}

hipError_t launch_dispatch_quant(int elem, const void* x, int64_t T, int64_t H, int64_t k, int64_t E,
                                 const int64_t* offsets, const int32_t* slots, void* q, void* s,
                                 hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  if (elem == ELEM_E5M2) launch_dq<ELEM_E5M2>(a, x, q, s, stream);
  else launch_dq<ELEM_E4M3>(a, x, q, s, stream);
  return hipGetLastError();
}

hipError_t launch_combine(const void* y, int64_t T, int64_t H, int64_t k, const int32_t* slots,
                          const float* weights, const void* residual, void* out,
                          hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, 0, nullptr, slots);
  hipLaunchKernelGGL(combine_kernel, move_grid(a), dim3(MOVE_THREADS), 0, stream, a,
                     (const uint16_t*)y, weights, (const uint16_t*)residual, (uint16_t*)out);
  return hipGetLastError();
}

// Four waves to a token fill the chip from 1024 tokens on; fewer tokens take
// their spans side by side.  2000 x 8 x 4096 take 56 us (54 at a copy's rate),
// 300 x 8 x 4096 11.8 (8.2), 280 x 11 x 2880 20.6 (7.2).
template <int KC, bool STREAM, int WAVES>
static void launch_cb_waves(const MoveArgs& a, const void* dout, const void* y, const float* weights,
                            void* dy, float* dweights, hipStream_t stream) {
  const int waves = a.spans < 1 ? 1 : a.spans < WAVES ? a.spans : WAVES;
  hipLaunchKernelGGL((combine_backward_kernel<KC, STREAM, WAVES>), dim3((unsigned)a.T), dim3(64 * waves),
                     0, stream, a, (const uint16_t*)dout, (const uint16_t*)y, weights, (uint16_t*)dy,
                     dweights);
}
template <int KC, bool STREAM>
static void launch_cb(const MoveArgs& a, const void* dout, const void* y, const float* weights,
                      void* dy, float* dweights, hipStream_t stream) {
  if (a.T < 1024) launch_cb_waves<KC, STREAM, 16>(a, dout, y, weights, dy, dweights, stream);
  else launch_cb_waves<KC, STREAM, 4>(a, dout, y, weights, dy, dweights, stream);
}

hipError_t launch_combine_backward(const void* dout, const void* y, int64_t T, int64_t H, int64_t k,
                                   int64_t E, const int64_t* offsets, const int32_t* slots,
                                   const float* weights, void* dy, float* dweights,
                                   hipStream_t stream) {
  const MoveArgs a = move_args(T, H, k, E, offsets, slots);
  if (stream_rows(2 * H, dy, 1024)) {
    if (k <= 8) launch_cb<8, true>(a, dout, y, weights, dy, dweights, stream);
    else launch_cb<16, true>(a, dout, y, weights, dy, dweights, stream);
  } else {
    if (k <= 8) launch_cb<8, false>(a, dout, y, weights, dy, dweights, stream);
    else launch_cb<16, false>(a, dout, y, weights, dy, dweights, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
