// SwiGLU between an MLP's two products, and its gradient from an 8-bit
// checkpoint, for gfx950.
//
// x [T, 2F] BF16 holds the gates in columns 0 .. F - 1 and the up values in F
// .. 2F - 1.  h = g sig(g) u with sig(g) = 1 / (1 + exp(-g)), computed in FP32
// and rounded to BF16, leaves quantised in 1x32 blocks: the down product's
// operand, without a BF16 copy in memory.  The checkpoint is x itself in 1x32
// blocks, half the bytes of x, and all that the backward pass needs:
//   dg = dh u sig(g) (1 + g (1 - sig(g))),  du = dh g sig(g).
//
// The kernels are bound by HBM.  A lane takes eight columns: 16 bytes of the
// gates and 16 of the up values, four lanes to a block of 32, so that a block's
// maximum needs two lane exchanges and all eight waves fit a SIMD (25 to 36
// registers).  Measured at 131072 x 2048 (E4M3): forward 223 us without the
// checkpoint (6.1 TB/s) and 328 with it (5.8); backward 346 us to BF16 (6.3) and
// 313 quantised (5.3).  One token of 18432: 8.8 us, the host's calls.
#include "mx_columns.h"
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

constexpr int ACT_THREADS = 256;

// sig(g) = p t with no overflow: exp(-|g|) <= 1.  FP32's normal values end near
// sig(-87), but a product with the up value or the gradient need not: below -80
// the sigmoid keeps exp(-80) in p and the rest in t, which the caller multiplies
// last.  Values are formed without t (which is 1) first, and once more in a wave
// that has such a gate (the quantised gradient in 313 us; 325 where a wave takes one
// of two forms, 323 with half of every product).
constexpr float DEEP_GATE = -80.0f;
struct Sigmoid {
  float p, t;
};
template <bool DEEP>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  const float x = DEEP ? fmaxf(-fabsf(g), DEEP_GATE) : -fabsf(g);
  const float e = __expf(x);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  Sigmoid s = {g >= 0.0f ? r : e * r, 1.0f};
  if (DEEP && g < DEEP_GATE) {
    const float t = __expf(g - DEEP_GATE);
    // from 2^-241 on it counts as 0, whatever the gate's size
    if (t == 0.0f) s.p = 0.0f;
    else s.t = t;
  }
  return s;
}

// Whether some lane of the wave has a gate below DEEP_GATE, by its eight gates'
// BF16 bits (a NaN with its sign bit set may count as one).
__device__ __forceinline__ bool any_deep(uint4 gates) {
  constexpr uint32_t DEEP_BITS = 0xC2A0;  // -80
  const uint32_t m = pk_max(pk_max(gates.x, gates.y), pk_max(gates.z, gates.w));
  return __any((m & 0xFFFFu) > DEEP_BITS || (m >> 16) > DEEP_BITS);
}

// Whether some lane of the wave needs the form with t for the gradient: for a
// gate, or for an up value of 1.875 2^127 or more, whose product with p (1 + g (1
// - p)), up to 1.1, may pass FP32's end before the gradient makes it smaller.
// The blocks' scales tell most waves that they have neither.
template <int CE>
__device__ __forceinline__ bool any_far(uint32_t gate_scale, uint32_t up_scale, uint4 gates) {
  constexpr uint32_t first = CE == ELEM_E5M2 ? 118 : 125;  // largest finite value 112; 56 with one less
  constexpr uint32_t end = CE == ELEM_E5M2 ? 240 : 247;    // largest values of 2^128; 1.75 2^127 with one less
  if (!__any(gate_scale >= first || up_scale >= end)) return false;
  return any_deep(gates) || __any(up_scale >= end);
}

template <bool DEEP>
__device__ __forceinline__ void swiglu8(const float g[8], const float u[8], float h[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const Sigmoid s = sigmoid<DEEP>(g[i]);
    h[i] = g[i] * s.p * u[i];
    if (DEEP) h[i] *= s.t;
  }
}

template <bool DEEP>
__device__ __forceinline__ void swiglu_backward8(const float g[8], const float u[8], const float d[8],
                                                 float dg[8], float du[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const Sigmoid s = sigmoid<DEEP>(g[i]);
    const float p = s.p;
    // p (1 + g (1 - p)) lies in -0.1 .. 1.1 and |g p| <= |g|, whatever finite g is
    // (below DEEP_GATE p is 2^-115, and 1 - p as good as 1 - p t)
    const float f = p * (1.0f + g[i] * (1.0f - p));
    // half of it for an up value of 2^127 or more (of these only: what is below
    // FP32's normal values would lose a bit, and a row's bits follow its neighbours)
    const bool end = DEEP && fabsf(u[i]) >= 0x1p127f;
    dg[i] = d[i] * (u[i] * (end ? 0.5f * f : f));
    if (DEEP) dg[i] *= end ? 2.0f * s.t : s.t;
    du[i] = d[i] * (g[i] * p);
    if (DEEP) du[i] *= s.t;
  }
}

__device__ __forceinline__ uint4 as_uint4(u32x4 v) { return make_uint4(v.x, v.y, v.z, v.w); }
__device__ __forceinline__ u32x4 as_vec(uint4 v) { return (u32x4){v.x, v.y, v.z, v.w}; }

// Rows t0 .. of the caller's slice; n8 = F / 8 chunks to a row, nchunks = rows * n8.
template <int EL, int CE, bool CKPT>
__global__ void __launch_bounds__(ACT_THREADS)
swiglu_quant_kernel(const uint16_t* __restrict__ x, uint32_t n8, uint32_t nchunks,
                    uint8_t* __restrict__ q, uint8_t* __restrict__ s, uint8_t* __restrict__ cq,
                    uint8_t* __restrict__ cs) {
  const uint32_t c = blockIdx.x * ACT_THREADS + threadIdx.x;
  if (c >= nchunks) return;
  const uint32_t row = c / n8, k = c - row * n8;
  const int64_t F = 8 * (int64_t)n8;
  const uint16_t* src = x + (int64_t)row * 2 * F + 8 * (int64_t)k;
  const uint4 vg = load_stream16(src), vu = load_stream16(src + F);
  float g[8], u[8], h[8];
  unpack8(as_vec(vg), g);
  unpack8(as_vec(vu), u);
  swiglu8<false>(g, u, h);
  if (__builtin_expect(any_deep(vg), 0)) swiglu8<true>(g, u, h);
  const uint4 vh = as_uint4(pack8(h));
  // a row's quads are whole: n8 is a multiple of 4, and so is nchunks
  const uint32_t sb = scale_byte_t<EL>(quad_max(chunk_absmax(vh)));
  *(uint2*)(q + 8 * (int64_t)c) = cvt8_t<EL>(vh, sb);
  if ((k & 3) == 0) s[c >> 2] = (uint8_t)sb;
  if (CKPT) {
    const uint32_t sg = scale_byte_t<CE>(quad_max(chunk_absmax(vg)));
    const uint32_t su = scale_byte_t<CE>(quad_max(chunk_absmax(vu)));
    const int64_t at = (int64_t)row * 2 * F + 8 * (int64_t)k;
    *(uint2*)(cq + at) = cvt8_t<CE>(vg, sg);
    *(uint2*)(cq + at + F) = cvt8_t<CE>(vu, su);
    if ((k & 3) == 0) {
      cs[at >> 5] = (uint8_t)sg;
      cs[(at + F) >> 5] = (uint8_t)su;
    }
  }
}

// OUT: -1 writes dx in BF16, otherwise it is the element type that dx's rows
// are quantised to.
template <int CE, int OUT>
__global__ void __launch_bounds__(ACT_THREADS)
swiglu_backward_kernel(const uint16_t* __restrict__ dh, const uint8_t* __restrict__ cq,
                       const uint8_t* __restrict__ cs, uint32_t n8, uint32_t nchunks,
                       uint16_t* __restrict__ dx, uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const uint32_t c = blockIdx.x * ACT_THREADS + threadIdx.x;
  if (c >= nchunks) return;
  const uint32_t row = c / n8, k = c - row * n8;
  const int64_t F = 8 * (int64_t)n8;
  const int64_t at = (int64_t)row * 2 * F + 8 * (int64_t)k;
  const u32x2 wg = __builtin_nontemporal_load((const u32x2*)(cq + at));
  const u32x2 wu = __builtin_nontemporal_load((const u32x2*)(cq + at + F));
  const uint4 vd = load_stream16(dh + 8 * (int64_t)c);
  const uint32_t sg = cs[at >> 5], su = cs[(at + F) >> 5];
  float g[8], u[8], d[8], dg[8], du[8];
  const uint4 vg = decode8_t<CE>(make_uint2(wg.x, wg.y), sg);
  unpack8(as_vec(vg), g);
  unpack8(as_vec(decode8_t<CE>(make_uint2(wu.x, wu.y), su)), u);
  unpack8(as_vec(vd), d);
  swiglu_backward8<false>(g, u, d, dg, du);
  u32x4 og = pack8(dg), ou = pack8(du);
  if (__builtin_expect(any_far<CE>(sg, su, vg), 0)) {
    swiglu_backward8<true>(g, u, d, dg, du);
    og = pack8(dg), ou = pack8(du);
  }
  if (OUT < 0) {
    __builtin_nontemporal_store(og, (u32x4*)(dx + at));
    __builtin_nontemporal_store(ou, (u32x4*)(dx + at + F));
  } else {
    constexpr int EL = OUT < 0 ? 0 : OUT;
    const uint32_t bg = scale_byte_t<EL>(quad_max(chunk_absmax(as_uint4(og))));
    const uint32_t bu = scale_byte_t<EL>(quad_max(chunk_absmax(as_uint4(ou))));
    *(uint2*)(q + at) = cvt8_t<EL>(as_uint4(og), bg);
    *(uint2*)(q + at + F) = cvt8_t<EL>(as_uint4(ou), bu);
    if ((k & 3) == 0) {
      s[at >> 5] = (uint8_t)bg;
      s[(at + F) >> 5] = (uint8_t)bu;
    }
  }
}

// Rows of one launch: chunk numbers, rounded up to a workgroup, stay below 2^31.
static int64_t slice_rows(int64_t F) {
  const int64_t rows = (((int64_t)1 << 31) - ACT_THREADS) / (F / 8);
  return rows;
}

template <int EL, int CE>
static hipError_t swiglu_quant_t(const uint16_t* x, int64_t T, int64_t F, uint8_t* q, uint8_t* s,
                                 uint8_t* cq, uint8_t* cs, hipStream_t stream) {
  const int64_t step = slice_rows(F);
  for (int64_t t = 0; t < T; t += step) {
    const int64_t rows = T - t < step ? T - t : step;
    const uint32_t nchunks = (uint32_t)(rows * (F / 8));
    const dim3 grid((nchunks + ACT_THREADS - 1) / ACT_THREADS), block(ACT_THREADS);
    if (cq)
      hipLaunchKernelGGL((swiglu_quant_kernel<EL, CE, true>), grid, block, 0, stream, x + t * 2 * F,
                         (uint32_t)(F / 8), nchunks, q + t * F, s + t * (F / 32), cq + t * 2 * F,
                         cs + t * (F / 16));
    else
      hipLaunchKernelGGL((swiglu_quant_kernel<EL, CE, false>), grid, block, 0, stream, x + t * 2 * F,
                         (uint32_t)(F / 8), nchunks, q + t * F, s + t * (F / 32), nullptr, nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_swiglu_quant(int elem, int ckpt_elem, const void* x, int64_t T, int64_t F, void* q,
                               void* s, void* cq, void* cs, hipStream_t stream) {
#define MX_SWIGLU(EL_, CE_)                                                                       \
  return swiglu_quant_t<EL_, CE_>((const uint16_t*)x, T, F, (uint8_t*)q, (uint8_t*)s, (uint8_t*)cq, \
                                  (uint8_t*)cs, stream)
  if (elem == ELEM_E4M3 && ckpt_elem == ELEM_E4M3) MX_SWIGLU(ELEM_E4M3, ELEM_E4M3);
  if (elem == ELEM_E5M2 && ckpt_elem == ELEM_E4M3) MX_SWIGLU(ELEM_E5M2, ELEM_E4M3);
  if (elem == ELEM_E4M3 && ckpt_elem == ELEM_E5M2) MX_SWIGLU(ELEM_E4M3, ELEM_E5M2);
  if (elem == ELEM_E5M2 && ckpt_elem == ELEM_E5M2) MX_SWIGLU(ELEM_E5M2, ELEM_E5M2);
#undef MX_SWIGLU
  return hipErrorInvalidValue;
}

template <int CE, int OUT>
static hipError_t swiglu_backward_t(const uint16_t* dh, const uint8_t* cq, const uint8_t* cs, int64_t T,
                                    int64_t F, uint16_t* dx, uint8_t* q, uint8_t* s,
                                    hipStream_t stream) {
  const int64_t step = slice_rows(F);
  for (int64_t t = 0; t < T; t += step) {
    const int64_t rows = T - t < step ? T - t : step;
    const uint32_t nchunks = (uint32_t)(rows * (F / 8));
    hipLaunchKernelGGL((swiglu_backward_kernel<CE, OUT>), dim3((nchunks + ACT_THREADS - 1) / ACT_THREADS),
                       dim3(ACT_THREADS), 0, stream, dh + t * F, cq + t * 2 * F, cs + t * (F / 16),
                       (uint32_t)(F / 8), nchunks, OUT < 0 ? dx + t * 2 * F : nullptr,
                       OUT < 0 ? nullptr : q + t * 2 * F, OUT < 0 ? nullptr : s + t * (F / 16));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_swiglu_backward(int ckpt_elem, int out_elem, const void* dh, const void* cq,
                                  const void* cs, int64_t T, int64_t F, void* dx, void* q, void* s,
                                  hipStream_t stream) {
#define MX_SWIGLU_B(CE_, OUT_)                                                                    \
  return swiglu_backward_t<CE_, OUT_>((const uint16_t*)dh, (const uint8_t*)cq, (const uint8_t*)cs, T, \
                                      F, (uint16_t*)dx, (uint8_t*)q, (uint8_t*)s, stream)
  if (ckpt_elem == ELEM_E4M3 && out_elem < 0) MX_SWIGLU_B(ELEM_E4M3, -1);
  if (ckpt_elem == ELEM_E4M3 && out_elem == ELEM_E4M3) MX_SWIGLU_B(ELEM_E4M3, ELEM_E4M3);
  if (ckpt_elem == ELEM_E4M3 && out_elem == ELEM_E5M2) MX_SWIGLU_B(ELEM_E4M3, ELEM_E5M2);
  if (ckpt_elem == ELEM_E5M2 && out_elem < 0) MX_SWIGLU_B(ELEM_E5M2, -1);
  if (ckpt_elem == ELEM_E5M2 && out_elem == ELEM_E4M3) MX_SWIGLU_B(ELEM_E5M2, ELEM_E4M3);
  if (ckpt_elem == ELEM_E5M2 && out_elem == ELEM_E5M2) MX_SWIGLU_B(ELEM_E5M2, ELEM_E5M2);
#undef MX_SWIGLU_B
  return hipErrorInvalidValue;
}

}  // namespace mx
