// Global gradient norm over many tensors, and clipping.
//
//   n = sqrt(sum over all tensors of g^2),  g *= min(1, max_norm / (n + 1e-6))
//
// Bound by HBM bandwidth: the norm of 2.1 GB takes 328 us (6.5 TB/s), clipping
// it 1157 (three passes, 5.5 TB/s).  The tensors are cut into pieces of 32 KiB;
// a launch takes up to GRAD_TENSORS tensors, whose addresses travel in the
// kernel's arguments (no table in device memory, so a captured graph holds
// them), and its workgroups take pieces in turn.  Squares are added in 64 bits:
// they neither overflow nor underflow for any finite gradient, and the norm and
// the scaled gradients are rounded once.  Every workgroup writes its sum to the
// workspace and the sums are added in a fixed order, so the norm is the same on
// every run.
//
// A tensor that does not start on 16 bytes is read and written element by
// element: 1157 us for the norm of 2.1 GB of BF16 and 2680 to clip it, 681 and
// 1634 of FP32.  Every workgroup that scales adds up the sums of all launches,
// which grows with the square of a list's length past 160 tensors.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_PIECE = 32768;                       // bytes
constexpr int GRAD_LOADS = GRAD_PIECE / 16 / GRAD_THREADS;
constexpr int GRAD_BLOCKS = 2048;                       // workgroups of one launch

struct GradTensor {
  void* p;
  int64_t n;               // elements
  int32_t first;           // its first piece in the launch
  int32_t f32;
};
struct GradTable {
  int count;
  int pieces;
  GradTensor t[GRAD_TENSORS];
};

// A piece's tensor and its elements [lo, lo + n).
struct GradPiece {
  char* p;
  int n;
  bool f32, vec;
};
template <int BYTES>
__device__ __forceinline__ GradPiece grad_piece(const GradTable& a, int piece) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].first <= piece) lo = mid;
    else hi = mid - 1;
  }
  GradPiece g;
  g.f32 = a.t[lo].f32 != 0;
  const int per = g.f32 ? BYTES / 4 : BYTES / 2;
  const int64_t at = (int64_t)(piece - a.t[lo].first) * per;
  const int64_t left = a.t[lo].n - at;
  g.n = left < per ? (int)left : per;
  g.p = (char*)a.t[lo].p + at * (g.f32 ? 4 : 2);
  g.vec = ((uintptr_t)g.p & 15) == 0;
  return g;
}

__device__ __forceinline__ double square(float f, double acc) {
  const double d = (double)f;
  return fma(d, d, acc);
}
__device__ __forceinline__ float bf_of(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ double square4(uint4 v, bool f32, double acc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (f32) {
      acc = square(__uint_as_float(w[i]), acc);
    } else {
      acc = square(__uint_as_float(w[i] << 16), acc);
      acc = square(__uint_as_float(w[i] & 0xFFFF0000u), acc);
    }
  }
  return acc;
}

// The coefficient stays in 64 bits: a norm past FP32's range has one that
// FP32 holds with few bits or none.
__device__ __forceinline__ float scaled(float g, double coef) { return (float)((double)g * coef); }
__device__ __forceinline__ uint4 scaled4(uint4 v, bool f32, double coef) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++)
    w[i] = f32 ? __float_as_uint(scaled(__uint_as_float(w[i]), coef))
               : cvt_pk_bf16(scaled(__uint_as_float(w[i] << 16), coef),
                             scaled(__uint_as_float(w[i] & 0xFFFF0000u), coef));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void scale1(char* p, int i, bool f32, double coef) {
  if (f32) {
    ((float*)p)[i] = scaled(((const float*)p)[i], coef);
  } else {
    const float f = scaled(bf_of(((const uint16_t*)p)[i]), coef);
    ((uint16_t*)p)[i] = (uint16_t)cvt_pk_bf16(f, f);
  }
}

// Sum over a workgroup, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < GRAD_THREADS / 64; w++) s += part[w];
  return s;
}

__global__ void __launch_bounds__(GRAD_THREADS) grad_square_kernel(GradTable a, double* sums) {
  __shared__ double part[GRAD_THREADS / 64];
  double acc = 0.0;
  for (int piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
    const GradPiece g = grad_piece<GRAD_PIECE>(a, piece);
    const int each = g.f32 ? 4 : 8, whole = g.vec ? g.n / each : 0;
    uint4 v[GRAD_LOADS];
#pragma unroll
    for (int u = 0; u < GRAD_LOADS; u++) {
      const int i = u * GRAD_THREADS + threadIdx.x;
      v[u] = i < whole ? load_stream16((const uint4*)g.p + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < GRAD_LOADS; u++) acc = square4(v[u], g.f32, acc);
    for (int i = whole * each + threadIdx.x; i < g.n; i += GRAD_THREADS)
      acc = square(g.f32 ? ((const float*)g.p)[i] : bf_of(((const uint16_t*)g.p)[i]), acc);
  }
  const double s = block_sum(acc, part);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// Short lists: one workgroup sums and scales in a single launch, a wave to a
// piece, of 4 KiB here.  CLIP as below.
constexpr int GRAD_SHORT_THREADS = 1024;
constexpr int GRAD_SHORT_PIECE = 4096;
template <bool CLIP>
__global__ void __launch_bounds__(GRAD_SHORT_THREADS)
grad_short_kernel(GradTable a, float max_norm, float* norm) {
  constexpr int WAVES = GRAD_SHORT_THREADS / 64, LOADS = GRAD_SHORT_PIECE / 16 / 64;
  __shared__ double part[WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  double acc = 0.0;
  for (int piece = wave; piece < a.pieces; piece += WAVES) {
    const GradPiece g = grad_piece<GRAD_SHORT_PIECE>(a, piece);
    const int each = g.f32 ? 4 : 8, whole = g.vec ? g.n / each : 0;
    uint4 v[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; u++)
      v[u] = lane + 64 * u < whole ? ((const uint4*)g.p)[lane + 64 * u] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < LOADS; u++) acc = square4(v[u], g.f32, acc);
    for (int i = whole * each + lane; i < g.n; i += 64)
      acc = square(g.f32 ? ((const float*)g.p)[i] : bf_of(((const uint16_t*)g.p)[i]), acc);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) acc += __shfl_xor(acc, m, 64);
  if (lane == 0) part[wave] = acc;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) sum += part[w];
  const double total = sqrt(sum);
  if (threadIdx.x == 0) *norm = (float)total;
  if (!CLIP) return;
  const double coef = (double)max_norm / (total + 1e-6);
  if (coef >= 1.0) return;                     // nothing to scale; a NaN goes on
  for (int piece = wave; piece < a.pieces; piece += WAVES) {
    const GradPiece g = grad_piece<GRAD_SHORT_PIECE>(a, piece);
    const int each = g.f32 ? 4 : 8, whole = g.vec ? g.n / each : 0;
    uint4 v[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; u++)
      v[u] = lane + 64 * u < whole ? ((const uint4*)g.p)[lane + 64 * u] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < LOADS; u++)
      if (lane + 64 * u < whole) ((uint4*)g.p)[lane + 64 * u] = scaled4(v[u], g.f32, coef);
    for (int i = whole * each + lane; i < g.n; i += 64) scale1(g.p, i, g.f32, coef);
  }
}

__device__ __forceinline__ double total_norm(const double* sums, int n, double* part) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += GRAD_THREADS) v += sums[i];
  return sqrt(block_sum(v, part));
}

__global__ void __launch_bounds__(GRAD_THREADS)
grad_norm_kernel(const double* sums, int n, float* norm) {
  __shared__ double part[GRAD_THREADS / 64];
  const double v = total_norm(sums, n, part);
  if (threadIdx.x == 0) *norm = (float)v;
}

__global__ void __launch_bounds__(GRAD_THREADS)
grad_scale_kernel(GradTable a, const double* sums, int n, float max_norm, float* norm) {
  __shared__ double part[GRAD_THREADS / 64];
  const double v = total_norm(sums, n, part);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  const double coef = (double)max_norm / (v + 1e-6);
  if (coef >= 1.0) return;                    // nothing to scale; a NaN goes on
  // the pieces that were read last come first: they are still in the caches
  for (int at = blockIdx.x; at < a.pieces; at += gridDim.x) {
    const GradPiece g = grad_piece<GRAD_PIECE>(a, a.pieces - 1 - at);
    const int each = g.f32 ? 4 : 8, whole = g.vec ? g.n / each : 0;
    uint4 v4[GRAD_LOADS];
#pragma unroll
    for (int u = 0; u < GRAD_LOADS; u++) {
      const int i = u * GRAD_THREADS + threadIdx.x;
      v4[u] = i < whole ? load_stream16((const uint4*)g.p + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < GRAD_LOADS; u++) {
      const int i = u * GRAD_THREADS + threadIdx.x;
      const uint4 w = scaled4(v4[u], g.f32, coef);
      if (i < whole) ((uint4*)g.p)[i] = w;
    }
    for (int i = whole * each + threadIdx.x; i < g.n; i += GRAD_THREADS) scale1(g.p, i, g.f32, coef);
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

// The table of tensors i0 .. of a list, as many as one launch takes; returns
// the next tensor.  Empty tensors are left out.  The caller bounds the list's
// bytes so that pieces are numbered in 32 bits.
static int64_t grad_table(int64_t i0, int64_t n, void* const* tensors, const int64_t* numels,
                          const int* f32, int bytes, GradTable* a) {
  a->count = 0;
  int64_t pieces = 0, i = i0;
  for (; i < n && a->count < GRAD_TENSORS; i++) {
    if (numels[i] == 0) continue;
    const int64_t per = f32[i] ? bytes / 4 : bytes / 2;
    GradTensor& t = a->t[a->count++];
    t.p = tensors[i], t.n = numels[i], t.first = (int32_t)pieces, t.f32 = f32[i];
    pieces += (numels[i] + per - 1) / per;
  }
  a->pieces = (int)pieces;
  return i;
}

// Up to 32 pieces (128 KiB) one workgroup takes no longer than two launches
// (5.5 us for the norm, 10 with clipping, at either side) and saves one.
constexpr int GRAD_SHORT_PIECES = 32;

static int grad_grid(const GradTable& a) { return a.pieces < GRAD_BLOCKS ? a.pieces : GRAD_BLOCKS; }

// Sums the workspace holds: one per workgroup of every launch.
size_t grad_workspace(int64_t n) {
  return sizeof(double) * (size_t)GRAD_BLOCKS * (size_t)((n + GRAD_TENSORS - 1) / GRAD_TENSORS);
}

hipError_t launch_grad(int64_t n, void* const* tensors, const int64_t* numels, const int* f32,
                       int clip, float max_norm, float* norm, void* workspace, hipStream_t stream) {
  double* sums = (double*)workspace;
  int filled = 0;
  GradTable a;
  if (grad_table(0, n, tensors, numels, f32, GRAD_SHORT_PIECE, &a) == n && a.pieces <= GRAD_SHORT_PIECES) {
    if (clip)
      hipLaunchKernelGGL(grad_short_kernel<true>, dim3(1), dim3(GRAD_SHORT_THREADS), 0, stream, a,
                         max_norm, norm);
    else
      hipLaunchKernelGGL(grad_short_kernel<false>, dim3(1), dim3(GRAD_SHORT_THREADS), 0, stream, a,
                         max_norm, norm);
    return hipGetLastError();
  }
  for (int64_t i = 0; i < n;) {
    i = grad_table(i, n, tensors, numels, f32, GRAD_PIECE, &a);
    if (a.count == 0) break;
    const int grid = grad_grid(a);
    hipLaunchKernelGGL(grad_square_kernel, dim3(grid), dim3(GRAD_THREADS), 0, stream, a, sums + filled);
    filled += grid;
  }
  if (!clip) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(GRAD_THREADS), 0, stream, sums, filled, norm);
    return hipGetLastError();
  }
  bool first = true;
  for (int64_t i = 0; i < n;) {
    i = grad_table(i, n, tensors, numels, f32, GRAD_PIECE, &a);
    if (a.count == 0) break;
    hipLaunchKernelGGL(grad_scale_kernel, dim3(grad_grid(a)), dim3(GRAD_THREADS), 0, stream, a, sums,
                       filled, max_norm, first ? norm : nullptr);
    first = false;
  }
  return hipGetLastError();
}

}  // namespace mx
