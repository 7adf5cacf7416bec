// Routing tokens to experts: scores, choice, weights and the expert order the
// grouped GEMM's rows are laid out by, and the weights' gradient.
//
// Forward, per token with logits x[E]:
//   s = softmax(x) or sigmoid(x);  v = s + bias (choice only), -inf where
//   x = -inf; with groups, only experts of the best groups stay (a group's
//   value is its best v or the sum of its best two); the top_k best v are
//   chosen, ties to the lowest index; w = scale * s[chosen], renormalised by
//   their sum.  Then a stable counting sort of the choices by expert.
//
// The choice follows the scores and not their 32-bit roundings.  Without a
// bias (and with groups valued by their best) both score functions keep the
// logits' order, so the logits themselves are compared; otherwise v is
// computed in 64 bits.
//
// A key for the choice is a double whose low 9 mantissa bits are replaced by
// the expert's index (E <= 512), so that keys are distinct, a tie falls to
// the lowest index and one v_max_f64 / v_min_f64 pair moves value and index
// together.  A 32-bit logit keeps all its bits; a 64-bit v keeps 43.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int ROUTE_LANES = 16;                 // lanes that share a token
constexpr int ROUTE_THREADS = 1024;
constexpr int ROUTE_TOKENS = ROUTE_THREADS / ROUTE_LANES;  // tokens of one pass of a workgroup
constexpr int ROUTE_MAX_EXPERTS = 512;
constexpr int ROUTE_MAX_GROUPS = 32;
constexpr int ROUTE_MAX_BLOCKS = 256;

#define MX_NEG_INF (-__builtin_inf())

// Lane exchanges inside a row of 16 lanes, as DPP moves: after the steps
// xor 1 and xor 2 all four lanes of a quad agree, so mirroring half a row
// and then the row stands for xor 4 and xor 8 in a reduction.
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <typename F, typename T>
__device__ __forceinline__ T row_reduce(T v, F f) {
  v = f(v, dpp<DPP_XOR1>(v));
  v = f(v, dpp<DPP_XOR2>(v));
  v = f(v, dpp<DPP_HALF_MIRROR>(v));
  return f(v, dpp<DPP_MIRROR>(v));
}
template <typename T>
__device__ __forceinline__ T row_sum(T v) {
  return row_reduce(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float row_max(float v) {
  return row_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ double row_max(double v) {
  return row_reduce(v, [](double a, double b) { return fmax(a, b); });
}

// Key of value v with index i: NaN below every number, infinities beyond
// every finite value, -0 as 0.
__device__ __forceinline__ double make_key(double v, int i) {
  v = v != v ? -1.7e308 : fmin(fmax(v + 0.0, -1.6e308), 1.6e308);
  const uint64_t b = (uint64_t)__double_as_longlong(v) & ~(uint64_t)511;
  const bool neg = (b >> 63) != 0;
  return __longlong_as_double((long long)(b | (uint64_t)(neg ? i : 511 - i)));
}
__device__ __forceinline__ int key_index(double k) {
  const uint64_t b = (uint64_t)__double_as_longlong(k);
  const int low = (int)(b & 511);
  return (b >> 63) ? low : 511 - low;
}
__device__ __forceinline__ double key_value(double k) {
  return __longlong_as_double((long long)((uint64_t)__double_as_longlong(k) & ~(uint64_t)511));
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void load_logit4(const float* p, float v[4]) {
  const float4 a = *(const float4*)p;
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void load_logit4(const uint16_t* p, float v[4]) {
  const uint2 a = *(const uint2*)p;
  v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
  v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store_logit4(float* p, const float v[4]) {
  *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_logit4(uint16_t* p, const float v[4]) {
  *(uint2*)p = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  *p = (uint16_t)cvt_pk_bf16(v, v);
}

// Chunk c of a token's row held by lane l: experts (16 c + l) * 4 .. + 3;
// -inf past the row.
template <typename IN, int C>
__device__ __forceinline__ void load_row(const IN* __restrict__ row, int E, bool vec, int l,
                                         bool live, float x[C][4]) {
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e0 = (c * ROUTE_LANES + l) * 4;
#pragma unroll
    for (int i = 0; i < 4; i++) x[c][i] = -__builtin_inff();
    if (!live) continue;
    if (vec) {
      if (e0 < E) load_logit4(row + e0, x[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (e0 + i < E) x[c][i] = load_logit(row + e0 + i);
    }
  }
}

// exp(x - m) where m is the row's largest number; a row whose largest is
// +inf shares its weight among the infinite logits.
__device__ __forceinline__ float exp_diff(float x, float m) { return x == m ? 1.0f : expf(x - m); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, n_groups, top_groups, group_max, softmax, renorm, vec;
  float scale;
  float* weights;
  int32_t* experts;
  int64_t* offsets;
  int32_t* slots;
  int32_t* hist;         // [blocks][E] counts of every workgroup's tokens
  int tokens_per_block;
  int blocks;
};

// The chosen groups of a token, as a mask: bit g for group g.
template <int C>
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& a, const double key[C][4], int l) {
  const int gs = a.E / a.n_groups;
  double gk[ROUTE_MAX_GROUPS / ROUTE_LANES];
#pragma unroll
  for (int r = 0; r < ROUTE_MAX_GROUPS / ROUTE_LANES; r++) gk[r] = MX_NEG_INF;
  for (int g = 0; g < a.n_groups; g++) {
    double b1 = MX_NEG_INF, b2 = MX_NEG_INF;
    const int lo = g * gs, hi = lo + gs;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = (c * ROUTE_LANES + l) * 4 + i;
        const double v = e >= lo && e < hi ? key[c][i] : MX_NEG_INF;
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
#define MX_TOP2(CTRL)                                       \
  {                                                         \
    const double o1 = dpp<CTRL>(b1), o2 = dpp<CTRL>(b2);    \
    b2 = fmax(fmin(b1, o1), fmax(b2, o2));                  \
    b1 = fmax(b1, o1);                                      \
  }
    MX_TOP2(DPP_XOR1) MX_TOP2(DPP_XOR2) MX_TOP2(DPP_HALF_MIRROR) MX_TOP2(DPP_MIRROR)
#undef MX_TOP2
    // a group with no unmasked expert stays at -inf
    double v = key_value(b1);
    if (!a.group_max && b2 != MX_NEG_INF) {
      const bool nan = b1 < -1.65e308 || b2 < -1.65e308;
      v = nan ? -1.7e308 : v + key_value(b2);
    }
    const double gkey = b1 == MX_NEG_INF ? MX_NEG_INF : make_key(v, g);
#pragma unroll
    for (int r = 0; r < ROUTE_MAX_GROUPS / ROUTE_LANES; r++)
      if (g == r * ROUTE_LANES + l) gk[r] = gkey;
  }
  uint32_t mask = 0;
  for (int j = 0; j < a.top_groups; j++) {
    double best = gk[0];
#pragma unroll
    for (int r = 1; r < ROUTE_MAX_GROUPS / ROUTE_LANES; r++) best = fmax(best, gk[r]);
    best = row_max(best);
    if (best != MX_NEG_INF) mask |= 1u << key_index(best);
#pragma unroll
    for (int r = 0; r < ROUTE_MAX_GROUPS / ROUTE_LANES; r++)
      if (gk[r] == best) gk[r] = MX_NEG_INF;
  }
  return mask;
}

// Descending list of the KC largest keys of the 16 lanes, in every lane.
template <int C, int KC>
__device__ __forceinline__ void top_keys(const double key[C][4], double top[KC]) {
#pragma unroll
  for (int j = 0; j < KC; j++) top[j] = MX_NEG_INF;
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      double v = key[c][i];
#pragma unroll
      for (int j = 0; j < KC; j++) {
        const double hi = fmax(top[j], v);
        v = fmin(top[j], v);
        top[j] = hi;
      }
    }
  // two descending lists: the larger of a[j] and b[KC - 1 - j] are the KC
  // largest of both, as a bitonic sequence; log2(KC) steps order it
#define MX_MERGE(CTRL)                                                          \
  {                                                                             \
    double o[KC];                                                               \
    _Pragma("unroll") for (int j = 0; j < KC; j++) o[j] = dpp<CTRL>(top[j]);    \
    _Pragma("unroll") for (int j = 0; j < KC; j++)                              \
      top[j] = fmax(top[j], o[KC - 1 - j]);                                     \
    _Pragma("unroll") for (int d = KC / 2; d > 0; d >>= 1)                      \
      _Pragma("unroll") for (int j = 0; j < KC; j++)                            \
        if (!(j & d)) {                                                         \
          const double hi = fmax(top[j], top[j + d]);                           \
          top[j + d] = fmin(top[j], top[j + d]);                                \
          top[j] = hi;                                                          \
        }                                                                       \
  }
  MX_MERGE(DPP_XOR1) MX_MERGE(DPP_XOR2) MX_MERGE(DPP_HALF_MIRROR) MX_MERGE(DPP_MIRROR)
#undef MX_MERGE
}

// One token of the 16 lanes: its experts and weights; returns lane l's choice
// (-1: none, or l >= k).
template <typename IN, int C, int KC, bool SCORED>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t, bool live, int l) {
  const IN* row = (const IN*)a.logits + t * a.E;
  float x[C][4];
  load_row<IN, C>(row, a.E, a.vec, l, live, x);

  // the row's largest number, whether it holds a NaN, and softmax's sum
  float m = -__builtin_inff();
  int nan = 0;
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      m = fmaxf(m, x[c][i]);
      nan |= x[c][i] != x[c][i];
    }
  m = row_max(m);
  nan = row_reduce(nan, [](int p, int q) { return p | q; });

  double key[C][4];
  float sum = 0.0f;
  if (SCORED) {
    double dsum = 1.0;
    if (a.softmax) {
      double part = 0.0;
#pragma unroll
      for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const double z = x[c][i] == m ? 1.0 : exp((double)x[c][i] - (double)m);
          part += z == z ? z : 0.0;
        }
      dsum = 1.0 / row_sum(part);
    }
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = (c * ROUTE_LANES + l) * 4 + i;
        double v;
        if (a.softmax)
          v = (x[c][i] == m ? 1.0 : exp((double)x[c][i] - (double)m)) * dsum;
        else
          v = 1.0 / (1.0 + exp(-(double)x[c][i]));
        if (a.bias && e < a.E) v += (double)a.bias[e];
        key[c][i] = x[c][i] == -__builtin_inff() || v == MX_NEG_INF ? MX_NEG_INF : make_key(v, e);
      }
  } else {
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = (c * ROUTE_LANES + l) * 4 + i;
        key[c][i] = x[c][i] == -__builtin_inff() ? MX_NEG_INF : make_key((double)x[c][i], e);
      }
  }
  if (a.softmax && !a.renorm) {
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float z = exp_diff(x[c][i], m);
        sum += z == z ? z : 0.0f;
      }
    sum = row_sum(sum);
  }

  if (a.n_groups > 1) {
    const uint32_t keep = choose_groups<C>(a, key, l);
    const int gs = a.E / a.n_groups;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int g = ((c * ROUTE_LANES + l) * 4 + i) / gs;
        if (g >= a.n_groups || !((keep >> g) & 1)) key[c][i] = MX_NEG_INF;
      }
  }

  double top[KC];
  top_keys<C, KC>(key, top);
  double mine = top[0];
#pragma unroll
  for (int j = 1; j < KC; j++) mine = l == j ? top[j] : mine;
  const bool has = live && l < a.k && l < KC && mine != MX_NEG_INF;
  const int e = has ? key_index(mine) : -1;

  // the chosen scores; renormalised ones as ratios of terms that share a
  // factor, so that they hold where every chosen score underflows
  const float xe = has ? load_logit(row + e) : -__builtin_inff();
  float w;
  if (a.renorm) {
    const float big = row_max(xe);
    float u;
    if (a.softmax) {
      u = exp_diff(xe, big);
    } else {
      const float s = fminf(big, 0.0f);      // sigmoid(x) exp(-s) = 1 / (exp(s) + exp(s - x))
      u = xe == -__builtin_inff() ? 0.0f : 1.0f / (expf(s) + expf(s - xe));
    }
    if (!has) u = 0.0f;
    w = u / row_sum(u);
  } else {
    w = a.softmax ? exp_diff(xe, m) / sum : 1.0f / (1.0f + expf(-xe));
  }
  if (a.softmax && nan) w = __builtin_nanf("");
  if (live && l < a.k) {
    a.weights[t * a.k + l] = has ? w * a.scale : 0.0f;
    a.experts[t * a.k + l] = e;
  }
  return e;
}

// Exclusive prefix sum over tot[0 .. E), in place, by the first wave.
__device__ __forceinline__ void scan_experts(int* tot, int E) {
  if (threadIdx.x < 64) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + (int)threadIdx.x;
      const int v = e < E ? tot[e] : 0;
      int s = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64);
        if ((int)threadIdx.x >= d) s += o;
      }
      if (e < E) tot[e] = carry + s - v;
      carry += __shfl(s, 63, 64);
    }
    if (threadIdx.x == 0) tot[E] = carry;
  }
}

// Rows of the choices [p0, p1) in the expert order: base[e] is the next free
// row of expert e before them.  Wave w ranks 64 consecutive choices, equal
// experts found by one ballot per bit of the expert's index.
__device__ __forceinline__ void place_pairs(const int32_t* experts,
                                            int32_t* slots, int64_t p0, int64_t p1,
                                            int E, int* base, int* wave_cnt) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int NW = ROUTE_THREADS / 64;
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  for (int64_t q = p0; q < p1; q += ROUTE_THREADS) {
    for (int i = threadIdx.x; i < NW * E; i += ROUTE_THREADS) wave_cnt[i] = 0;
    __syncthreads();
    const int64_t p = q + threadIdx.x;
    const int e = p < p1 ? experts[p] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < nbits; b++) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) wave_cnt[wave * E + e] = __popcll(same);
    __syncthreads();
    for (int x = threadIdx.x; x < E; x += ROUTE_THREADS) {
      int run = base[x];
      for (int w = 0; w < NW; w++) {
        const int n = wave_cnt[w * E + x];
        wave_cnt[w * E + x] = run;
        run += n;
      }
      base[x] = run;
    }
    __syncthreads();
    if (p < p1) slots[p] = e >= 0 ? wave_cnt[wave * E + e] + rank : -1;
    __syncthreads();
  }
}

// Choices and weights of a workgroup's tokens and its count per expert; with
// one workgroup, the expert order too.
template <typename IN, int C, int KC, bool SCORED>
__global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(RouteArgs a) {
  __shared__ int cnt[ROUTE_MAX_EXPERTS + 1];
  __shared__ int wave_cnt[ROUTE_THREADS / 64 * ROUTE_MAX_EXPERTS];
  const int l = threadIdx.x & (ROUTE_LANES - 1);
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) cnt[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  for (int64_t b = t0; b < t1; b += ROUTE_TOKENS) {
    const int64_t t = b + threadIdx.x / ROUTE_LANES;
    const int e = route_token<IN, C, KC, SCORED>(a, t < t1 ? t : t1 - 1, t < t1, l);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (a.blocks > 1) {
    for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS)
      a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
    return;
  }
  scan_experts(cnt, a.E);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += ROUTE_THREADS) a.offsets[e] = cnt[e];
  __syncthreads();
  place_pairs(a.experts, a.slots, t0 * a.k, t1 * a.k, a.E, cnt, wave_cnt);
}

// The expert order of workgroup b's choices: its base row per expert is the
// expert's offset plus the counts of the workgroups before b.
__global__ void __launch_bounds__(ROUTE_THREADS) route_place_kernel(RouteArgs a) {
  __shared__ int tot[ROUTE_MAX_EXPERTS + 1];
  __shared__ int base[ROUTE_MAX_EXPERTS];
  __shared__ int wave_cnt[ROUTE_THREADS / 64 * ROUTE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) tot[e] = base[e] = 0;
  __syncthreads();
  const int b = blockIdx.x;
  // thread = (segment of the workgroups, expert)
  const int segs = ROUTE_THREADS / a.E;          // E <= 512: at least two
  const int seg = (int)threadIdx.x / a.E, e = (int)threadIdx.x - seg * a.E;
  if (seg < segs) {
    int all = 0, before = 0;
    for (int i = seg; i < a.blocks; i += segs) {
      const int n = a.hist[(int64_t)i * a.E + e];
      all += n;
      before += i < b ? n : 0;
    }
    atomicAdd(&tot[e], all);
    atomicAdd(&base[e], before);
  }
  __syncthreads();
  scan_experts(tot, a.E);
  __syncthreads();
  for (int x = threadIdx.x; x < a.E; x += ROUTE_THREADS) base[x] += tot[x];
  if (b == 0)
    for (int x = threadIdx.x; x <= a.E; x += ROUTE_THREADS) a.offsets[x] = tot[x];
  __syncthreads();
  const int64_t t0 = (int64_t)b * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  place_pairs(a.experts, a.slots, t0 * a.k, t1 * a.k, a.E, base, wave_cnt);
}

// ---------------------------------------------------------------------------
// Gradient of the weights with respect to the logits.  With a_j = s_j / S
// over the chosen scores and G = sum_j g_j a_j:
//   softmax, renormalised:  dx[e_j] = scale a_j (g_j - G)
//   sigmoid, renormalised:  dx[e_j] = scale a_j (g_j - G) (1 - s_j)
//   sigmoid:                dx[e_j] = scale g_j s_j (1 - s_j)
//   softmax:                dx[e] = p_e (scale g_j [e = e_j] - scale sum_j g_j p_ej)
// The first three are zero off the chosen experts and read only their logits.
// ---------------------------------------------------------------------------
struct RouteBackwardArgs {
  const float* dweights;
  const void* logits;
  const int32_t* experts;
  void* dlogits;
  int64_t T;
  int E, k, softmax, renorm, vec;
  float scale;
};

template <typename IN, int C>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteBackwardArgs a) {
  const int l = threadIdx.x & (ROUTE_LANES - 1);
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / ROUTE_LANES;
  const bool live = t < a.T;
  const int64_t tt = live ? t : a.T - 1;
  const IN* row = (const IN*)a.logits + tt * a.E;
  const bool dense = a.softmax && !a.renorm;
  int e = l < a.k ? a.experts[tt * a.k + l] : -1;
  if (e >= a.E) e = -1;
  const bool has = e >= 0;
  const float g = has ? a.dweights[tt * a.k + l] : 0.0f;
  const float xe = has ? load_logit(row + e) : -__builtin_inff();
  float x[C][4];
  float m = -__builtin_inff(), sum = 0.0f;
  float d = 0.0f, dot = 0.0f;                  // lane l's choice's own term; the row's common term
  if (dense) {
    load_row<IN, C>(row, a.E, a.vec, l, true, x);
    int nan = 0;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        m = fmaxf(m, x[c][i]);
        nan |= x[c][i] != x[c][i];
      }
    m = row_max(m);
    nan = row_reduce(nan, [](int p, int q) { return p | q; });
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        x[c][i] = x[c][i] == -__builtin_inff() ? 0.0f : exp_diff(x[c][i], m);
        sum += x[c][i];
      }
    sum = row_sum(sum);
    const float inv = sum > 0.0f || nan ? 1.0f / sum : 0.0f;   // a row of masked experts: no gradient
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) x[c][i] *= inv;
    const float p = has && xe != -__builtin_inff() ? exp_diff(xe, m) * inv : 0.0f;
    d = has ? a.scale * g * p : 0.0f;
    dot = row_sum(d);
  } else if (a.renorm) {
    const float big = row_max(xe);
    float u = 0.0f;
    if (has && xe != -__builtin_inff()) {
      if (a.softmax) {
        u = exp_diff(xe, big);
      } else {
        const float s = fminf(big, 0.0f);
        u = 1.0f / (expf(s) + expf(s - xe));
      }
    }
    const float S = row_sum(u);
    const float aj = S == 0.0f ? 0.0f : u / S;
    const float G = row_sum(g * aj);
    d = a.scale * aj * (g - G);
    if (!a.softmax) d *= 1.0f / (1.0f + expf(xe));
  } else {
    const float s = 1.0f / (1.0f + expf(-xe));
    d = a.scale * g * s / (1.0f + expf(xe));
  }
  if (!has) d = 0.0f;

  float out[C][4];
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) out[c][i] = dense ? -x[c][i] * dot : 0.0f;
  const int lane0 = (int)(threadIdx.x & 63) & ~(ROUTE_LANES - 1);
  for (int j = 0; j < a.k; j++) {
    const int ej = __shfl(e, lane0 + j, 64);
    const float dj = __shfl(d, lane0 + j, 64);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        out[c][i] += (c * ROUTE_LANES + l) * 4 + i == ej ? dj : 0.0f;
  }
  if (!live) return;
  IN* dst = (IN*)a.dlogits + t * a.E;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e0 = (c * ROUTE_LANES + l) * 4;
    if (a.vec) {
      if (e0 < a.E) store_logit4(dst + e0, out[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (e0 + i < a.E) store_logit(dst + e0 + i, out[c][i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static void route_split(int64_t T, int* blocks, int* tokens_per_block) {
  int64_t per = (T + ROUTE_MAX_BLOCKS - 1) / ROUTE_MAX_BLOCKS;
  per = (per + ROUTE_TOKENS - 1) / ROUTE_TOKENS * ROUTE_TOKENS;
  if (per < ROUTE_TOKENS) per = ROUTE_TOKENS;
  *tokens_per_block = (int)per;
  *blocks = (int)((T + per - 1) / per);
}

size_t route_workspace(int64_t T, int64_t E) {
  int blocks, per;
  route_split(T, &blocks, &per);
  return blocks > 1 ? sizeof(int32_t) * (size_t)blocks * (size_t)E : 0;
}

template <typename IN, int C, int KC>
static void launch_route_kc(bool scored, const RouteArgs& a, hipStream_t stream) {
  if (scored)
    hipLaunchKernelGGL((route_kernel<IN, C, KC, true>), dim3(a.blocks), dim3(ROUTE_THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL((route_kernel<IN, C, KC, false>), dim3(a.blocks), dim3(ROUTE_THREADS), 0, stream, a);
}
template <typename IN, int C>
static void launch_route_c(bool scored, const RouteArgs& a, hipStream_t stream) {
  if (a.k <= 8) launch_route_kc<IN, C, 8>(scored, a, stream);
  else launch_route_kc<IN, C, 16>(scored, a, stream);
}
template <typename IN>
static void launch_route_in(bool scored, const RouteArgs& a, hipStream_t stream) {
  if (a.E <= 64) launch_route_c<IN, 1>(scored, a, stream);
  else if (a.E <= 128) launch_route_c<IN, 2>(scored, a, stream);
  else if (a.E <= 256) launch_route_c<IN, 4>(scored, a, stream);
  else launch_route_c<IN, 8>(scored, a, stream);
}

hipError_t launch_route(int softmax, int f32, const void* logits, const float* bias, int64_t T,
                        int64_t E, int64_t k, int64_t n_groups, int64_t top_groups, int group_max,
                        int renorm, float scale, float* weights, int32_t* experts,
                        int64_t* offsets, int32_t* slots, void* workspace, hipStream_t stream) {
  RouteArgs a;
  a.logits = logits, a.bias = bias, a.T = T, a.E = (int)E, a.k = (int)k;
  a.n_groups = (int)n_groups, a.top_groups = (int)top_groups, a.group_max = group_max;
  a.softmax = softmax, a.renorm = renorm, a.scale = scale;
  a.weights = weights, a.experts = experts, a.offsets = offsets, a.slots = slots;
  a.hist = (int32_t*)workspace;
  // four logits at once where every row starts on their alignment
  a.vec = E % 4 == 0 && ((uintptr_t)logits & (f32 ? 15 : 7)) == 0;
  route_split(T, &a.blocks, &a.tokens_per_block);
  const bool scored = bias != nullptr || (n_groups > 1 && !group_max);
  if (f32) launch_route_in<float>(scored, a, stream);
  else launch_route_in<uint16_t>(scored, a, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 1) return e;
  hipLaunchKernelGGL(route_place_kernel, dim3(a.blocks), dim3(ROUTE_THREADS), 0, stream, a);
  return hipGetLastError();
}

template <typename IN>
static void launch_route_backward_in(const RouteBackwardArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T * ROUTE_LANES + 255) / 256));
  if (a.E <= 64) hipLaunchKernelGGL((route_backward_kernel<IN, 1>), grid, dim3(256), 0, stream, a);
  else if (a.E <= 128) hipLaunchKernelGGL((route_backward_kernel<IN, 2>), grid, dim3(256), 0, stream, a);
  else if (a.E <= 256) hipLaunchKernelGGL((route_backward_kernel<IN, 4>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((route_backward_kernel<IN, 8>), grid, dim3(256), 0, stream, a);
}

hipError_t launch_route_backward(int softmax, int f32, int64_t T, int64_t E, int64_t k, int renorm,
                                 float scale, const float* dweights, const void* logits,
                                 const int32_t* experts, void* dlogits, hipStream_t stream) {
  RouteBackwardArgs a;
  a.dweights = dweights, a.logits = logits, a.experts = experts, a.dlogits = dlogits;
  a.T = T, a.E = (int)E, a.k = (int)k, a.softmax = softmax, a.renorm = renorm, a.scale = scale;
  const uintptr_t align = f32 ? 15 : 7;
  a.vec = E % 4 == 0 && (((uintptr_t)logits | (uintptr_t)dlogits) & align) == 0;
  if (f32) launch_route_backward_in<float>(a, stream);
  else launch_route_backward_in<uint16_t>(a, stream);
  return hipGetLastError();
}

}  // namespace mx
