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
// bias both score functions keep the logits' order, so the logits themselves
// are compared (and only a group's best two are scored, in 64 bits).  With a
// bias v is first taken from 32-bit scores; where two values that the choice
// turns on lie closer than their error, the wave chooses again from 64 bits.
//
// A key for the choice is a double whose low 9 mantissa bits are replaced by
// the expert's index (E <= 512), so that keys are distinct, a tie falls to
// the lowest index and one v_max_f64 / v_min_f64 pair moves value and index
// together.  A 32-bit logit keeps all its bits; a 64-bit v keeps 43.
//
// Bound by instructions where E is large: 65536 x 256 logits with bias and
// groups take 55 us (14 at the rate of a copy), of which the vector units work
// 73% of route_kernel's 45 and 46% of the place kernel's 10.  By latency where
// it is small: 16384 x 64 take 10 us, the units working 42% and 33% of two
// kernels of 5.5 and 4.6; one token 4.8, where filling 64 floats takes 3.9.
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

constexpr int ROUTE_MAX_EXPERTS = 512;
constexpr int ROUTE_MAX_GROUPS = 32;
constexpr int ROUTE_MAX_BLOCKS = 256;           // one to a compute unit; each sums the counts of all
constexpr int ROUTE_TOKENS = 64;                // a workgroup's tokens are a multiple

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

// Larger and smaller of two values of which neither is NaN.  fmax and fmin
// quiet a possible signalling NaN with an instruction of its own for every
// operand that comes from a lane exchange or from bit operations, which the
// sorting below mostly consists of.
__device__ __forceinline__ double larger(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double smaller(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Over the L = 8 or 16 lanes that share a token.
template <int L, typename F, typename T>
__device__ __forceinline__ T row_reduce(T v, F f) {
  v = f(v, dpp<DPP_XOR1>(v));
  v = f(v, dpp<DPP_XOR2>(v));
  v = f(v, dpp<DPP_HALF_MIRROR>(v));
  return L == 8 ? v : f(v, dpp<DPP_MIRROR>(v));
}
template <int L, typename T>
__device__ __forceinline__ T row_sum(T v) {
  return row_reduce<L>(v, [](T a, T b) { return a + b; });
}
// Largest of numbers (no NaN).
template <int L, typename T>
__device__ __forceinline__ T row_max(T v) {
  return row_reduce<L>(v, [](T a, T b) { return larger(a, b); });
}

// Key of value v with index i: NaN below every number, infinities beyond
// every finite value, -0 as 0.  A negative value holds the index itself, a
// positive one its 9-bit complement, so that the lower index is the larger key.
__device__ __forceinline__ double make_key(double v, int i) {
  v = v != v ? -1.7e308 : fmin(fmax(v + 0.0, -1.6e308), 1.6e308);
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t neg = (uint32_t)((int32_t)(b >> 32) >> 31);
  const uint32_t low = ((uint32_t)b & ~511u) | ((511u - (uint32_t)i) ^ (neg & 511u));
  return __longlong_as_double((long long)((b & 0xFFFFFFFF00000000ull) | low));
}
// The same for a 32-bit value below +inf that is not NaN nor -0: a double
// made from it has its low 29 bits free.
__device__ __forceinline__ double make_key32(float v, int i) {
  const uint64_t b = (uint64_t)__double_as_longlong((double)v);
  const uint32_t neg = (uint32_t)((int32_t)(b >> 32) >> 31);
  const uint32_t low = (uint32_t)b | ((511u - (uint32_t)i) ^ (neg & 511u));
  return __longlong_as_double(
      (long long)((b & 0xFFFFFFFF00000000ull) | (v == -__builtin_inff() ? 0u : low)));
}
__device__ __forceinline__ int key_index(double k) {
  const uint64_t b = (uint64_t)__double_as_longlong(k);
  const int low = (int)(b & 511);
  return (b >> 63) ? low : 511 - low;
}
__device__ __forceinline__ double key_value(double k) {
  return __longlong_as_double((long long)((uint64_t)__double_as_longlong(k) & ~(uint64_t)511));
}

// Experts e0 .. e0 + 3 of a row; -inf past it.
template <typename IN>
__device__ __forceinline__ void load_chunk(const IN* __restrict__ row, int E, int e0, float x[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) x[i] = -__builtin_inff();
  if (e0 + 4 <= E) {
    load4(row + e0, x);
  } else if (e0 < E) {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (e0 + i < E) x[i] = load1(row + e0 + i);
  }
}

// Chunk c of a token's row held by lane l: experts (L c + l) * 4 .. + 3.
template <typename IN, int L, int C>
__device__ __forceinline__ void load_row(const IN* __restrict__ row, int E, int l, bool live,
                                         float x[C][4]) {
#pragma unroll
  for (int c = 0; c < C; c++) {
    if (live) {
      load_chunk(row, E, (c * L + l) * 4, x[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) x[c][i] = -__builtin_inff();
    }
  }
}

// exp(x - m) where m is the row's largest number; a row whose largest is
// +inf shares its weight among the infinite logits.
__device__ __forceinline__ float exp_diff(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// 2^(n + f) for whole n and |f| <= 1/2 to 2^-46.7 of its value (2^-1074 where
// that is more), three bits more than a key keeps: the Taylor series of
// e^(f ln 2) to the 11th power, whose remainder (ln 2 / 2)^12 / 12! = 2^-47.2
// weighs 2^-46.7 where the value is sqrt(1/2).  A third of the library
// function's instructions; all of the choice's 64-bit work.
__device__ __forceinline__ double pow2_64(double n, double f) {
  constexpr double L = 0.693147180559945309417;
  constexpr double c2 = L * L / 2, c3 = c2 * L / 3, c4 = c3 * L / 4, c5 = c4 * L / 5, c6 = c5 * L / 6,
                   c7 = c6 * L / 7, c8 = c7 * L / 8, c9 = c8 * L / 9, c10 = c9 * L / 10,
                   c11 = c10 * L / 11;
  double s = fma(c11, f, c10);
  s = fma(s, f, c9);
  s = fma(s, f, c8);
  s = fma(s, f, c7);
  s = fma(s, f, c6);
  s = fma(s, f, c5);
  s = fma(s, f, c4);
  s = fma(s, f, c3);
  s = fma(s, f, c2);
  s = fma(s, f, L);
  s = fma(s, f, 1.0);
  return ldexp(s, (int)n);
}
// e^x for x <= 0; 0 below 2^-1075.  NaN stays NaN.  The rounding of log2(e)
// adds |x| 2^-54 of the value: 2^-44.5 at the end of the normal numbers.
__device__ __forceinline__ double exp_64(double x) {
  constexpr double LOG2E = 1.44269504088896340736;
  x = x != x ? x : fmax(x, -800.0);
  const double n = rint(x * LOG2E);
  return pow2_64(n, fma(x, LOG2E, -n));
}
// 1 / d for 1 <= d <= 512: the hardware's estimate (at least 2^-20) after two
// Newton steps, each of which squares the error.
__device__ __forceinline__ double rcp_64(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(fma(-d, r, 1.0), r, r);
  return fma(fma(-d, r, 1.0), r, r);
}
// 1 / (1 + e^-x), by e^-|x| so that small scores keep their bits and
// nothing saturates.
__device__ __forceinline__ double sigmoid_64(double x) {
  const double e = exp_64(-fabs(x)), r = rcp_64(1.0 + e);
  return x < 0.0 ? e * r : r;
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, n_groups, top_groups, group_max, groups_pow2, softmax, renorm;
  float scale;
  float* weights;
  int32_t* experts;
  int64_t* offsets;
  int32_t* slots;
  uint32_t* hist;        // [blocks][(E + 1) / 2] counts of every workgroup's tokens, two a word
  int tokens_per_block;
  int blocks;
};

// Compare-exchange: the larger key first.
__device__ __forceinline__ void order(double& a, double& b) {
  const double hi = larger(a, b);
  b = smaller(a, b);
  a = hi;
}

// A lane's N keys in falling order after every half is: a bitonic sequence
// (first half falling, second rising) in log2(N) steps.
template <int N>
__device__ __forceinline__ void bitonic(double* v) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1)
#pragma unroll
    for (int j = 0; j < N; j++)
      if (!(j & d)) order(v[j], v[j + d]);
}

// Two falling lists a, b of n keys into a: all 2 n of them while they fit KC,
// otherwise the n largest (the larger of a[j] and b[n - 1 - j], a bitonic
// sequence).
template <int KC, int N>
__device__ __forceinline__ void merge(double* a, const double* b) {
  if constexpr (2 * N <= KC) {
#pragma unroll
    for (int j = 0; j < N; j++) a[N + j] = b[N - 1 - j];
    bitonic<2 * N>(a);
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) a[j] = larger(a[j], b[N - 1 - j]);
    bitonic<N>(a);
  }
}

template <int KC, int N, int CTRL>
__device__ __forceinline__ void merge_lanes(double* a) {
  double o[N];
#pragma unroll
  for (int j = 0; j < N; j++) o[j] = dpp<CTRL>(a[j]);
  merge<KC, N>(a, o);
}

constexpr int grown(int n, int kc) { return 2 * n <= kc ? 2 * n : n; }

__device__ __forceinline__ void sort4(double v[4]) {
  order(v[0], v[1]);
  order(v[2], v[3]);
  order(v[0], v[2]);
  order(v[1], v[3]);
  order(v[1], v[2]);
}

// Descending list of the KC largest keys of the L lanes, in every lane, from
// the lanes' sorted chunks: chunks are merged in a lane, then lanes.
template <int L, int C, int KC>
__device__ __forceinline__ void top_keys(const double key[C][4], double top[KC]) {
  double half[C > 4 ? 2 : 1][KC];
  constexpr int N1 = C >= 2 ? grown(4, KC) : 4;      // after pairs of chunks
  constexpr int N2 = C >= 4 ? grown(N1, KC) : N1;    // after fours
#pragma unroll
  for (int h = 0; h < (C > 4 ? 2 : 1); h++) {
    double pair[2][KC];
#pragma unroll
    for (int p = 0; p < (C >= 4 ? 2 : 1); p++) {
      const int c = 4 * h + 2 * p;
#pragma unroll
      for (int i = 0; i < 4; i++) pair[p][i] = key[c][i];
      if constexpr (C >= 2) merge<KC, 4>(pair[p], key[c + 1]);
    }
#pragma unroll
    for (int j = 0; j < N1; j++) half[h][j] = pair[0][j];
    if constexpr (C >= 4) merge<KC, N1>(half[h], pair[1]);
  }
  constexpr int N3 = C > 4 ? grown(N2, KC) : N2;
#pragma unroll
  for (int j = 0; j < N2; j++) top[j] = half[0][j];
  if constexpr (C > 4) merge<KC, N2>(top, half[1]);
  constexpr int N4 = grown(N3, KC), N5 = grown(N4, KC), N6 = grown(N5, KC), N7 = grown(N6, KC);
  static_assert((L == 16 ? N7 : N6) == KC, "L lanes of four keys fill the list");
  merge_lanes<KC, N3, DPP_XOR1>(top);
  merge_lanes<KC, N4, DPP_XOR2>(top);
  merge_lanes<KC, N5, DPP_HALF_MIRROR>(top);
  if constexpr (L == 16) merge_lanes<KC, N6, DPP_MIRROR>(top);
}

// Best two of two falling pairs.
__device__ __forceinline__ void top2(double& a1, double& a2, double b1, double b2) {
  a2 = larger(smaller(a1, b1), larger(a2, b2));
  a1 = larger(a1, b1);
}
__device__ __forceinline__ void top2(float& a1, float& a2, float b1, float b2) {
  a2 = larger(__builtin_amdgcn_fmed3f(a1, b1, a2), b2);   // a1 >= a2: the median is min(a1, b1) or a2
  a1 = larger(a1, b1);
}
template <int CTRL, typename T>
__device__ __forceinline__ void top2_lanes(T& a1, T& a2) {
  top2(a1, a2, dpp<CTRL>(a1), dpp<CTRL>(a2));
}

// A group's value from its best two 32-bit choice values b1 >= b2 (logits
// where there is no bias: scored here, softmax up to a factor that the row's
// groups share); -inf with no unmasked expert.
template <bool SCORED>
__device__ __forceinline__ float group_value(const RouteArgs& a, float b1, float b2, float m) {
  constexpr float LOG2E = 1.44269504088896340736f;
  if (a.group_max) return b1;
  float v = b1, w = b2;
  if (!SCORED) {
    if (a.softmax) {
      v = __builtin_amdgcn_exp2f((b1 - m) * LOG2E);
      w = __builtin_amdgcn_exp2f((b2 - m) * LOG2E);
    } else {
      v = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(b1 * -LOG2E));
      w = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(b2 * -LOG2E));
    }
  }
  return b1 == -__builtin_inff() ? b1 : v + (b2 == -__builtin_inff() ? 0.0f : w);
}

// What the 32-bit choice of groups has to tell: how far the last chosen group
// lies above the first left out, and whether more were taken than asked for
// (equal values).
struct GroupChoice {
  float gap;
  bool equal;
};

// Masks (-inf) the values of all but the top_groups best groups, where a group
// is a power of two of chunks: the lanes of a group are neighbours in a row,
// and log2 of their number of exchanges gives all groups' best two at once.
template <int L, int C, bool SCORED>
__device__ __forceinline__ GroupChoice keep_groups_pow2(const RouteArgs& a, float v[C][4], float m, int l) {
  constexpr float NEG = -__builtin_inff();
  const int chunks = a.E / a.n_groups / 4;           // a group's chunks
  float b1[C], b2[C];
#pragma unroll
  for (int c = 0; c < C; c++) {
    b1[c] = larger(v[c][0], v[c][1]);
    b2[c] = -larger(-v[c][0], -v[c][1]);
#pragma unroll
    for (int i = 2; i < 4; i++) {
      b2[c] = __builtin_amdgcn_fmed3f(b1[c], b2[c], v[c][i]);
      b1[c] = larger(b1[c], v[c][i]);
    }
    if (chunks > 1) top2_lanes<DPP_XOR1>(b1[c], b2[c]);
    if (chunks > 2) top2_lanes<DPP_XOR2>(b1[c], b2[c]);
    if (chunks > 4) top2_lanes<DPP_HALF_MIRROR>(b1[c], b2[c]);
    if (L == 16 && chunks > 8) top2_lanes<DPP_MIRROR>(b1[c], b2[c]);
  }
  if (chunks > L) {                        // a group of several rows of chunks
    const int per = chunks / L;
#pragma unroll
    for (int c = 1; c < C; c++)
      if (c & (per - 1)) top2(b1[c], b2[c], b1[c - 1], b2[c - 1]);
#pragma unroll
    for (int c = C - 2; c >= 0; c--)
      if ((c + 1) & (per - 1)) b1[c] = b1[c + 1], b2[c] = b2[c + 1];
  }
  float g[C];
  bool kept[C];
#pragma unroll
  for (int c = 0; c < C; c++) {
    g[c] = group_value<SCORED>(a, b1[c], b2[c], m);
    kept[c] = false;
  }
  float last = 0.0f, best = 0.0f;
  for (int j = 0;; j++) {
    last = best;
    best = g[0];
#pragma unroll
    for (int c = 1; c < C; c++) best = larger(best, g[c]);
    best = row_max<L>(best);
    if (j == a.top_groups) break;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const bool hit = g[c] == best && best != NEG;
      kept[c] |= hit;
      g[c] = hit ? NEG : g[c];
    }
  }
  int n = 0;
#pragma unroll
  for (int c = 0; c < C; c++) {
    n += kept[c];
#pragma unroll
    for (int i = 0; i < 4; i++) v[c][i] = kept[c] ? v[c][i] : NEG;
  }
  GroupChoice r;
  r.gap = last - best;
  r.equal = row_sum<L>(n) > a.top_groups * chunks;
  return r;
}

// The same for groups of any size, one after the other; lane l holds the
// values of groups l, l + L, ...
template <int L, int C, bool SCORED>
__device__ __forceinline__ GroupChoice keep_groups(const RouteArgs& a, float v[C][4], float m, int l) {
  constexpr float NEG = -__builtin_inff();
  constexpr int R = ROUTE_MAX_GROUPS / L;
  const int gs = a.E / a.n_groups;
  float g[R];
#pragma unroll
  for (int r = 0; r < R; r++) g[r] = NEG;
  for (int q = 0; q < a.n_groups; q++) {
    float b1 = NEG, b2 = NEG;
    const int lo = q * gs - 4 * l;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float w = (unsigned)(c * L * 4 + i - lo) < (unsigned)gs ? v[c][i] : NEG;
        b2 = __builtin_amdgcn_fmed3f(b1, b2, w);
        b1 = larger(b1, w);
      }
    top2_lanes<DPP_XOR1>(b1, b2);
    top2_lanes<DPP_XOR2>(b1, b2);
    top2_lanes<DPP_HALF_MIRROR>(b1, b2);
    if (L == 16) top2_lanes<DPP_MIRROR>(b1, b2);
    const float value = group_value<SCORED>(a, b1, b2, m);
#pragma unroll
    for (int r = 0; r < R; r++) g[r] = q == r * L + l ? value : g[r];
  }
  const int row0 = (int)(threadIdx.x & 63) & ~(L - 1);
  uint32_t mask = 0;
  float last = 0.0f, best = 0.0f;
  for (int j = 0;; j++) {
    last = best;
    best = g[0];
#pragma unroll
    for (int r = 1; r < R; r++) best = larger(best, g[r]);
    best = row_max<L>(best);
    if (j == a.top_groups) break;
#pragma unroll
    for (int r = 0; r < R; r++) {
      const bool hit = g[r] == best && best != NEG;
      mask |= (uint32_t)(__ballot(hit) >> row0 & ((1u << L) - 1)) << (r * L);
      g[r] = hit ? NEG : g[r];
    }
  }
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int q = ((c * L + l) * 4 + i) / gs;
      v[c][i] = q < a.n_groups && (mask >> q & 1) ? v[c][i] : NEG;
    }
  GroupChoice r;
  r.gap = last - best;
  r.equal = __popc(mask) > a.top_groups;
  return r;
}

// The 32-bit choice values of a lane's logits: the logits themselves, or with
// a bias scores and bias, whose scores err bounds the error of:
//   sigmoid: exp2 and reciprocal are off by one step each; the argument's
//     rounding and log2(e)'s (0.22 half steps) weigh s (1 - s) |x| < 0.23 of
//     1.22 half steps, 1 + e half a step: under 2^-22 for s <= 1; doubled.
//   softmax: an exponential is off by 2.2 |x - m| half steps (difference,
//     product, log2(e)) and a step of its own.  For a score p <= 1 / sum, where
//     p |x - m| <= 1 / (e sum), that and the reciprocal's step make under 5 half
//     steps of 1 / sum.  The sum is off by the exponentials' mean, where
//     |x - m| averages at most ln E: under 16 half steps; and by at most 4 C +
//     4 = 36 additions.  Under 64 half steps of 1 / sum, 2^-18 / sum; doubled.
// The scores of a group's best two logits (group_value): as these, with a sum
// of 1.
template <int L, int C, bool SCORED>
__device__ __forceinline__ void choice_values(const RouteArgs& a, const float x[C][4], float m, int l,
                                              float v[C][4], float& err) {
  constexpr float NEG = -__builtin_inff();
  constexpr float LOG2E = 1.44269504088896340736f;
  if (!SCORED) {
    err = 0x1p-21f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[c][i] = x[c][i] + 0.0f;
    return;
  }
  float b[C][4], inv = 1.0f;
  load_row<float, L, C>(a.bias, a.E, l, true, b);
  if (a.softmax) {
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[c][i] = __builtin_amdgcn_exp2f((x[c][i] - m) * LOG2E);
        sum += v[c][i];
      }
    inv = __builtin_amdgcn_rcpf(row_sum<L>(sum));
    err = 0x1p-17f * inv;
  } else {
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        v[c][i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[c][i] * -LOG2E));
    err = 0x1p-21f;
  }
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) v[c][i] = x[c][i] == NEG ? NEG : fmaf(v[c][i], inv, b[c][i]);
}

// What the lanes know of a token once its experts are chosen.
struct Choice {
  double mine;     // lane l's chosen key, -inf for none
  float m, sum;    // softmax: the row's largest logit and, where weights need it, its sum
  bool nan;        // softmax: the row holds a NaN
  bool again;      // the 32-bit values do not tell: choose from 64 bits
};

// The choice of one token from 32-bit values.
// bias_max: the bias' largest magnitude, -inf aside; +inf with a NaN or +inf.
template <typename IN, int L, int C, int KC, bool SCORED>
__device__ __forceinline__ Choice choose(const RouteArgs& a, int64_t t, bool live, int l,
                                         float bias_max) {
  Choice r;
  float x[C][4];
  load_row<IN, L, C>((const IN*)a.logits + t * a.E, a.E, l, live, x);
  r.m = r.sum = 0.0f;
  r.nan = false;
  int odd = 0;                       // NaN and +inf take the 64-bit keys
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) odd |= !(x[c][i] <= 3.402823466e38f);
  r.again = odd || (SCORED && !(bias_max < 1e30f));
  if (a.softmax) {
    r.m = -__builtin_inff();
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) r.m = fmaxf(r.m, x[c][i]);   // passes over NaN
    r.m = row_max<L>(r.m);
    if (!a.renorm) {
      float m = r.m;                 // kept here: the compiler would run the exponentials for every row
      asm volatile("" : "+v"(m));
#pragma unroll
      for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) r.sum += exp_diff(x[c][i], m);
      r.sum = row_sum<L>(r.sum);
    }
  }

  double key[C][4], top[KC];
  float v[C][4], err;
  choice_values<L, C, SCORED>(a, x, r.m, l, v, err);
  const float near = 2.0f * (err + (1.0f + bias_max) * 0x1p-23f);  // twice the error of a value
  if (a.n_groups > 1) {
    const GroupChoice g = a.groups_pow2 ? keep_groups_pow2<L, C, SCORED>(a, v, r.m, l)
                                        : keep_groups<L, C, SCORED>(a, v, r.m, l);
    // sums of two values; the logits of single experts are exact
    r.again |= g.equal || g.gap <= (!a.group_max ? 2.0f * near : SCORED ? near : 0.0f);
  }
#pragma unroll
  for (int c = 0; c < C; c++) {
#pragma unroll
    for (int i = 0; i < 4; i++) key[c][i] = make_key32(v[c][i], (c * L + l) * 4 + i);
    sort4(key[c]);
  }
  top_keys<L, C, KC>(key, top);
  if (SCORED) {
    // chosen next to chosen, and the last of them next to the rest
    double last = top[0];
#pragma unroll
    for (int j = 1; j < KC; j++) {
      r.again |= j < a.k && top[j] != MX_NEG_INF && top[j - 1] - top[j] <= (double)near;
      last = j < a.k ? top[j] : last;
    }
    const double edge = last - (double)near;
    int at = 0;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) at += key[c][i] >= edge;
    r.again |= last != MX_NEG_INF && row_sum<L>(at) != a.k;
  }
  r.mine = top[0];
#pragma unroll
  for (int j = 1; j < KC; j++) r.mine = l == j ? top[j] : r.mine;
  r.mine = l < KC ? r.mine : MX_NEG_INF;
  return r;
}

// Over all 64 lanes.
template <typename F, typename T>
__device__ __forceinline__ T wave_reduce(T v, F f) {
  v = row_reduce<16>(v, f);
  v = f(v, __shfl_xor(v, 16, 64));
  return f(v, __shfl_xor(v, 32, 64));
}
template <typename T>
__device__ __forceinline__ T wave_max(T v) {
  return wave_reduce(v, [](T a, T b) { return larger(a, b); });
}

// The choice of one token by a whole wave from 64 bits, for the rows whose
// 32-bit values do not tell: equal values fall to the lowest index, NaN below
// every number.  It is seldom taken, but a workgroup waits for its last wave:
// 64 lanes hold the row in two chunks each, so that no step repeats.  Every
// lane gets the list.
template <typename IN, int KC, bool SCORED>
__device__ __forceinline__ void choose_exact(const RouteArgs& a, int64_t t, double top[KC], Choice& r) {
  constexpr int L = 64, C = ROUTE_MAX_EXPERTS / (4 * L);
  constexpr float NEG = -__builtin_inff();
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));            // nothing of this is kept for the tokens that do not need it
  const IN* row = (const IN*)a.logits + t * a.E;
  float x[C][4];
  load_row<IN, L, C>(row, a.E, l, true, x);
  float m = NEG;
  int nan = 0;
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      m = fmaxf(m, x[c][i]);             // passes over NaN
      nan |= x[c][i] != x[c][i];
    }
  r.m = m = wave_max(m);
  r.nan = a.softmax && __any(nan);
  r.sum = 0.0f;

  // keys: logits without a bias, otherwise scores (softmax: z = exp(x - m),
  // 1 for a logit at the largest, infinite ones among them, over their sum)
  // and bias
  double key[C][4], inv = 1.0;
  if (a.softmax) {
    double part = 0.0;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const double z = x[c][i] == m ? 1.0 : exp_64((double)x[c][i] - (double)m);
        key[c][i] = z;
        part += z == z && x[c][i] != NEG ? z : 0.0;
      }
    part = wave_reduce(part, [](double p, double q) { return p + q; });
    r.sum = (float)part;
    inv = rcp_64(fmax(part, 1.0));
  } else if (SCORED) {
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) key[c][i] = sigmoid_64((double)x[c][i]);
  }
  float b[C][4];
  if (SCORED) load_row<float, L, C>(a.bias, a.E, l, true, b);
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const double v = SCORED ? key[c][i] * inv + (double)b[c][i] : (double)x[c][i];
      key[c][i] = x[c][i] == NEG || v == MX_NEG_INF ? MX_NEG_INF : make_key(v, (c * L + l) * 4 + i);
    }

  if (a.n_groups > 1) {
    const int gs = a.E / a.n_groups;
    const double top_logit = fmin((double)m, 1.5e308);   // a key holds a +inf logit as 1.6e308
    double gk = MX_NEG_INF;              // lane q: the key of group q
    for (int q = 0; q < a.n_groups; q++) {
      double b1 = MX_NEG_INF, b2 = MX_NEG_INF;
#pragma unroll
      for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          top2(b1, b2, (unsigned)((c * L + l) * 4 + i - q * gs) < (unsigned)gs ? key[c][i] : MX_NEG_INF,
               MX_NEG_INF);
      top2_lanes<DPP_XOR1>(b1, b2);
      top2_lanes<DPP_XOR2>(b1, b2);
      top2_lanes<DPP_HALF_MIRROR>(b1, b2);
      top2_lanes<DPP_MIRROR>(b1, b2);
      top2(b1, b2, __shfl_xor(b1, 16, 64), __shfl_xor(b2, 16, 64));
      top2(b1, b2, __shfl_xor(b1, 32, 64), __shfl_xor(b2, 32, 64));
      double v = key_value(b1), w = key_value(b2);
      if (!a.group_max) {
        const bool two = b2 != MX_NEG_INF;
        const bool bad = b1 < -1.65e308 || (two && b2 < -1.65e308);   // NaN
        if (!SCORED) {                                 // logits: score them
          if (a.softmax) {
            v = v >= top_logit ? 1.0 : exp_64(v - m);
            w = w >= top_logit ? 1.0 : exp_64(w - m);
          } else {
            v = sigmoid_64(v);
            w = sigmoid_64(w);
          }
        }
        v = bad ? -1.7e308 : v + (two ? w : 0.0);
      }
      if (l == q && b1 != MX_NEG_INF) gk = make_key(v, q);
    }
    uint32_t keep = 0;
    for (int j = 0; j < a.top_groups; j++) {
      const double best = wave_max(gk);
      if (best != MX_NEG_INF) keep |= 1u << key_index(best);
      if (gk == best) gk = MX_NEG_INF;
    }
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int q = ((c * L + l) * 4 + i) / gs;
        if (q >= a.n_groups || !(keep >> q & 1)) key[c][i] = MX_NEG_INF;
      }
  }

#pragma unroll
  for (int c = 0; c < C; c++) sort4(key[c]);
  top_keys<16, C, KC>(key, top);         // of each row of 16 lanes
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    double o[KC];
#pragma unroll
    for (int j = 0; j < KC; j++) o[j] = __shfl_xor(top[j], d, 64);
    merge<KC, KC>(top, o);
  }
}

// One token of L lanes: its experts and weights; returns lane l's choice
// (-1: none, or l >= k).
template <typename IN, int L, int C, int KC, bool SCORED>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t, bool live, int l,
                                           float bias_max) {
  Choice r = choose<IN, L, C, KC, SCORED>(a, t, live, l, bias_max);
  for (uint64_t todo = __ballot(live && r.again); todo != 0;) {
    const int first = __ffsll((unsigned long long)todo) - 1, g = first / L;
    todo &= ~(((1ull << L) - 1) << (g * L));
    double top[KC];
    Choice q;
    choose_exact<IN, KC, SCORED>(a, __shfl(t, first, 64), top, q);
    if ((int)(threadIdx.x & 63) / L == g) {
      r.m = q.m, r.sum = q.sum, r.nan = q.nan;
      r.mine = MX_NEG_INF;
#pragma unroll
      for (int j = 0; j < KC; j++) r.mine = l == j ? top[j] : r.mine;
    }
  }
  const bool has = live && l < a.k && r.mine != MX_NEG_INF;
  const int e = has ? key_index(r.mine) : -1;

  // the chosen scores; renormalised ones as ratios of terms that share a
  // factor, so that they hold where every chosen score underflows
  const float xe = has ? load1((const IN*)a.logits + t * a.E + e) : -__builtin_inff();
  float w;
  if (a.renorm) {
    const float big = row_reduce<L>(xe, [](float p, float q) { return fmaxf(p, q); });  // NaN aside
    float u;
    if (a.softmax) {
      u = exp_diff(xe, big);
    } else {
      const float s = fminf(big, 0.0f);      // sigmoid(x) exp(-s) = 1 / (exp(s) + exp(s - x))
      u = xe == -__builtin_inff() ? 0.0f : 1.0f / (expf(s) + expf(s - xe));
    }
    if (!has) u = 0.0f;
    w = u / row_sum<L>(u);
  } else {
    w = a.softmax ? exp_diff(xe, r.m) / r.sum : 1.0f / (1.0f + expf(-xe));
  }
  if (r.nan) w = __builtin_nanf("");
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
template <int THREADS>
__device__ __forceinline__ void place_pairs(const int32_t* experts,
                                            int32_t* slots, int64_t p0, int64_t p1,
                                            int E, int* base, int* wave_cnt) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int NW = THREADS / 64;
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  for (int64_t q = p0; q < p1; q += THREADS) {
    const int64_t p = q + threadIdx.x;
    const bool one = p1 - q <= 64;               // the first wave's alone: no counts to share
    if (one && wave > 0) return;
    if (!one) {
      for (int i = threadIdx.x; i < NW * E; i += THREADS) wave_cnt[i] = 0;
      __syncthreads();
    }
    const int e = p < p1 ? experts[p] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < nbits; b++) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (one) {
      if (p < p1) slots[p] = e >= 0 ? base[e] + rank : -1;
      return;
    }
    if (e >= 0 && rank == 0) wave_cnt[wave * E + e] = __popcll(same);
    __syncthreads();
    for (int x = threadIdx.x; x < E; x += THREADS) {
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
template <typename IN, int L, int C, int KC, bool SCORED, int THREADS>
__global__ void __launch_bounds__(THREADS) route_kernel(RouteArgs a) {
  __shared__ int cnt[ROUTE_MAX_EXPERTS + 1];
  __shared__ int wave_cnt[THREADS / 64 * ROUTE_MAX_EXPERTS];
  const int l = threadIdx.x & (L - 1);
  for (int e = threadIdx.x; e < a.E; e += THREADS) cnt[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  float bias_max = 0.0f;
  if (SCORED) {
    int odd = 0;
    for (int e = l; e < a.E; e += L) {
      const float b = a.bias[e];
      odd |= !(b <= 3.402823466e38f);            // NaN or +inf
      bias_max = fmaxf(bias_max, b == -__builtin_inff() ? 0.0f : fabsf(b));
    }
    bias_max = __any(odd) ? __builtin_inff() : row_max<L>(bias_max);
  }
  for (int64_t b = t0 + threadIdx.x / 64 * (64 / L); b < t1; b += THREADS / L) {
    const int64_t t = b + (threadIdx.x & 63) / L;
    // what follows from the lane alone (bounds, indices and groups of 4 C
    // experts) would otherwise be kept across the loop, in more registers
    // than there are
    int lane = l;
    asm volatile("" : "+v"(lane));
    const int e = route_token<IN, L, C, KC, SCORED>(a, t < t1 ? t : t1 - 1, t < t1, lane, bias_max);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (a.blocks > 1) {
    // an expert's count is at most the workgroup's tokens: 16 bits
    const int words = (a.E + 1) / 2;
    for (int i = threadIdx.x; i < words; i += THREADS)
      a.hist[(int64_t)blockIdx.x * words + i] =
          (uint32_t)cnt[2 * i] | (2 * i + 1 < a.E ? (uint32_t)cnt[2 * i + 1] << 16 : 0u);
    return;
  }
  scan_experts(cnt, a.E);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += THREADS) a.offsets[e] = cnt[e];
  if (t1 * a.k > 64) __syncthreads();            // place_pairs moves the counts on
  place_pairs<THREADS>(a.experts, a.slots, 0, t1 * a.k, a.E, cnt, wave_cnt);
}

// The expert order of workgroup b's choices: its base row per expert is the
// expert's offset plus the counts of the workgroups before b.
constexpr int PLACE_THREADS = 1024;
__global__ void __launch_bounds__(PLACE_THREADS) route_place_kernel(RouteArgs a) {
  __shared__ int tot[ROUTE_MAX_EXPERTS + 1];
  __shared__ int base[ROUTE_MAX_EXPERTS];
  __shared__ int wave_cnt[PLACE_THREADS / 64 * ROUTE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.E; e += PLACE_THREADS) tot[e] = base[e] = 0;
  __syncthreads();
  const int b = blockIdx.x;
  // thread = (segment of the workgroups, two experts)
  const int words = (a.E + 1) / 2;               // <= 256: four to 16 segments
  const int segs = PLACE_THREADS / words < 16 ? PLACE_THREADS / words : 16;
  const int seg = (int)threadIdx.x / words, i = (int)threadIdx.x - seg * words;
  if (seg < segs) {
    int all0 = 0, all1 = 0, before0 = 0, before1 = 0;
    constexpr int BATCH = 16;                    // loads in flight: the counts come from other XCDs' L2
    for (int w0 = seg; w0 < a.blocks; w0 += BATCH * segs) {
      uint32_t n[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; u++) {
        const int w = w0 + u * segs;
        n[u] = w < a.blocks ? a.hist[(int64_t)w * words + i] : 0;
      }
#pragma unroll
      for (int u = 0; u < BATCH; u++) {
        const int n0 = (int)(n[u] & 0xFFFF), n1 = (int)(n[u] >> 16);
        all0 += n0, all1 += n1;
        before0 += w0 + u * segs < b ? n0 : 0, before1 += w0 + u * segs < b ? n1 : 0;
      }
    }
    atomicAdd(&tot[2 * i], all0);
    atomicAdd(&base[2 * i], before0);
    if (2 * i + 1 < a.E) {
      atomicAdd(&tot[2 * i + 1], all1);
      atomicAdd(&base[2 * i + 1], before1);
    }
  }
  __syncthreads();
  scan_experts(tot, a.E);
  __syncthreads();
  for (int x = threadIdx.x; x < a.E; x += PLACE_THREADS) base[x] += tot[x];
  if (b == 0)
    for (int x = threadIdx.x; x <= a.E; x += PLACE_THREADS) a.offsets[x] = tot[x];
  __syncthreads();
  const int64_t t0 = (int64_t)b * a.tokens_per_block;
  const int64_t t1 = t0 + a.tokens_per_block < a.T ? t0 + a.tokens_per_block : a.T;
  place_pairs<PLACE_THREADS>(a.experts, a.slots, t0 * a.k, t1 * a.k, a.E, base, wave_cnt);
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
  int E, k, softmax, renorm;
  float scale;
};

template <typename IN, int C>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteBackwardArgs a) {
  constexpr int L = 16;
  const int l = threadIdx.x & (L - 1);
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const bool live = t < a.T;
  const int64_t tt = live ? t : a.T - 1;
  const IN* row = (const IN*)a.logits + tt * a.E;
  const bool dense = a.softmax && !a.renorm;
  int e = l < a.k ? a.experts[tt * a.k + l] : -1;
  if (e >= a.E) e = -1;
  const bool has = e >= 0;
  const float g = has ? a.dweights[tt * a.k + l] : 0.0f;
  const float xe = has ? load1(row + e) : -__builtin_inff();
  float x[C][4];
  float m = -__builtin_inff(), sum = 0.0f;
  float d = 0.0f, dot = 0.0f;                  // lane l's choice's own term; the row's common term
  if (dense) {
    load_row<IN, L, C>(row, a.E, l, true, x);
    int nan = 0;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        m = fmaxf(m, x[c][i]);
        nan |= x[c][i] != x[c][i];
      }
    m = row_max<L>(m);
    nan = row_reduce<L>(nan, [](int p, int q) { return p | q; });
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        x[c][i] = x[c][i] == -__builtin_inff() ? 0.0f : exp_diff(x[c][i], m);
        sum += x[c][i];
      }
    sum = row_sum<L>(sum);
    const float inv = sum > 0.0f || nan ? 1.0f / sum : 0.0f;   // a row of masked experts: no gradient
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) x[c][i] *= inv;
    const float p = has && xe != -__builtin_inff() ? exp_diff(xe, m) * inv : 0.0f;
    d = has ? a.scale * g * p : 0.0f;
    dot = row_sum<L>(d);
  } else if (a.renorm) {
    const float big = row_max<L>(xe);
    float u = 0.0f;
    if (has && xe != -__builtin_inff()) {
      if (a.softmax) {
        u = exp_diff(xe, big);
      } else {
        const float s = fminf(big, 0.0f);
        u = 1.0f / (expf(s) + expf(s - xe));
      }
    }
    const float S = row_sum<L>(u);
    const float aj = S == 0.0f ? 0.0f : u / S;
    const float G = row_sum<L>(g * aj);
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
  const int lane0 = (int)(threadIdx.x & 63) & ~(L - 1);
  for (int j = 0; j < a.k; j++) {
    const int ej = __shfl(e, lane0 + j, 64);
    const float dj = __shfl(d, lane0 + j, 64);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        out[c][i] += (c * L + l) * 4 + i == ej ? dj : 0.0f;
  }
  if (!live) return;
  IN* dst = (IN*)a.dlogits + t * a.E;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e0 = (c * L + l) * 4;
    if (e0 + 4 <= a.E) {
      store4(dst + e0, out[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 3; i++)
        if (e0 + i < a.E) store1(dst + e0 + i, out[c][i]);
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
  if (per > 32768) per = 32768;                  // counts of 16 bits
  *tokens_per_block = (int)per;
  *blocks = (int)((T + per - 1) / per);
}

size_t route_workspace(int64_t T, int64_t E) {
  int blocks, per;
  route_split(T, &blocks, &per);
  return blocks > 1 ? sizeof(uint32_t) * (size_t)blocks * (size_t)((E + 1) / 2) : 0;
}

// Threads by a token's logits in a lane, 4 C, which most of the registers
// hold: 1024 threads leave 128 to each, 768 170, 512 256.  Two variants of 9 to
// 16 choices (KC = 16) need more than that leaves: C = 4 with a bias spills 17
// (32768 x 256, top 12: 40.8 us), C = 8 without one 4 (32768 x 512, top 12:
// 44.9; top 8, which does not, 36.4).  Up to 16 tokens, 256.
template <typename IN, int L, int C, int KC, bool SCORED, int THREADS>
static void launch_route_threads(const RouteArgs& a, hipStream_t stream) {
  if (a.T <= 16)
    hipLaunchKernelGGL((route_kernel<IN, L, C, KC, SCORED, 256>), dim3(1), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((route_kernel<IN, L, C, KC, SCORED, THREADS>), dim3(a.blocks), dim3(THREADS), 0,
                       stream, a);
}
template <typename IN, int L, int C, int KC>
static void launch_route_lanes(bool scored, const RouteArgs& a, hipStream_t stream) {
  constexpr int SCORED_THREADS = C <= 4 ? 1024 : L == 8 ? 768 : 512;
  if (scored) launch_route_threads<IN, L, C, KC, true, SCORED_THREADS>(a, stream);
  else launch_route_threads<IN, L, C, KC, false, 1024>(a, stream);
}
// Lanes to a token: eight, where they hold its logits (32 each) and its
// choices; merging lists of lanes is most of the work, and eight lanes take
// one step less of it for twice the tokens of a wave.
template <typename IN>
static void launch_route_in(bool scored, const RouteArgs& a, hipStream_t stream) {
  if (a.k <= 8) {
    if (a.E <= 64) launch_route_lanes<IN, 8, 2, 8>(scored, a, stream);
    else if (a.E <= 128) launch_route_lanes<IN, 8, 4, 8>(scored, a, stream);
    else if (a.E <= 256) launch_route_lanes<IN, 8, 8, 8>(scored, a, stream);
    else launch_route_lanes<IN, 16, 8, 8>(scored, a, stream);
  } else {
    if (a.E <= 64) launch_route_lanes<IN, 16, 1, 16>(scored, a, stream);
    else if (a.E <= 128) launch_route_lanes<IN, 16, 2, 16>(scored, a, stream);
    else if (a.E <= 256) launch_route_lanes<IN, 16, 4, 16>(scored, a, stream);
    else launch_route_lanes<IN, 16, 8, 16>(scored, a, stream);
  }
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
  a.hist = (uint32_t*)workspace;
  const int64_t chunks = E / n_groups / 4;
  a.groups_pow2 = n_groups > 1 && E % (4 * n_groups) == 0 && (chunks & (chunks - 1)) == 0;
  route_split(T, &a.blocks, &a.tokens_per_block);
  const bool scored = bias != nullptr;
  if (f32) launch_route_in<float>(scored, a, stream);
  else launch_route_in<uint16_t>(scored, a, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 1) return e;
  hipLaunchKernelGGL(route_place_kernel, dim3(a.blocks), dim3(PLACE_THREADS), 0, stream, a);
  return hipGetLastError();
}

template <typename IN>
static void launch_route_backward_in(const RouteBackwardArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T * 16 + 255) / 256));
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
  if (f32) launch_route_backward_in<float>(a, stream);
  else launch_route_backward_in<uint16_t>(a, stream);
  return hipGetLastError();
}

}  // namespace mx
