// Products with 4-bit MX weights for gfx950 where the weight's bytes count:
// tens to hundreds of rows, or sizes that the large tiles do not take.  C = A *
// B^T as in gemm4.hip, which has the lane layouts; any N and any K that is a
// multiple of 32.
//
// Small tiles and many stages: the loads of NS - 1 K steps are in flight, so
// that a compute unit keeps some 60 KB of the weight on its way.  Where the
// result has fewer tiles than the chip has places, K is split over workgroups
// whose FP32 sums a second kernel adds in the order of the splits.  One row is
// bound by the weight's bytes: 151936 x 4096 in 65.5 us (5.05 TB/s), 18432 x
// 7168 in 15.0 (4.7 TB/s, launch and host included).
#include "gemm4.h"
#include "mx_columns.h"

namespace mx {

// A tile of 32 WM FM rows x 32 WN FN columns, WM WN waves, FM x FN accumulators
// of 32x32 each.  A K step is 128 KH elements (256 with 4-bit A).  A stage holds
// the A tile in panels of 128 bytes a row, the B tile in rows of 64 KH bytes
// (128 with 4-bit A) and the step's scale words, a dword of four scale bytes a
// row and 128 elements: A's rows, padded to whole waves, then B's.  Chunk
// swizzles and the meeting of blocks are those of gemm4.hip, panel by panel.
// TWO: stages for two workgroups on a compute unit.  Stages, with an 8-bit A and
// a 4-bit one: 3 and 3 for 32 rows, 4 and 6 for 64, 3 and 4 for 128, 4 and 3 for
// 128 x 256, 3 and 4 for 128 rows of a group.
template <int FA, int WM, int WN, int FM, int FN, int KH_, bool TWO>
struct Deep4 {
  static constexpr bool A4 = FA == ELEM_E2M1;
  static constexpr int WAVES = WM * WN;
  static constexpr int BMR = 32 * WM * FM, BNR = 32 * WN * FN;
  static constexpr int KH = A4 ? 2 : KH_;               // scale dwords of a row and step
  static constexpr int KS = 128 * KH;
  static constexpr int PANELS = A4 ? 1 : KH;            // of A
  static constexpr int BROW = 64 * KH;
  static constexpr int A_PANEL = BMR * 128;
  static constexpr int A_BYTES = PANELS * A_PANEL, B_BYTES = BNR * BROW;
  static constexpr int A_OPS = A_BYTES / 1024 / WAVES;  // 1 KB loads of a wave and step
  static constexpr int B_OPS = B_BYTES / 1024 / WAVES;
  static constexpr int OPS = A_OPS + B_OPS + KH;
  static constexpr int A_ROWS = (BMR + 63) / 64 * 64;   // A's places among the scale rows
  static_assert(A_ROWS + BNR <= 64 * WAVES, "a wave loads the scales of 64 rows");
  static_assert(A_OPS * 1024 * WAVES == A_BYTES && B_OPS * 1024 * WAVES == B_BYTES, "whole loads");
  static constexpr int S_BYTES = 256 * WAVES;           // one array of scale words
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + KH * S_BYTES;
  static constexpr int NS = (TWO ? 81920 : 163840) / STAGE_BYTES;  // 3 to 6
  static_assert(NS >= 2 && (NS - 1) * OPS < 64, "vmcnt holds 6 bits");

  const uint8_t* __restrict__ a;
  const uint8_t* __restrict__ sa;
  const uint8_t* __restrict__ b;
  const uint8_t* __restrict__ sb;
  int64_t m0, m_end, n0, N, K;
  int kt0, kt1;         // K steps of this workgroup
  int full;             // steps that lie in K wholly; at most one more follows
  lds_u8* st;
  u32x4 ra, rb, rs;
  uint32_t off_a[A_OPS], off_b[B_OPS], off_s;  // this lane's offsets at step 0
  uint32_t pos_a[A_OPS], pos_b;                // and its chunks' bytes within a step's row
  uint32_t row_a, row_b, nkb;                  // bytes of a row

  __device__ __forceinline__ void setup(int wave, int lane) {
    const int64_t mrows = m_end - m0, nrows = (N - n0) < BNR ? (N - n0) : BNR;
    row_a = (uint32_t)(A4 ? K >> 1 : K);
    row_b = (uint32_t)(K >> 1);
    nkb = (uint32_t)(K >> 5);
    full = (int)(K / KS);
    ra = make_rsrc(a + m0 * row_a, mrows * row_a);
    rb = make_rsrc(b + n0 * row_b, nrows * row_b);
    // A: load t covers rows 8 (t % (BMR / 8)) .. + 7 of panel t / (BMR / 8);
    // lane i lands in row i / 8 of them at chunk i % 8, logical (i % 8) ^ swz(row)
#pragma unroll
    for (int u = 0; u < A_OPS; u++) {
      const int t = wave + WAVES * u, row = 8 * (t % (BMR / 8)) + (lane >> 3);
      pos_a[u] = 128 * (t / (BMR / 8)) + 16 * ((lane & 7) ^ swz(row));
      off_a[u] = (uint32_t)row * row_a + pos_a[u];
    }
    constexpr int CH = BROW / 16;
#pragma unroll
    for (int u = 0; u < B_OPS; u++) {
      const int row = (wave + WAVES * u) * (64 / CH) + lane / CH;
      pos_b = 16 * ((lane % CH) ^ (CH == 8 ? swz(row) : (row >> 2) & 3));  // the same for every u
      off_b[u] = (uint32_t)row * row_b + pos_b;
    }
    // scale rows 64 wave .. 64 wave + 63
    const bool isb = 64 * wave >= A_ROWS;
    const int row = 64 * wave + lane - (isb ? A_ROWS : 0);
    const int64_t rows = isb ? nrows : mrows;
    rs = make_rsrc(isb ? sb + n0 * nkb : sa + m0 * nkb, rows * nkb);
    off_s = row < rows && 64 * wave < A_ROWS + BNR ? (uint32_t)row * nkb : OOB;
    if (nkb < 4) off_s = OOB;  // rows shorter than a dword: short_scales() loads them
  }

  // Load D (of OPS: A's, B's, the scales') of step kt into the stage at `to`.
  // WHOLE: the step lies in K and in this workgroup's part, its offset is
  // scalar.  Otherwise chunks past K read as zero, and a step past the last
  // touches no memory.
  template <bool WHOLE>
  __device__ __forceinline__ void issue_one(lds_u8* to, int kt, int d, int wave) {
    if (d < A_OPS) {
      const uint32_t ka = (uint32_t)kt * (128 * PANELS);
      lds_u8* const at = to + (wave + WAVES * d) * 1024;
      if constexpr (WHOLE) dma16_at(at, off_a[d], ra, ka);
      else dma16(at, kt < kt1 && ka + pos_a[d] < row_a ? off_a[d] + ka : OOB, ra);
    } else if (d < A_OPS + B_OPS) {
      const int u = d - A_OPS;
      const uint32_t kb = (uint32_t)kt * BROW;
      lds_u8* const at = to + A_BYTES + (wave + WAVES * u) * 1024;
      if constexpr (WHOLE) dma16_at(at, off_b[u], rb, kb);
      else dma16(at, kt < kt1 && kb + pos_b < row_b ? off_b[u] + kb : OOB, rb);
    } else {
      const int h = d - A_OPS - B_OPS;
      const uint32_t ks = (uint32_t)kt * (KS / 32) + 4 * h;
      lds_u8* const at = to + A_BYTES + B_BYTES + S_BYTES * h + 256 * wave;
      // a dword that would pass the row's last scale byte ends there instead
      // and is shifted when it is read
      if constexpr (WHOLE) dma4_at(at, off_s, rs, ks);
      else dma4(at, kt < kt1 && ks < nkb ? off_s + (ks + 4 <= nkb ? ks : nkb - 4) : OOB, rs);
    }
  }
  // Loads D0 .. D1 - 1 of step kt
  template <bool WHOLE, int D0, int D1>
  __device__ __forceinline__ void issue(lds_u8* to, int kt, int wave) {
#pragma unroll
    for (int d = D0; d < D1; d++) issue_one<WHOLE>(to, kt, d, wave);
  }

  // A row's scale words of a step: with 8-bit A word h holds byte S for half S
  // of panel h, with 4-bit A word 0 byte S + 2 h for MFMA h of half S.
  __device__ __forceinline__ static void scale(const lds_u8* stage, int row, uint32_t* w) {
    typedef const __attribute__((address_space(3))) uint32_t lds_u32;
#pragma unroll
    for (int h = 0; h < KH; h++) w[h] = *(lds_u32*)(stage + A_BYTES + B_BYTES + S_BYTES * h + 4 * row);
  }
  template <bool WHOLE>
  __device__ __forceinline__ void shape(uint32_t* w, int kt, int g) const {
    if constexpr (!WHOLE) {  // past K the payload is 0, and so may be its scales
#pragma unroll
      for (int h = 0; h < KH; h++) {
        const uint32_t at = (uint32_t)kt * (KS / 32) + 4 * h;
        if (at + 4 > nkb) w[h] = at < nkb ? w[h] >> (8 * (at + 4 - nkb)) : 0u;
      }
    }
    if (A4) {
      w[0] = __builtin_amdgcn_perm(w[KH - 1], w[0], g ? 0x07050301u : 0x06040200u);
    } else {
#pragma unroll
      for (int h = 0; h < KH; h++) w[h] >>= 16 * g;
    }
  }

  // A step's MFMAs come in UNITS of half a panel (half a step with 4-bit A).
  // While one unit is multiplied the fragments of the next are read, those of a
  // step's first unit with the last unit of the step before, and a share of a
  // later step's loads is issued.
  static constexpr int UNITS = 2 * PANELS;
  static constexpr int MFMAS = FM * FN * (A4 ? 2 : 1);  // of a unit
  struct Frags {
    v8i a[FM], b[FN];
  };
  // Fragment r of a unit: A's, then B's
  template <int U>
  __device__ __forceinline__ static void read_one(const lds_u8* cur, Frags& f, int r, int wm, int wn, int lane) {
    constexpr int h = U / 2, S = U % 2;
    const int g = lane >> 5, i = lane & 31;
    if (r < FM) {
      f.a[r] = read_frag(cur + h * A_PANEL, 32 * FM * wm + 32 * r + i, S, g);
    } else {
      const int x = r - FM, row = 32 * FN * wn + 32 * x + i;
      if (A4) {
        f.b[x] = read_frag(cur + A_BYTES, row, S, g);
      } else {
        const int c = 4 * h + 2 * g + S;
        const v4i v = *(const lds_v4i*)(cur + A_BYTES + row * BROW +
                                        ((c ^ (BROW == 128 ? swz(row) : (row >> 2) & 3)) << 4));
        f.b[x] = (v8i){v.x, v.y, v.z, v.w, 0, 0, 0, 0};
      }
    }
  }
  // MFMA m of a unit
  template <int U>
  __device__ __forceinline__ static void mma_one(const Frags& f, int m, v16f (&acc)[FN][FM],
                                                 const uint32_t (&sar)[FM][KH],
                                                 const uint32_t (&sbr)[FN][KH]) {
    constexpr int h = U / 2, S = U % 2;
    const int x = m / FM % FN, y = m % FM;
    if constexpr (A4) {
      if (m < FM * FN)
        acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            low(f.b[x]), low(f.a[y]), acc[x][y], ELEM_E2M1, ELEM_E2M1, S, (int)sbr[x][0], S, (int)sar[y][0]);
      else
        acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            high(f.b[x]), high(f.a[y]), acc[x][y], ELEM_E2M1, ELEM_E2M1, S + 2, (int)sbr[x][0], S + 2,
            (int)sar[y][0]);
    } else {
      acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          f.b[x], f.a[y], acc[x][y], ELEM_E2M1, FA, S, (int)sbr[x][h], S, (int)sar[y][h]);
    }
  }
  // Multiplies unit U out of f, reads unit V of the stage at `from` into nx and
  // issues share P of step kl's loads into the stage at `to`.  The order is
  // held: a wave issues in order, so loads in a bunch (18 cycles of the
  // compute unit each) would hold its MFMAs back; in a bunch after the barrier
  // they took as long as the MFMAs, 2050 cycles a step of a 128 x 128 tile
  // where the MFMAs need 1024.
  template <int U, int V, int P, bool WHOLE>
  __device__ __forceinline__ void unit(const Frags& f, Frags& nx, const lds_u8* from, lds_u8* to, int kl,
                                       int wave, int wm, int wn, int lane, const uint32_t (&sar)[FM][KH],
                                       const uint32_t (&sbr)[FN][KH], v16f (&acc)[FN][FM]) {
    constexpr int D0 = P * OPS / UNITS, D1 = (P + 1) * OPS / UNITS, R = FM + FN;
#pragma unroll
    for (int m = 0; m < MFMAS; m++) {
      mma_one<U>(f, m, acc, sar, sbr);
#pragma unroll
      for (int r = m * R / MFMAS; r < (m + 1) * R / MFMAS; r++) read_one<V>(from, nx, r, wm, wn, lane);
#pragma unroll
      for (int d = D0 + m * (D1 - D0) / MFMAS; d < D0 + (m + 1) * (D1 - D0) / MFMAS; d++)
        issue_one<WHOLE>(to, kl, d, wave);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ static void read_scales(const lds_u8* cur, int wm, int wn, int lane,
                                                     uint32_t (&sar)[FM][KH], uint32_t (&sbr)[FN][KH]) {
    const int i = lane & 31;
#pragma unroll
    for (int f = 0; f < FM; f++) scale(cur, 32 * FM * wm + 32 * f + i, sar[f]);
#pragma unroll
    for (int f = 0; f < FN; f++) scale(cur, A_ROWS + 32 * FN * wn + 32 * f + i, sbr[f]);
  }
  template <bool WHOLE>
  __device__ __forceinline__ void shape_scales(int kt, int lane, uint32_t (&sar)[FM][KH],
                                               uint32_t (&sbr)[FN][KH]) const {
#pragma unroll
    for (int f = 0; f < FM; f++) shape<WHOLE>(sar[f], kt, lane >> 5);
#pragma unroll
    for (int f = 0; f < FN; f++) shape<WHOLE>(sbr[f], kt, lane >> 5);
  }

  // K below 128, one step: the scale bytes of each row one by one, placed as
  // shape() expects them of the last dword of a row.
  __device__ __forceinline__ void short_scales(int wave, int lane) {
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
    const bool isb = 64 * wave >= A_ROWS;
    const int row = 64 * wave + lane - (isb ? A_ROWS : 0);
    const int64_t rows = isb ? N - n0 : m_end - m0;
    if (row < rows && row < (isb ? BNR : BMR)) {
      const uint8_t* p = isb ? sb + (n0 + row) * nkb : sa + (m0 + row) * nkb;
      uint32_t w = 0;
      for (uint32_t e = 0; e < nkb; e++) w |= (uint32_t)p[e] << (8 * (4 - nkb + e));
      *(lds_u32*)(st + A_BYTES + B_BYTES + 256 * wave + 4 * lane) = w;
    }
    __syncthreads();
  }

  // Step kt on stage `cur`, its first unit in f0 and its scales shaped; leaves
  // the same of step kt + 1.  On the way the loads of step kt - 1 + NS, into the
  // stage `old` of step kt - 1, are completed, and those of kt + NS begun.
  // WHOLE: all of these are whole steps.
  template <bool WHOLE>
  __device__ __forceinline__ void step(lds_u8* old, lds_u8* cur, const lds_u8* nxt, int kt, int wave, int wm,
                                       int wn, int lane, Frags& f0, uint32_t (&sar)[FM][KH],
                                       uint32_t (&sbr)[FN][KH], v16f (&acc)[FN][FM]) {
    Frags f1;
    const int kl = kt - 1 + NS;
    unit<0, 1, 1, WHOLE>(f0, f1, cur, old, kl, wave, wm, wn, lane, sar, sbr, acc);
    if constexpr (UNITS == 4) {
      unit<1, 2, 2, WHOLE>(f1, f0, cur, old, kl, wave, wm, wn, lane, sar, sbr, acc);
      unit<2, 3, 3, WHOLE>(f0, f1, cur, old, kl, wave, wm, wn, lane, sar, sbr, acc);
    }
    // every wave has read this stage; the next one has landed for every wave
    wait_vm<(NS - 2) * OPS>();
    __syncthreads();
    uint32_t nar[FM][KH], nbr[FN][KH];
    read_scales(nxt, wm, wn, lane, nar, nbr);
    unit<UNITS - 1, 0, 0, WHOLE>(f1, f0, nxt, cur, kl + 1, wave, wm, wn, lane, sar, sbr, acc);
    shape_scales<WHOLE>(kt + 1, lane, nar, nbr);
#pragma unroll
    for (int h = 0; h < KH; h++) {
#pragma unroll
      for (int f = 0; f < FM; f++) sar[f][h] = nar[f][h];
#pragma unroll
      for (int f = 0; f < FN; f++) sbr[f][h] = nbr[f][h];
    }
  }

  __device__ __forceinline__ void run(v16f (&acc)[FN][FM], int wave, int lane) {
    const int wm = wave % WM, wn = wave / WM;
    constexpr int FIRST = OPS / UNITS;  // loads of a step's share 0
#pragma unroll
    for (int x = 0; x < FN; x++)
#pragma unroll
      for (int y = 0; y < FM; y++) acc[x][y] = (v16f){};
    const int last = kt1 < full ? kt1 : full;  // the end of whole steps
    // NS - 1 steps and the first share of one more are on their way
#pragma unroll 1
    for (int p = 0; p < NS - 1; p++) {
      if (kt0 + p < last) issue<true, 0, OPS>(st + p * STAGE_BYTES, kt0 + p, wave);
      else issue<false, 0, OPS>(st + p * STAGE_BYTES, kt0 + p, wave);
    }
    lds_u8* old = st + (NS - 1) * STAGE_BYTES;
    if (kt0 + NS - 1 < last) issue<true, 0, FIRST>(old, kt0 + NS - 1, wave);
    else issue<false, 0, FIRST>(old, kt0 + NS - 1, wave);
    wait_vm<(NS - 2) * OPS + FIRST>();
    __syncthreads();
    if (nkb < 4) short_scales(wave, lane);
    Frags f0;
    uint32_t sar[FM][KH], sbr[FN][KH];
    read_scales(st, wm, wn, lane, sar, sbr);
#pragma unroll
    for (int r = 0; r < FM + FN; r++) read_one<0>(st, f0, r, wm, wn, lane);
    shape_scales<false>(kt0, lane, sar, sbr);
    lds_u8* cur = st;
    lds_u8* const end = st + NS * STAGE_BYTES;
    int kt = kt0;
    for (; kt < last - NS; kt++) {
      lds_u8* nxt = cur + STAGE_BYTES == end ? st : cur + STAGE_BYTES;
      step<true>(old, cur, nxt, kt, wave, wm, wn, lane, f0, sar, sbr, acc);
      old = cur;
      cur = nxt;
    }
    for (; kt < kt1; kt++) {
      lds_u8* nxt = cur + STAGE_BYTES == end ? st : cur + STAGE_BYTES;
      step<false>(old, cur, nxt, kt, wave, wm, wn, lane, f0, sar, sbr, acc);
      old = cur;
      cur = nxt;
    }
    wait_vm_all();  // no load may still be writing LDS when the workgroup ends
  }

  __device__ __forceinline__ static v8i low(v8i v) { return (v8i){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
  __device__ __forceinline__ static v8i high(v8i v) { return (v8i){v[4], v[5], v[6], v[7], 0, 0, 0, 0}; }

  // The FP32 sums of one split into its share of the workspace, whole tiles in
  // rows of ldw columns: a lane writes groups of four consecutive columns.
  __device__ __forceinline__ void store_partial(const v16f (&acc)[FN][FM], float* __restrict__ ws, int64_t ldw,
                                                int wave, int lane) const {
    const int wm = wave % WM, wn = wave / WM, g = lane >> 5, i = lane & 31;
#pragma unroll
    for (int fn = 0; fn < FN; fn++)
#pragma unroll
      for (int fm = 0; fm < FM; fm++) {
        const v16f& v = acc[fn][fm];
        const int64_t m = m0 + 32 * FM * wm + 32 * fm + i;
        if (m >= m_end) continue;
#pragma unroll
        for (int r4 = 0; r4 < 4; r4++) {
          const int64_t n = n0 + 32 * FN * wn + 32 * fn + 8 * r4 + 4 * g;
          *(v4f*)(ws + m * ldw + n) = (v4f){v[4 * r4], v[4 * r4 + 1], v[4 * r4 + 2], v[4 * r4 + 3]};
        }
      }
  }
};

// Dense: blockIdx.y is the split of K, blockIdx.x the tile, the rows of one
// part of the weight side by side.
template <int FA, int WM, int WN, int FM, int FN, int KH, bool TWO>
__global__ void __launch_bounds__(64 * WM * WN)
gemm4_deep_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                  const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb, uint16_t* __restrict__ c,
                  int64_t M, int64_t N, int64_t K, float* __restrict__ ws, int64_t ldw) {
  typedef Deep4<FA, WM, WN, FM, FN, KH, TWO> T;
  __shared__ __attribute__((aligned(16))) uint8_t stages[T::NS * T::STAGE_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t nm = (uint32_t)((M + T::BMR - 1) / T::BMR);
  // workgroups are dealt to the 8 XCDs in turn: each takes a contiguous part of
  // the tiles, so that those of one part of the weight share its L2
  const uint32_t per = gridDim.x >> 3, rem = gridDim.x & 7, x = blockIdx.x & 7;
  const uint32_t tile = x * per + (x < rem ? x : rem) + (blockIdx.x >> 3);
  const uint32_t nt = tile / nm, mt = tile - nt * nm;
  T t;
  t.a = a, t.sa = sa, t.b = b, t.sb = sb;
  t.m0 = (int64_t)mt * T::BMR;
  t.m_end = t.m0 + T::BMR < M ? t.m0 + T::BMR : M;
  t.n0 = (int64_t)nt * T::BNR;
  t.N = N, t.K = K;
  const int64_t nks = (K + T::KS - 1) / T::KS;
  t.kt0 = (int)(nks * blockIdx.y / gridDim.y);
  t.kt1 = (int)(nks * (blockIdx.y + 1) / gridDim.y);
  t.st = (lds_u8*)stages;
  t.setup(wave, lane);
  v16f acc[FN][FM];
  t.run(acc, wave, lane);
  if (gridDim.y == 1) store_bf16(acc, c, N, t.m0 + 32 * FM * (wave % WM), t.m_end, t.n0 + 32 * FN * (wave / WM), lane);
  else t.store_partial(acc, ws + (int64_t)blockIdx.y * M * ldw, ldw, wave, lane);
}

// The splits' sums, added in their order and rounded to BF16; a thread takes
// four columns.
__global__ void __launch_bounds__(256)
gemm4_join_kernel(const float* __restrict__ ws, int64_t M, int64_t N, int64_t ldw, int splits,
                  uint16_t* __restrict__ c) {
  const uint32_t n = 4 * (blockIdx.x * 256 + threadIdx.x);
  const int64_t m = blockIdx.y;
  if (n >= N) return;
  const float* p = ws + m * ldw + n;
  v4f v = *(const v4f*)p;
  for (int s = 1; s < splits; s++) v += *(const v4f*)(p + s * M * ldw);
  const uint32_t w[2] = {cvt_pk_bf16(v.x, v.y), cvt_pk_bf16(v.z, v.w)};
  uint16_t* dst = c + m * N + n;
  if (n + 4 <= N) {
    *(u32x2_at2*)dst = (u32x2_at2){w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (n + e < N) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Row tile number `slot` of BMR rows among those of all groups, counted group
// by group: its group and its rows [m0, m_end).  Offsets are clamped into [0,
// rows] and made non-decreasing, as the large tiles do: bad ones name rows of
// [0, rows) only, no row twice, and no more tiles than good ones.  False past
// the last.
template <int BMR>
__device__ __forceinline__ bool row_tile(const int64_t* __restrict__ offsets, int64_t G, int64_t rows,
                                         uint32_t slot, int lane, int64_t& g, int64_t& m0, int64_t& m_end) {
  uint32_t before = 0;
  int64_t top = 0;  // the largest offset so far
  int64_t next_lo = 0, next_hi = 0;
  if (lane < G) next_lo = offsets[lane], next_hi = offsets[lane + 1];
  for (int64_t base = 0; base < G; base += 64) {
    const bool in = base + lane < G;
    int64_t lo = next_lo, hi = next_hi;
    if (base + 64 + lane < G) next_lo = offsets[base + 64 + lane], next_hi = offsets[base + 65 + lane];
    lo = lo < 0 ? 0 : (lo > rows ? rows : lo);
    hi = hi < 0 ? 0 : (hi > rows ? rows : hi);
    if (__any(in && (lo < top || hi < lo))) {  // running maxima, where some offset is smaller
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(lo, d);
        if (lane >= d && y > lo) lo = y;
      }
      lo = lo < top ? top : lo;
      hi = hi < lo ? lo : hi;
    }
    top = readlane64(lo, 63);  // (a part that is not full is the last)
    const uint32_t n = in ? (uint32_t)((hi - lo + BMR - 1) / BMR) : 0;
    uint32_t sum = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t y = __shfl_up(sum, d);
      if (lane >= d) sum += y;
    }
    const uint32_t tile = slot - (before + sum - n);
    const uint64_t hit = __ballot(tile < n);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      g = base + l;
      const int64_t end = __shfl(hi, l);
      m0 = __shfl(lo, l) + (int64_t)__shfl(tile, l) * BMR;
      m_end = m0 + BMR < end ? m0 + BMR : end;
      return true;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
  }
  return false;
}

// Grouped: blockIdx.y is the row tile (and those gridDim.y further on),
// blockIdx.x the column tile, so that a group with most of the rows has as many
// workgroups as its tiles (1536 rows, all in one of 64 groups of 4096 x 4096: 49
// us; 354 where a workgroup took its group's tiles in turn).  128 rows over 64
// such groups: 90 us, at 4.9 TB/s the weights of the groups that have rows.
template <int FA, int WM, int WN, int FM, int FN, int KH, bool TWO>
__global__ void __launch_bounds__(64 * WM * WN)
grouped4_deep_kernel(const int64_t* __restrict__ offsets, int64_t G, int64_t rows,
                     const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                     const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                     uint16_t* __restrict__ c, int64_t N, int64_t K) {
  typedef Deep4<FA, WM, WN, FM, FN, KH, TWO> T;
  __shared__ __attribute__((aligned(16))) uint8_t stages[T::NS * T::STAGE_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  T t;
  t.a = a, t.sa = sa;
  t.n0 = (int64_t)blockIdx.x * T::BNR;
  t.N = N, t.K = K;
  t.kt0 = 0, t.kt1 = (int)((K + T::KS - 1) / T::KS);
  t.st = (lds_u8*)stages;
  for (uint32_t slot = blockIdx.y;; slot += gridDim.y) {
    int64_t g;
    if (!row_tile<T::BMR>(offsets, G, rows, slot, lane, g, t.m0, t.m_end)) break;
    t.b = b + g * N * (K >> 1), t.sb = sb + g * N * (K >> 5);
    t.setup(wave, lane);
    v16f acc[FN][FM];
    t.run(acc, wave, lane);
    store_bf16(acc, c, N, t.m0 + 32 * FM * (wave % WM), t.m_end, t.n0 + 32 * FN * (wave / WM), lane);
    __syncthreads();  // every wave is done with the stages
  }
}

// Which tile, measured at K = 7168 and 18432 with N = 18432 and 7168 (us, 8-bit
// A).  Up to 32 rows 32 x 128, two workgroups to a compute unit (1 x 18432 x
// 7168: 15.0, one to a unit 17.0); up to 64 rows 64 x 128 (64 x 18432: 22.2, two
// to a unit 26.3); above, 128 x 128 while its tiles find a unit each (512 x 7168
// x 18432: 70, against 117 with 128 x 256), 128 x 256 beyond (2048 rows: 318
// against 361).  K is split so far as workgroups still find a unit each and the
// steps saved outweigh the second launch and the partial sums' way through
// memory (1 x 7168 x 18432: 15.3 in four, 31 whole; 1 x 4096 x 4096: 8.2 to 9.8
// whole, 12.4 in four).  Sizes alone decide, as they do on the workspace's bytes, for the
// 256 units of the card; on fewer the same workgroups run in more rounds.
enum Shape4 { TILE_32, TILE_64, TILE_128, TILE_WIDE };

struct Plan4 {
  Shape4 shape;
  int64_t tiles, ldw;
  int splits;
};

static Plan4 plan_of(int64_t M, int64_t N, int64_t K) {
  const int64_t n128 = (N + 127) / 128, t128 = (M + 127) / 128 * n128;
  Plan4 p;
  p.ldw = n128 * 128;
  if (M <= 32) p.shape = TILE_32, p.tiles = n128;
  else if (M <= 64) p.shape = TILE_64, p.tiles = n128;
  else if (t128 <= 256) p.shape = TILE_128, p.tiles = t128;
  else p.shape = TILE_WIDE, p.tiles = (M + 127) / 128 * ((N + 255) / 256);
  p.splits = 1;
  if (p.shape == TILE_WIDE) return p;
  // microseconds: a step of 256 elements by the tile's height, eight for the
  // second launch, and partial sums written and read at 4 TB/s
  const double step = p.shape == TILE_32 ? 0.55 : p.shape == TILE_64 ? 0.85 : 1.1;
  const int64_t steps = (K + 255) / 256;
  double best = steps * step;
  for (int s = 2; s <= 16 && s * p.tiles <= 256 && s <= steps; s++) {
    const double us = (steps + s - 1) / s * step + 8.0 + 8e-6 / 4 * s * M * p.ldw;
    if (us < best) best = us, p.splits = s;
  }
  return p;
}

size_t gemm4_deep_workspace(int64_t M, int64_t N, int64_t K) {
  const Plan4 p = plan_of(M, N, K);
  return p.splits == 1 ? 0 : (size_t)(p.splits * M * p.ldw * 4);
}

template <int FA>
static void launch_deep(int64_t M, int64_t N, int64_t K, const uint8_t* a, const uint8_t* sa,
                        const uint8_t* b, const uint8_t* sb, uint16_t* c, float* ws, hipStream_t stream) {
  const Plan4 p = plan_of(M, N, K);
  const dim3 grid((unsigned)p.tiles, (unsigned)p.splits);
#define MX_DEEP(WM_, WN_, FM_, FN_, KH_, TWO_)                                                    \
  hipLaunchKernelGGL((gemm4_deep_kernel<FA, WM_, WN_, FM_, FN_, KH_, TWO_>), grid, dim3(64 * WM_ * WN_), 0, \
                     stream, a, sa, b, sb, c, M, N, K, ws, p.ldw)
  switch (p.shape) {
    case TILE_32: MX_DEEP(1, 4, 1, 1, 2, true); break;
    case TILE_64: MX_DEEP(2, 2, 1, 2, 2, false); break;
    case TILE_128: MX_DEEP(2, 2, 2, 2, 2, false); break;
    case TILE_WIDE: MX_DEEP(2, 4, 2, 2, 1, false); break;
  }
#undef MX_DEEP
  if (p.splits > 1)
    hipLaunchKernelGGL(gemm4_join_kernel, dim3((unsigned)((N + 1023) / 1024), (unsigned)M), dim3(256), 0, stream,
                       ws, M, N, p.ldw, p.splits, c);
}

hipError_t launch_gemm4_deep(int a_elem, int64_t M, int64_t N, int64_t K, const void* a,
                             const void* sa, const void* b, const void* sb, void* c, void* ws,
                             hipStream_t stream) {
  const uint8_t *A = (const uint8_t*)a, *SA = (const uint8_t*)sa, *B = (const uint8_t*)b,
                *SB = (const uint8_t*)sb;
  uint16_t* C = (uint16_t*)c;
  if (a_elem == ELEM_E4M3) launch_deep<ELEM_E4M3>(M, N, K, A, SA, B, SB, C, (float*)ws, stream);
  else if (a_elem == ELEM_E5M2) launch_deep<ELEM_E5M2>(M, N, K, A, SA, B, SB, C, (float*)ws, stream);
  else if (a_elem == ELEM_E2M1) launch_deep<ELEM_E2M1>(M, N, K, A, SA, B, SB, C, (float*)ws, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int FA>
static void launch_grouped_deep(int64_t G, const int64_t* offsets, int64_t T, int64_t N, int64_t K,
                                const uint8_t* a, const uint8_t* sa, const uint8_t* b, const uint8_t* sb,
                                uint16_t* c, hipStream_t stream) {
  // 64 groups of 4096 x 4096: 16 rows each 129 us in tiles of 32 rows, 157 in
  // 128; 62 rows each 262 and 194
  const bool few = T <= 24 * G;
  // no more row tiles than this: each group ends in at most one that is short
  const int64_t slots = T / (few ? 32 : 128) + G;
  const dim3 grid((unsigned)((N + 127) / 128), (unsigned)(slots < 65535 ? slots : 65535));
  if (few)
    hipLaunchKernelGGL((grouped4_deep_kernel<FA, 1, 4, 1, 1, 2, true>), grid, dim3(256), 0, stream, offsets, G, T,
                       a, sa, b, sb, c, N, K);
  else
    hipLaunchKernelGGL((grouped4_deep_kernel<FA, 2, 2, 2, 2, 1, FA != ELEM_E2M1>), grid, dim3(256), 0, stream,
                       offsets, G, T, a, sa, b, sb, c, N, K);
}

hipError_t launch_grouped_gemm4_deep(int a_elem, int64_t G, const int64_t* offsets, int64_t T,
                                     int64_t N, int64_t K, const void* a, const void* sa,
                                     const void* b, const void* sb, void* c, hipStream_t stream) {
  const uint8_t *A = (const uint8_t*)a, *SA = (const uint8_t*)sa, *B = (const uint8_t*)b,
                *SB = (const uint8_t*)sb;
  uint16_t* C = (uint16_t*)c;
  if (a_elem == ELEM_E4M3) launch_grouped_deep<ELEM_E4M3>(G, offsets, T, N, K, A, SA, B, SB, C, stream);
  else if (a_elem == ELEM_E5M2) launch_grouped_deep<ELEM_E5M2>(G, offsets, T, N, K, A, SA, B, SB, C, stream);
  else if (a_elem == ELEM_E2M1) launch_grouped_deep<ELEM_E2M1>(G, offsets, T, N, K, A, SA, B, SB, C, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace mx
