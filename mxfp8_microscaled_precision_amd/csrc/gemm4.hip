// Products with 4-bit MX weights for gfx950: C[m][n] = sum_k A[m][k] B[n][k]
// with B in E2M1 (two codes to a byte) and A in E4M3, E5M2 or E2M1, one E8M0
// scale per 32 K-elements of each operand row, FP32 accumulation and a BF16
// result; dense, and grouped by device-side expert offsets.  The pages name
// 4-bit weights with 8-bit activations for serving and 4-bit training of the
// routed experts (practice page, w4a8-mx; torchtitan-npu MXFP8/HiF8 tutorial,
// step-2 environment table, ENABLE_MXFP4_QAT).  This file has the large tiles
// for many rows; gemm4_deep.hip has the small ones, for everything else.
//
// Lane layout of v_mfma_scale_f32_32x32x64, found by one-hot operands on the
// device: lane l = 32 g + i holds row i; in 4 bits its 16 bytes are K 32 g ..
// 32 g + 31; in 8 bits its first 16 bytes are K 16 g .. 16 g + 15 and its last
// 16 are K 32 + 16 g ..; its scale byte is that of K 32 g .. 32 g + 31 in both.
// The order of K is free, so long as A and B agree: which block of the data
// stands in which hardware block is chosen for the loads.
#include "gemm4.h"

namespace mx {

// One workgroup tile of 256 x 256 results: four waves of 128 x 128, 4 x 4
// accumulators of 32x32 each.  A K step is 128 bytes of an A row: 128 elements
// in 8 bits, 256 in 4.  Both operands are staged through a double-buffered
// LDS tile; 16-byte chunks are swizzled by row so that the 16 lanes served
// together read 16 bank groups: rows of 128 bytes as in gemm_common.h, B's
// rows of 64 bytes (8-bit A) with chunk c of row r at c ^ (r / 4 & 3).
//
// Which blocks meet.  4-bit A: a 16-byte chunk of either operand is one block;
// half S of a step reads chunks 2 S + g and 4 + 2 S + g (g: lane half), two
// MFMAs of blocks (2 S, 2 S + 1) and (4 + 2 S, 4 + 2 S + 1).  8-bit A: half S
// multiplies blocks S and 2 + S, of which A's lanes hold 16 bytes each (chunks
// 2 S + g and 4 + 2 S + g) and B's lane half g the block 2 g + S (chunk 2 g +
// S).
//
// WHOLE: K is a multiple of 512 and N of 8, and the scales begin at 16-byte
// addresses.  Otherwise chunks past the end of a row are not loaded (they read
// as zero), the scales are loaded in dwords at any address, the last one of a
// row ending with the row, and the result leaves in pieces of 16 bytes at any
// address.
template <int FA, bool WHOLE>
struct Tile4 {
  static constexpr int F = 4;
  static constexpr bool A4 = FA == ELEM_E2M1;
  static constexpr int ROWS = 64 * F;
  static constexpr int KS = A4 ? 256 : 128;    // elements of a K step
  static constexpr int SB = KS / 32;           // scale bytes of a row and step
  static constexpr int GS = 16 / SB;           // steps that 16 scale bytes last
  static constexpr int BROW = A4 ? 128 : 64;   // bytes of a B row and step
  static constexpr int A_BYTES = ROWS * 128, B_BYTES = ROWS * BROW;
  static constexpr int A_OPS = 2 * F, B_OPS = A4 ? 2 * F : F;  // 1 KB loads of a wave and step
  static constexpr int DS_READS = A4 ? 4 * F : 3 * F;          // 16-byte LDS reads of half a step

  const uint8_t* __restrict__ a;
  const uint8_t* __restrict__ sa;
  const uint8_t* __restrict__ b;
  const uint8_t* __restrict__ sb;
  int64_t m0, m_end, n0, N, K;
  int64_t nks, nkb;
  uint32_t row_a, row_b;  // bytes of a row, for a lane's chunks at pos_a and pos_b of a step
  uint32_t pos_a, pos_b;
  lds_u8 *st0, *st1;  // stages: A tile, then B tile
  lds_u8 *ss0, *ss1;  // scale tiles of 16 bytes a row: A's rows, then B's
  u32x4 ra, rb, rsa, rsb;
  uint32_t voff_a, voff_b, a_step, b_step, svoff;
  lds_u8* pf_scratch;  // L2 prefetch as in the 8-bit GEMM (gemm.hip)
  uint32_t pf_row_a, pf_row_b, pf_a, pf_b;

  __device__ __forceinline__ void setup(int wave, int lane) {
    const int64_t mrows = m_end - m0, nrows = (N - n0) < ROWS ? (N - n0) : ROWS;
    const int64_t pa = A4 ? K >> 1 : K, pb = K >> 1;
    nks = (K + KS - 1) / KS;
    nkb = K >> 5;
    ra = make_rsrc(a + m0 * pa, mrows * pa);
    rb = make_rsrc(b + n0 * pb, nrows * pb);
    rsa = make_rsrc(sa + m0 * nkb, mrows * nkb);
    rsb = make_rsrc(sb + n0 * nkb, nrows * nkb);
    // A: load t = wave + 4 u covers LDS rows 8 t .. 8 t + 7; lane i lands in
    // row r = 8 t + i / 8 at physical chunk i % 8, logical (i % 8) ^ swz(r)
    const int sw = (4 * wave + (lane >> 4)) & 7;
    row_a = (uint32_t)pa, row_b = (uint32_t)pb;
    pos_a = 16 * ((lane & 7) ^ sw);
    voff_a = (uint32_t)((8 * wave + (lane >> 3)) * pa) + pos_a;
    a_step = (uint32_t)(32 * pa);
    if (A4) {
      pos_b = pos_a;
      voff_b = (uint32_t)((8 * wave + (lane >> 3)) * pb) + pos_b;
      b_step = (uint32_t)(32 * pb);
    } else {
      // rows of 64 bytes: load t covers LDS rows 16 t .. 16 t + 15; lane i
      // lands in row 16 t + i / 4 at chunk i % 4, logical (i % 4) ^ (i / 16)
      pos_b = 16 * ((lane & 3) ^ (lane >> 4));
      voff_b = (uint32_t)((16 * wave + (lane >> 2)) * pb) + pos_b;
      b_step = (uint32_t)(64 * pb);
    }
    svoff = (uint32_t)((64 * wave + lane) * nkb);
    pf_row_a = (uint32_t)((64 * wave + lane) * pa);
    pf_row_b = (uint32_t)((64 * wave + lane) * pb);
  }

  // Loads of step kt into stage st; a step past the last touches no memory.
  __device__ __forceinline__ void load_a(lds_u8* st, int64_t kt, int u, int wave) {
    const bool in = WHOLE ? kt < nks : (uint32_t)(128 * kt) + pos_a < row_a;
    const uint32_t base = in ? (uint32_t)(128 * kt) : OOB;
    dma16(st + (wave + 4 * u) * 1024, voff_a + base + u * a_step, ra);
  }
  __device__ __forceinline__ void load_b(lds_u8* st, int64_t kt, int u, int wave) {
    const bool in = WHOLE ? kt < nks : (uint32_t)(BROW * kt) + pos_b < row_b;
    const uint32_t base = in ? (uint32_t)(BROW * kt) : OOB;
    dma16(st + A_BYTES + (wave + 4 * u) * 1024, voff_b + base + u * b_step, rb);
  }
  __device__ __forceinline__ void issue_stage(lds_u8* st, int64_t kt, int wave) {
#pragma unroll
    for (int u = 0; u < A_OPS; u++) load_a(st, kt, u, wave);
#pragma unroll
    for (int u = 0; u < B_OPS; u++) load_b(st, kt, u, wave);
  }

  // Scale bytes of GS steps: 16 bytes a row if WHOLE, otherwise four planes of a
  // dword a row
  __device__ __forceinline__ void issue_scales(lds_u8* buf, int64_t group, int wave) {
    if constexpr (WHOLE) {
      const uint32_t off = 16 * group < nkb ? svoff + (uint32_t)(16 * group) : OOB;
      dma16(buf + wave * 1024, off, rsa);
      dma16(buf + 4096 + wave * 1024, off, rsb);
    } else {
#pragma unroll
      for (int d = 0; d < 4; d++) {
        const uint32_t at = (uint32_t)(16 * group) + 4 * d, n = (uint32_t)nkb;
        const uint32_t off = at < n ? svoff + (at + 4 <= n ? at : n - 4) : OOB;
        dma4(buf + d * 1024 + wave * 256, off, rsa);
        dma4(buf + 4096 + d * 1024 + wave * 256, off, rsb);
      }
    }
  }

  // A row's scale bytes of one step (8 of them: `hi` the last four) as the
  // word whose byte S + 2 h (4-bit A: MFMA h of half S) or S (8-bit A) is this
  // lane half's.
  __device__ __forceinline__ static uint32_t shape_scale(uint32_t lo, uint32_t hi, int g) {
    if (A4) return __builtin_amdgcn_perm(hi, lo, g ? 0x07050301u : 0x06040200u);
    return lo >> (16 * g);
  }
  // Scales of step kt, the one numbered q of the GS whose scales buf holds
  __device__ __forceinline__ void read_scales(const lds_u8* buf, int q, int64_t kt, int wm, int wn, int lane,
                                              uint32_t* sar, uint32_t* sbr) {
    const int g = lane >> 5, i = lane & 31;
    if constexpr (WHOLE) {
#pragma unroll
      for (int f = 0; f < F; f++) {
        const lds_u8* pa = buf + (32 * F * wm + 32 * f + i) * 16 + SB * q;
        const lds_u8* pb = buf + 4096 + (32 * F * wn + 32 * f + i) * 16 + SB * q;
        if (A4) {
          const v2i x = *(const lds_v2i*)pa, y = *(const lds_v2i*)pb;
          sar[f] = shape_scale((uint32_t)x.x, (uint32_t)x.y, g);
          sbr[f] = shape_scale((uint32_t)y.x, (uint32_t)y.y, g);
        } else {
          sar[f] = *(const lds_u16*)(pa + 2 * g);
          sbr[f] = *(const lds_u16*)(pb + 2 * g);
        }
      }
    } else {
      typedef const __attribute__((address_space(3))) uint32_t lds_u32;
      // a dword that ended with the row holds bytes of the block before it;
      // one past the row was not loaded and is 0
      const int over0 = (int)(SB * kt + 4 - nkb), over1 = over0 + 4;
      const int sh0 = over0 > 0 ? (8 * over0) & 31 : 0, sh1 = over1 > 0 ? (8 * over1) & 31 : 0;
      const lds_u8* plane = buf + q * (SB / 4) * 1024;
#pragma unroll
      for (int f = 0; f < F; f++) {
        const lds_u8* pa = plane + 4 * (32 * F * wm + 32 * f + i);
        const lds_u8* pb = plane + 4096 + 4 * (32 * F * wn + 32 * f + i);
        uint32_t a1 = 0, b1 = 0;
        if (A4) a1 = *(lds_u32*)(pa + 1024) >> sh1, b1 = *(lds_u32*)(pb + 1024) >> sh1;
        sar[f] = shape_scale(*(lds_u32*)pa >> sh0, a1, g);
        sbr[f] = shape_scale(*(lds_u32*)pb >> sh0, b1, g);
      }
    }
  }

  // Fragment f of an operand for half S of the step in stage st
  template <int S>
  __device__ __forceinline__ static v8i frag_a(const lds_u8* st, int wm, int f, int lane) {
    return read_frag(st, 32 * F * wm + 32 * f + (lane & 31), S, lane >> 5);
  }
  template <int S>
  __device__ __forceinline__ static v8i frag_b(const lds_u8* st, int wn, int f, int lane) {
    const int row = 32 * F * wn + 32 * f + (lane & 31), g = lane >> 5;
    if (A4) return read_frag(st + A_BYTES, row, S, g);
    const v4i x = *(const lds_v4i*)(st + A_BYTES + row * 64 + (((2 * g + S) ^ ((row >> 2) & 3)) << 4));
    return (v8i){x.x, x.y, x.z, x.w, 0, 0, 0, 0};
  }
  template <int S>
  __device__ __forceinline__ static void read_frags(const lds_u8* st, int wm, int wn, int lane, v8i* af,
                                                    v8i* bf) {
#pragma unroll
    for (int f = 0; f < F; f++) af[f] = frag_a<S>(st, wm, f, lane);
#pragma unroll
    for (int f = 0; f < F; f++) bf[f] = frag_b<S>(st, wn, f, lane);
  }

  __device__ __forceinline__ static v8i half_of(v8i v, int h) {
    return h ? (v8i){v[4], v[5], v[6], v[7], 0, 0, 0, 0} : (v8i){v[0], v[1], v[2], v[3], 0, 0, 0, 0};
  }
  template <int S>
  __device__ __forceinline__ static void mma(const v8i* af, const v8i* bf, const uint32_t* sar,
                                             const uint32_t* sbr, v16f (&acc)[F][F]) {
    if constexpr (A4) {
#pragma unroll
      for (int fn = 0; fn < F; fn++)
#pragma unroll
        for (int fm = 0; fm < F; fm++)
          acc[fn][fm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              half_of(bf[fn], 0), half_of(af[fm], 0), acc[fn][fm], ELEM_E2M1, ELEM_E2M1, S, (int)sbr[fn],
              S, (int)sar[fm]);
#pragma unroll
      for (int fn = 0; fn < F; fn++)
#pragma unroll
        for (int fm = 0; fm < F; fm++)
          acc[fn][fm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              half_of(bf[fn], 1), half_of(af[fm], 1), acc[fn][fm], ELEM_E2M1, ELEM_E2M1, S + 2,
              (int)sbr[fn], S + 2, (int)sar[fm]);
    } else {
#pragma unroll
      for (int fn = 0; fn < F; fn++)
#pragma unroll
        for (int fm = 0; fm < F; fm++)
          acc[fn][fm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              bf[fn], af[fm], acc[fn][fm], ELEM_E2M1, FA, S, (int)sbr[fn], S, (int)sar[fm]);
    }
  }
  __device__ __forceinline__ static void clear(v16f (&acc)[F][F]) {
#pragma unroll
    for (int x = 0; x < F; x++)
#pragma unroll
      for (int y = 0; y < F; y++) acc[x][y] = (v16f){};
  }

  // Phase A of step kt: MFMAs of half 0 on registers F0, reads of half 1 into
  // F1; barrier: every wave has read stage kt, stage kt + 1 has landed; phase
  // B: loads of stage kt + 2 into the buffer just released, MFMAs of half 1,
  // reads of half 0 of stage kt + 1 and of its scales.  The waits leave the
  // two latest vector-memory operations in flight: a step's L2 prefetches.
  __device__ __forceinline__ void prefetch(int64_t kt, int wave) {
    const uint32_t live = kt < nks ? 0u : OOB;
    prefetch_lines(pf_scratch + wave * 512, (pf_row_a + (uint32_t)(128 * kt)) | pf_a | live, ra);
    prefetch_lines(pf_scratch + wave * 512 + 256, (pf_row_b + (uint32_t)(BROW * kt)) | pf_b | live, rb);
  }
  // The next step's scales are number q of those at sread; `group` starts the
  // load of the next group's into sdma.
  __device__ __forceinline__ void step(lds_u8* cur, lds_u8* nxt, const lds_u8* sread, int q, bool group,
                                       lds_u8* sdma, int64_t kt, int wave, int wm, int wn, int lane, uint32_t* sc_a,
                                       uint32_t* sc_b, v8i* f0a, v8i* f0b, v8i* f1a, v8i* f1b,
                                       v16f (&acc)[F][F]) {
    uint32_t nx_a[F], nx_b[F];
    read_frags<1>(cur, wm, wn, lane, f1a, f1b);
    mma<0>(f0a, f0b, sc_a, sc_b, acc);
    interleave<DS_READS>();
    wait_vm_but_prefetch();
    __syncthreads();
    if (group) issue_scales(sdma, kt / GS + 1, wave);
    read_scales(sread, q, kt + 1, wm, wn, lane, nx_a, nx_b);
#pragma unroll
    for (int f = 0; f < F; f++) {
      f0a[f] = frag_a<0>(nxt, wm, f, lane);
#pragma unroll
      for (int u = f * A_OPS / F; u < (f + 1) * A_OPS / F; u++) load_a(cur, kt + 2, u, wave);
    }
#pragma unroll
    for (int f = 0; f < F; f++) {
      f0b[f] = frag_b<0>(nxt, wn, f, lane);
#pragma unroll
      for (int u = f * B_OPS / F; u < (f + 1) * B_OPS / F; u++) load_b(cur, kt + 2, u, wave);
    }
    prefetch(kt + PF_DIST, wave);
    mma<1>(f1a, f1b, sc_a, sc_b, acc);
    interleave<DS_READS + 2 * F>();
#pragma unroll
    for (int f = 0; f < F; f++) {
      sc_a[f] = nx_a[f];
      sc_b[f] = nx_b[f];
    }
  }
  // MFMA, LDS read, MFMA, ... for half a step's instructions
  template <int NDS>
  __device__ __forceinline__ static void interleave() {
    constexpr int n = F * F * (A4 ? 2 : 1), per = (NDS + n - 1) / n;
#pragma unroll
    for (int i = 0; i < n; i++) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
    }
  }

  // The prologue in parts, for a caller that starts a tile's loads while it
  // stores the last one's result: first() loads stage 0 and its scales,
  // second() stage 1; run() waits for stage 0 (with `stored`, NST stores
  // were issued between the two) and runs the K loop.
  __device__ __forceinline__ void first(int wave) {
    issue_stage(st0, 0, wave);
    issue_scales(ss0, 0, wave);
  }
  __device__ __forceinline__ void second(int wave) { issue_stage(st1, 1, wave); }
  template <int NST>
  __device__ __forceinline__ void run(v16f (&acc)[F][F], int wave, int lane, bool stored) {
    const int wm = wave & 1, wn = wave >> 1;
    clear(acc);
    if (stored)
      wait_vm<NST + A_OPS + B_OPS>();
    else
      wait_vm<A_OPS + B_OPS>();
    __syncthreads();
    uint32_t sc_a[F], sc_b[F];
    v8i f0a[F], f0b[F], f1a[F], f1b[F];
    read_scales(ss0, 0, 0, wm, wn, lane, sc_a, sc_b);
    prefetch(2, wave);
    read_frags<0>(st0, wm, wn, lane, f0a, f0b);
    constexpr int STEPS = WHOLE ? GS : 2;  // whole groups, or pairs: a step past the last adds zeros
    for (int64_t k0 = 0; k0 < nks; k0 += STEPS) {
      const int64_t j = k0 / GS;
      lds_u8 *scur = (j & 1) ? ss1 : ss0, *snxt = (j & 1) ? ss0 : ss1;
#pragma unroll
      for (int u = 0; u < STEPS; u++) {
        const int64_t kt = k0 + u;
        const int q = WHOLE || GS == 2 ? (u + 1) % GS : (int)(kt + 1) % GS;
        const bool group = WHOLE || GS == 2 ? u == 0 : kt % GS == 0;
        step(u & 1 ? st1 : st0, u & 1 ? st0 : st1, q == 0 ? snxt : scur, q, group, snxt, kt, wave, wm, wn, lane,
             sc_a, sc_b, f0a, f0b, f1a, f1b, acc);
      }
    }
  }
};

// Persistent: one workgroup per compute unit
// walks tiles bid, bid + grid, ...; a tile's first loads run while the last
// one's result is stored.  Bound by the matrix unit and the power it may draw:
// 32768 x 18432 x 7168 with both operands in 4 bits takes 1.98 to 2.14 ms (4.0
// to 4.4 PFLOP/s), the unit busy 60% of the time at a clock of 1.54 GHz.  Rows
// that end off a K step of 128 elements cost more (2048 x 7168 x 18432 240 us,
// x 18304 298, x 18400, whose rows begin inside a line, 380).
template <int FA, bool WHOLE>
__global__ void __launch_bounds__(NT)
gemm4_persistent_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                        const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                        uint16_t* __restrict__ c, int64_t M, int64_t N, int64_t K) {
  __shared__ __attribute__((aligned(16))) uint8_t smem0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t smem1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sscale[2 * SCALE_TILE];
  __shared__ __attribute__((aligned(16))) uint8_t spf[2048];
  const int64_t nm = (M + BM - 1) / BM, nn = (N + BN - 1) / BN, tiles = nm * nn;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typedef Tile4<FA, WHOLE> T;
  auto make = [&](int64_t t, T& tl) {
    int64_t mt, nt;
    tile_of(t, nm, nn, mt, nt);
    tl.a = a, tl.sa = sa, tl.b = b, tl.sb = sb;
    tl.m0 = mt * BM;
    tl.m_end = (mt + 1) * BM < M ? (mt + 1) * BM : M;
    tl.n0 = nt * BN;
    tl.N = N, tl.K = K;
    tl.st0 = (lds_u8*)smem0, tl.st1 = (lds_u8*)smem1;
    tl.ss0 = (lds_u8*)sscale, tl.ss1 = (lds_u8*)sscale + SCALE_TILE;
    tl.pf_scratch = (lds_u8*)spf;
    tl.pf_a = (nt % (32 / GM_TILES) == 0) ? 0u : OOB;
    tl.pf_b = (mt % GM_TILES == 0 && !tile_runs_rr((uint32_t)nm, (uint32_t)nn)) ? 0u : OOB;
  };
  int64_t t = blockIdx.x;
  if (t >= tiles) return;
  T tl;
  make(t, tl);
  tl.setup(wave, lane);
  tl.first(wave);
  bool stored = false;
  for (;;) {
    tl.second(wave);
    v16f acc[4][4];
    tl.template run<32>(acc, wave, lane, stored);
    const int64_t m0 = tl.m0, m_end = tl.m_end, n0 = tl.n0;
    // every load has landed (none may still be writing LDS) and every wave
    // is past its last read of the stage and scale buffers
    wait_vm_all();
    __syncthreads();
    t += gridDim.x;
    const bool more = __builtin_amdgcn_readfirstlane((int)(t < tiles)) != 0;
    if (more) {
      make(t, tl);
      tl.setup(wave, lane);
      tl.first(wave);
    }
    if constexpr (WHOLE) {
      store_tile_bf16_lds_halves(acc, (lds_u8*)smem1, c, N, m0, m_end, n0, N, wave & 1, wave >> 1, wave,
                                 lane);
      stored = true;
    } else {
      store_bf16(acc, c, N, m0 + 128 * (wave & 1), m_end, n0 + 128 * (wave >> 1), lane);
    }
    if (!more) break;
  }
}

// Grouped: every workgroup derives the tile list from the device-side offsets
// (clamped into [0, T] and made non-decreasing, so bad offsets never address
// outside the operands) and walks it with a static stride, the tiles of a
// group in the dense kernel's order.  131072 tokens over 64 experts of
// 4096 x 4096, 8-bit A: 1.81 to 1.92 ms (2.3 to 2.4 PFLOP/s), the matrix unit busy 63% of the
// time at 1.79 GHz.
template <int FA, bool WHOLE>
__global__ void __launch_bounds__(NT)
grouped_gemm4_kernel(int64_t G, const int64_t* __restrict__ offsets, int64_t T_, int64_t N, int64_t K,
                     const uint8_t* __restrict__ a, const uint8_t* __restrict__ sa,
                     const uint8_t* __restrict__ b, const uint8_t* __restrict__ sb,
                     uint16_t* __restrict__ c) {
  __shared__ __attribute__((aligned(16))) uint8_t smem0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t smem1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sscale[2 * SCALE_TILE];
  __shared__ __attribute__((aligned(16))) uint8_t spf[2048];
  __shared__ int64_t s_off[MAX_GROUPS + 1];
  __shared__ int64_t s_pre[MAX_GROUPS + 1];
  const int64_t nn = (N + BN - 1) / BN;
  for (int64_t g = threadIdx.x; g <= G; g += NT) {
    const int64_t o = offsets[g];
    s_off[g] = o < 0 ? 0 : (o > T_ ? T_ : o);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t prev = 0, acc = 0;
    for (int64_t g = 0; g < G; g++) {
      const int64_t lo = s_off[g] > prev ? s_off[g] : prev;
      const int64_t hi = s_off[g + 1] > lo ? s_off[g + 1] : lo;
      s_off[g] = lo;
      prev = lo;
      s_pre[g] = acc;
      acc += ((hi - lo + BM - 1) / BM) * nn;
    }
    s_off[G] = s_off[G] > prev ? s_off[G] : prev;
    s_pre[G] = acc;
  }
  __syncthreads();
  const int64_t total = s_pre[G];
  const int64_t nwg = gridDim.x, bid = blockIdx.x;
  const int64_t wg = (bid & 7) * (nwg >> 3) + (bid >> 3);  // contiguous tile runs per XCD
  // tile indices fit in 32 bits (the host checks the tile count)
  const uint32_t span = GM_TILES * (uint32_t)nn;
  int64_t g = 0;  // largest g with s_pre[g] <= t: searched once, then advanced
  {
    int64_t hi = G;
    while (hi - g > 1) {
      const int64_t mid = (g + hi) >> 1;
      if (s_pre[mid] <= wg) g = mid; else hi = mid;
    }
  }
  typedef Tile4<FA, WHOLE> T;
  auto make = [&](int64_t t, T& tl) {
    while (s_pre[g + 1] <= t) g++;  // s_pre[G] = total > t stops it
    const uint32_t local = (uint32_t)(t - s_pre[g]);
    const uint32_t nmg = (uint32_t)((s_off[g + 1] - s_off[g] + BM - 1) / BM);
    const uint32_t run = local / span;
    const uint32_t top = run * GM_TILES;
    const uint32_t gsz = (nmg - top) < (uint32_t)GM_TILES ? (nmg - top) : (uint32_t)GM_TILES;
    const uint32_t in = local - run * span;
    const uint32_t nt = in / gsz;
    const int64_t mt = top + (in - nt * gsz);
    tl.a = a, tl.sa = sa;
    tl.b = b + g * N * (K >> 1);
    tl.sb = sb + g * N * (K >> 5);
    tl.m0 = s_off[g] + mt * BM;
    tl.m_end = (tl.m0 + BM) < s_off[g + 1] ? tl.m0 + BM : s_off[g + 1];
    tl.n0 = (int64_t)nt * BN;
    tl.N = N, tl.K = K;
    tl.st0 = (lds_u8*)smem0, tl.st1 = (lds_u8*)smem1;
    tl.ss0 = (lds_u8*)sscale, tl.ss1 = (lds_u8*)sscale + SCALE_TILE;
    tl.pf_scratch = (lds_u8*)spf;
    tl.pf_a = (nt % (32 / GM_TILES) == 0) ? 0u : OOB;
    tl.pf_b = (mt == top && nn > 32) ? 0u : OOB;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t t = wg;
  if (t >= total) return;
  T tl;
  make(t, tl);
  tl.setup(wave, lane);
  tl.first(wave);
  bool stored = false;
  for (;;) {
    tl.second(wave);
    v16f acc[4][4];
    tl.template run<32>(acc, wave, lane, stored);
    const int64_t m0 = tl.m0, m_end = tl.m_end, n0 = tl.n0;
    wait_vm_all();
    __syncthreads();
    t += nwg;
    const bool more = __builtin_amdgcn_readfirstlane((int)(t < total)) != 0;
    if (more) {
      make(t, tl);
      tl.setup(wave, lane);
      tl.first(wave);
    }
    if constexpr (WHOLE) {
      store_tile_bf16_lds_halves(acc, (lds_u8*)smem1, c, N, m0, m_end, n0, N, wave & 1, wave >> 1, wave,
                                 lane);
      stored = true;
    } else {
      store_bf16(acc, c, N, m0 + 128 * (wave & 1), m_end, n0 + 128 * (wave >> 1), lane);
    }
    if (!more) break;
  }
}

// Whole groups of 16 scale bytes, whole 16-byte chunks of a result row and
// 32-bit offsets within a tile's rows of the result.
static bool whole(int64_t N, int64_t K) {
  return K % 512 == 0 && N % 8 == 0 && (int64_t)BM * N * 2 < ((int64_t)1 << 31);
}

// Scales may begin at any address; the whole form loads them 16 bytes at a time.
// (A row of it has a multiple of 16, so the first row's address decides.)  The
// choice of the tiles goes by sizes alone, as the workspace does.
static bool whole_scales(const void* sa, const void* sb) {
  return (((uintptr_t)sa | (uintptr_t)sb) & 15) == 0;
}

// Large tiles where they are done first: a round of them, a tile on each of 256
// compute units, takes 1.5 to 2 times as long as a round of the small ones with
// half their rows (us, large against small, rounds in brackets, 8-bit A.
// Whole: 2048 x 7168 x 18432 240 (1) and 318 (2), 4096 x 4352 x 4096 91 (2) and
// 103 (3), 1024 x 7168 x 18432 203 (1) and 136 (1).  Otherwise: 2048 x 7168 x
// 18400 380 (1) and 391 (2), 8192 x 8192 x 2880 196 (4) and 268 (8), 4096 x 4130
// x 2080 79 (2) and 68 (3), 2048 x 18432 x 544 50 (3) and 44 (5)).  Up to 128 rows half a large tile would be empty, and the rounds are
// as many.  K from 128 on: a row has a whole dword of scales.
static bool many(int64_t M, int64_t N, int64_t K) {
  const int64_t large = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  const int64_t small = ((M + 127) / 128) * ((N + 255) / 256);
  return K >= 128 && 100 * ((large + 255) / 256) <= (whole(N, K) ? 67 : 58) * ((small + 255) / 256);
}

template <int FA>
static void launch_many(int64_t M, int64_t N, int64_t K, const uint8_t* a, const uint8_t* sa,
                        const uint8_t* b, const uint8_t* sb, uint16_t* c, int num_cus,
                        hipStream_t stream) {
  const int64_t tiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  const int64_t cus = (num_cus > 8 ? num_cus : 256) / 8 * 8;
  const dim3 grid((unsigned)(tiles < cus ? tiles : cus));
  if (whole(N, K) && whole_scales(sa, sb))
    hipLaunchKernelGGL((gemm4_persistent_kernel<FA, true>), grid, dim3(NT), 0, stream, a, sa, b, sb, c, M, N, K);
  else
    hipLaunchKernelGGL((gemm4_persistent_kernel<FA, false>), grid, dim3(NT), 0, stream, a, sa, b, sb, c, M, N, K);
}

size_t gemm4_workspace(int64_t M, int64_t N, int64_t K) {
  return many(M, N, K) ? 0 : gemm4_deep_workspace(M, N, K);
}

hipError_t launch_gemm4(int a_elem, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                        const void* b, const void* sb, void* c, void* workspace, int num_cus,
                        hipStream_t stream) {
  if (!many(M, N, K)) return launch_gemm4_deep(a_elem, M, N, K, a, sa, b, sb, c, workspace, stream);
  const uint8_t *A = (const uint8_t*)a, *SA = (const uint8_t*)sa, *B = (const uint8_t*)b,
                *SB = (const uint8_t*)sb;
  uint16_t* C = (uint16_t*)c;
  if (a_elem == ELEM_E4M3) launch_many<ELEM_E4M3>(M, N, K, A, SA, B, SB, C, num_cus, stream);
  else if (a_elem == ELEM_E5M2) launch_many<ELEM_E5M2>(M, N, K, A, SA, B, SB, C, num_cus, stream);
  else if (a_elem == ELEM_E2M1) launch_many<ELEM_E2M1>(M, N, K, A, SA, B, SB, C, num_cus, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_grouped_gemm4(int a_elem, int64_t G, const int64_t* offsets, int64_t T, int64_t N,
                                int64_t K, const void* a, const void* sa, const void* b,
                                const void* sb, void* c, int num_cus, hipStream_t stream) {
  if (G < 1 || G > MAX_GROUPS) return hipErrorInvalidValue;
  // Large tiles from 96 rows a group on (us, large against small, 64 groups of
  // 4096 x 4096: 128 rows each 267 and 261 with an 8-bit A, 187 and 234 with a
  // 4-bit one, 192 rows each 284 and 339, 78 rows each 255 and 205), where rows do
  // not fill the loads from 192 (4096 x 2080: 256 rows each 260 and 263, with a
  // 4-bit A 192 rows each 156 and 222, 128 rows each 213 and 165); and from 150
  // tiles on, with half a tile empty in each group (8 groups of N x 4096: 157 tiles
  // 46 and 54, 114 tiles 47 and 35; one group: 258 tiles 54 and 83, 70 tiles 44 and
  // 24), where rows do not fill the loads from 256 (8 groups of 4096 x 2880: 189
  // tiles 51 and 42)
  bool w = whole(N, K);
  const int64_t halves = (2 * T / BM + G) * ((N + BN - 1) / BN);
  if (K < 128 || T < (w ? 96 : 192) * G || halves < 2 * (w ? 150 : 256))
    return launch_grouped_gemm4_deep(a_elem, G, offsets, T, N, K, a, sa, b, sb, c, stream);
  w = w && whole_scales(sa, sb);
  const int64_t upper = ((T + BM - 1) / BM + G) * ((N + BN - 1) / BN);
  int64_t wgs = ((num_cus > 0 ? num_cus : 256) + 7) / 8 * 8;
  if (upper < wgs) wgs = (upper + 7) / 8 * 8;
#define MX_GROUPED4(FA_, WHOLE_)                                                                  \
  hipLaunchKernelGGL((grouped_gemm4_kernel<FA_, WHOLE_>), dim3((unsigned)wgs), dim3(NT), 0, stream, G, \
                     offsets, T, N, K, (const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b,  \
                     (const uint8_t*)sb, (uint16_t*)c)
  if (a_elem == ELEM_E4M3 && w) MX_GROUPED4(ELEM_E4M3, true);
  else if (a_elem == ELEM_E4M3) MX_GROUPED4(ELEM_E4M3, false);
  else if (a_elem == ELEM_E5M2 && w) MX_GROUPED4(ELEM_E5M2, true);
  else if (a_elem == ELEM_E5M2) MX_GROUPED4(ELEM_E5M2, false);
  else if (a_elem == ELEM_E2M1 && w) MX_GROUPED4(ELEM_E2M1, true);
  else if (a_elem == ELEM_E2M1) MX_GROUPED4(ELEM_E2M1, false);
  else return hipErrorInvalidValue;
#undef MX_GROUPED4
  return hipGetLastError();
}

}  // namespace mx
