// Table gradient for operators that own their operands' layout: the cross
// entropy of a sketched head (a range of the vocabulary at a time, tokens
// counted on the device, dY as the sum of two f16 values) and the backward
// from an 8-bit checkpoint (X in a padded workspace).
//
//   dLUT[i][g][c] = sum_{j in g, idx[i][j] = c} sum_t dY[t][i] X[t][j]
//
// As k_gemm_dlut_dma (skm_gemm_bwd.h), one block owns 128 rows x one group (or
// a column / token range of it), accumulates the dW tile of up to 512 columns
// at a time over all tokens on the matrix cores, its operands copied from
// memory into a three-stage LDS ring (global_load_lds), and sums the tile into
// table entries. It differs in
//   * the binning, by plain reads and writes of private bins (dl_bins);
//   * where the copies are issued: between the MFMAs, not at the head of the
//     step, where they held both waves of a SIMD up;
//   * the width of the tile: the last columns of a group take 3, 2 or 1 tiles
//     per wave instead of 4 (a group of 1376 columns costs 11 / 12 of three
//     full chunks, one of 128 a quarter of one);
//   * ragged tokens: the last step's rows of dY past the tokens are read from
//     16 zero bytes, so every token count takes this kernel.
//   * a second addend of dY shares the step's X fragments (k_dlut_piece's TWO).
// Bound by the K loop's LDS reads (1.5 per MFMA; 1 with two addends). 8192
// tokens, 4096 x 11008 in 8 groups, b = 4: 717 us as k_gemm_dlut_dma, 603-640 us
// here (1155-1225 TFLOP/s); two addends, 32000 x 4096, three quarters of 4096
// tokens: 1447 us with the tokens taken twice, 1219 us (1321 TFLOP/s).
#pragma once

#include "skm_gemm_bwd.h"

namespace skm {

namespace {

struct DlPiece {
  static constexpr bool PIECE = true;
  const int32_t* count;    // tokens; NULL = m. X holds zeros up to a multiple of 32
  int64_t ldy;             // row stride of dY, as above
  int64_t lo_off;          // dY + lo_off: a second addend of dY (k_dlut_piece's TWO)
  const float* inv_scale;  // the sums are multiplied by *inv_scale; NULL = 1
  const void* zeros;       // 16 zero bytes read in place of dY's rows past the
                           // tokens; NULL = those rows exist and hold zeros
};

// dd_dma16 without its compiler fence, for copies placed between reads of other
// stages and MFMAs (dd_barrier and the waits keep them apart from the reads of
// their own stage).
__device__ __forceinline__ void dd_dma16_free(const void* src, uint32_t lds) {
  uint32_t keep;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(keep)
      : "v"(src), "s"(lds));
}

// ---- binning with private bins ------------------------------------------------
// A lane holds one weight row i = 64 wm +
// 32 a + lane % 32 and, per 32-column tile b, the 16 columns 8 q + 4 (lane /
// 32) + k. Every lane adds into its own copies of its row's bins, entry-major
// / lane-minor (per wave [a][b / 2][entry][64 lanes], 128 KB in all, over the
// operand ring, which is free between chunks): the 64 lanes of an access hit
// 64 banks whatever the indices are, and since no other lane touches a copy,
// an addition is a read, an add and a write. (An LDS fp32 atomic add takes 3
// cycles per lane: 92 us for the 65536 additions of a block, the whole cost of
// a call with few tokens; with 8192 tokens a chunk's matrix work takes 200 us.)
// The four copies of a wave are four independent chains of 32 additions, which
// hides most of the read latency. A lane's indices are whole 32-column units
// of its row, loaded straight into registers. The sixteen copies of an entry
// (4 column waves x 2 x 2 lane halves) are then added in a fixed order into
// the registers of the thread that owns it: thread t has entries K/4 (t / 128)
// .. of row t % 128.
constexpr uint32_t DP_COPY = 16u * 256u;      // one copy: 16 entries x 64 lanes
constexpr uint32_t DP_WAVE = 4u * DP_COPY;
static_assert(8u * DP_WAVE <= DD_LDS, "the bins of 8 waves fit the block's LDS");

// NBT: the wave's 32-column tiles (its columns start at j0 + 32 NBT wn)
template <int B, int NBT>
__device__ __forceinline__ void dl_bins(const f32x16 (&acc)[2][4], const uint8_t* __restrict__ idx_packed,
                                        uint32_t lane, int wave, int t, int64_t i0, int64_t n, int64_t d, int64_t j0,
                                        int64_t jend, float (&bins)[4]) {
  constexpr int K = 1 << B;
  const int wm = wave & 1, wn = wave >> 1;
  // (opaque copies: the addresses below would be hoisted out of the chunk loop
  // and stay live across the K loop)
  asm volatile("" : "+v"(lane), "+v"(t));
  const uint32_t h = lane >> 5;
  const uint32_t mine = (uint32_t)wave * DP_WAVE + lane * 4u;
  constexpr int HALF = (NBT + 1) / 2;  // tiles of a row's first copy
  const int64_t jw = j0 + 32 * NBT * wn;
  uint32_t w[2][NBT][B];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int64_t i = i0 + 64 * wm + 32 * a + (lane & 31u);
    const uint8_t* row = idx_packed + (i < n ? i : n - 1) * (d * B / 8);
#pragma unroll
    for (int b = 0; b < NBT; ++b) {
      const int64_t j = jw + 32 * b;  // (past the range: any unit of the row, its sums are dropped)
      load_unit<B>(row, (j < jend ? j : j0) / 32, w[a][b]);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
#pragma unroll
    for (int c = 0; c < K; ++c) st_w(mine + (uint32_t)v * DP_COPY + (uint32_t)c * 256u, 0u);
  // the four fields 8 q + 4 h .. + 3 of tile (a, b)'s unit, from bit 0 on
  auto fields = [&](int a, int b, int q) -> uint32_t {
    if constexpr (B == 4) {
      return w[a][b][q] >> (16u * h);
    } else if constexpr (B == 2) {
      return w[a][b][q >> 1] >> (16u * (q & 1) + 8u * h);
    } else {
      const int b0 = 24 * q, b1 = 24 * q + 12;  // first bit for either half
      const uint32_t w0 = h ? w[a][b][b1 >> 5] : w[a][b][b0 >> 5];
      const uint32_t w1 = h ? w[a][b][(b1 >> 5) < 2 ? (b1 >> 5) + 1 : 2] : w[a][b][(b0 >> 5) < 2 ? (b0 >> 5) + 1 : 2];
      return __builtin_amdgcn_alignbit(w1, w0, (24u * q + 12u * h) & 31u);
    }
  };
#pragma unroll
  for (int bb = 0; bb < HALF; ++bb) {
    // tiles bb and HALF + bb; a tile is inside the range or not as a whole
    // (wave-uniform), and the second one is not when the first is not
    if (jw + 32 * bb >= jend) break;
    const bool two = HALF + bb < NBT && jw + 32 * (HALF + bb) < jend;
    constexpr int NV = NBT > 1 ? 4 : 2;  // chains: (row tile, copy), or the row tiles
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t f[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int a = NBT > 1 ? v >> 1 : v, b = NBT > 1 ? (v & 1) * HALF + bb : bb;
        f[v] = fields(a, b < NBT ? b : bb, q);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t at[NV];
        float s[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          at[v] = mine + (uint32_t)(NBT > 1 ? v : 2 * v) * DP_COPY + (((f[v] >> (B * k)) & (uint32_t)(K - 1)) << 8);
          s[v] = __builtin_bit_cast(float, ld_w(at[v]));
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int a = NBT > 1 ? v >> 1 : v, b = NBT > 1 ? (v & 1) * HALF + bb : bb;
          const float x = b < NBT && (b < HALF || two) ? acc[a][b < NBT ? b : 0][4 * q + k] : 0.0f;
          st_w(at[v], __builtin_bit_cast(uint32_t, s[v] + x));
        }
      }
    }
  }
  __syncthreads();
  const uint32_t r = (uint32_t)t & 127u, c0 = ((uint32_t)t >> 7) * (uint32_t)(K / 4);
#pragma unroll
  for (int k = 0; k < K / 4; ++k) {
    float s = bins[k];
#pragma unroll
    for (int v = 0; v < 16; ++v)  // column wave, copy, lane half
      s += __builtin_bit_cast(float, ld_w(((r >> 6) + 2u * (v >> 2)) * DP_WAVE +
                                          (2u * ((r >> 5) & 1u) + ((v >> 1) & 1)) * DP_COPY + (c0 + k) * 256u +
                                          ((r & 31u) + 32u * (v & 1)) * 4u));
    bins[k] = s;
  }
}

// the block's entries, times scale
template <int B>
__device__ __forceinline__ void dl_put_bins(float* __restrict__ dLUT, int64_t i0, int64_t n, int gpr, int g,
                                            int accumulate, int t, const float (&bins)[4], float scale) {
  constexpr int K = 1 << B;
  const int64_t i = i0 + (t & 127);
  if (i >= n) return;
  float* dst = dLUT + (i * gpr + g) * K + (t >> 7) * (K / 4);
#pragma unroll
  for (int k = 0; k < K / 4; ++k) dst[k] = accumulate ? dst[k] + bins[k] * scale : bins[k] * scale;
}


template <int V> struct tiles_tag { static constexpr int value = V; };
template <bool V> struct bool_tag { static constexpr bool value = V; };

// TWO: dY is the sum of two addends. A step holds both and multiplies them by
// the same X fragments, 1 LDS read per MFMA instead of 1.5 (and X is copied
// once), as against the tokens once per addend.
template <bool TWO> struct DpStage {
  static constexpr uint32_t X0 = (TWO ? 2u : 1u) * DD_TA;       // X behind dY
  static constexpr uint32_t BYTES = DD_STAGE - DD_TA + X0;
  static constexpr uint32_t LDS = 3u * BYTES > DD_LDS ? 3u * BYTES : DD_LDS;
};
static_assert(DpStage<true>::LDS <= 160u * 1024u, "three stages fit the CU's LDS");

template <int B, typename TX, bool TWO>
__global__ void __launch_bounds__(512, 1)
k_dlut_piece(const TX* __restrict__ dY, const TX* __restrict__ X, const uint8_t* __restrict__ idx_packed, int64_t m,
             int64_t n, int64_t d, int gpr, int gband, float* __restrict__ dLUT, int accumulate, int tsplits,
             int csplits, int64_t split_tokens, int64_t split_cols, int64_t part_stride, DlPiece pa) {
  typedef mfma32<TX> MF;
  extern __shared__ uint32_t smem[];  // dynamic LDS only: starts at address 0
  (void)smem;

  const int t = threadIdx.x;
  const uint32_t lane = (uint32_t)(t & 63);
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  if (pa.count) m = *pa.count;
  // block order as in k_gemm_dlut_dma: one split (varying slowest), in it
  // `gband` groups of consecutive row blocks per XCD
  const uint32_t lba = xcd_block(blockIdx.x, gridDim.x);
  const uint32_t nb0 = gridDim.x / (uint32_t)(tsplits * csplits);
  const uint32_t sp = lba / nb0, lb = lba % nb0;
  const uint32_t cr = sp / (uint32_t)tsplits;  // column range of the group
  {
    const int64_t tok0 = (int64_t)(sp % (uint32_t)tsplits) * split_tokens;
    dY += tok0 * pa.ldy;
    X += tok0 * d;
    m = m - tok0 < split_tokens ? m - tok0 : split_tokens;
    dLUT += (int64_t)sp * part_stride;
  }
  const uint32_t rblocks = nb0 / (uint32_t)gpr;
  const uint32_t gi = lb % (uint32_t)gband, rest = lb / (uint32_t)gband;
  const int64_t i0 = (int64_t)(rest % rblocks) * DL_BM;
  const int g = (int)((rest / rblocks) * (uint32_t)gband + gi);
  const int64_t G = d / gpr;
  const int64_t jg0 = (int64_t)g * G + (int64_t)cr * split_cols;
  const int64_t jend = (int64_t)g * G + G < jg0 + split_cols ? (int64_t)g * G + G : jg0 + split_cols;
  // steps of 32 tokens (a token range may start past the tokens that exist: no
  // step, zeros)
  const int KS = m <= 0 ? 0 : (int)((m + DL_BK - 1) / DL_BK);
  constexpr uint32_t X0 = DpStage<TWO>::X0, STAGE = DpStage<TWO>::BYTES;
  constexpr int NA = TWO ? 4 : 2;      // fragments of dY in a half step
  constexpr int NC = TWO ? 6 : 5;      // copies of a wave in a step

  // ---- DMA roles: this wave's token rows 4 wave .. +3. dY: one 1 KB
  // instruction (lane = row (lane / 16) x slot (lane % 16)); X: one
  // instruction per row (lane = slot).
  const uint32_t ycg = (lane & 15u) ^ (((lane >> 4) & 3u) << 2);
  const int64_t yrow = i0 + 8 * (int64_t)ycg <= pa.ldy - 8 ? i0 + 8 * (int64_t)ycg : pa.ldy - 8;
  const TX* ysrc = dY + (int64_t)(4u * (uint32_t)wave + (lane >> 4)) * pa.ldy + yrow;
  const uint32_t ydst = 1024u * (uint32_t)wave;
  const uint32_t xdst = X0 + 4096u * (uint32_t)wave;
  const int64_t ystep = (int64_t)DL_BK * pa.ldy;
  const int64_t xstep = (int64_t)DL_BK * d;
  // lanes whose row of dY in the last step is past the tokens
  const bool past = !TWO && pa.zeros && (int64_t)(KS - 1) * DL_BK + 4 * wave + (int)(lane >> 4) >= m;

  // ---- matrix roles: fragment addresses relative to a stage
  const int wm = wave & 1, wn = wave >> 1;
  const uint32_t fs = lane & 15u;
  const uint32_t frow = 8u * (lane >> 5) + (fs >> 2);
  const uint32_t fx = (fs >> 2) << 2;  // swizzle of the fragment's rows (frow % 4 == fs / 4)
  const uint32_t fin = 2u * ((lane >> 4) & 1u) + ((fs & 3u) >> 1);
  const uint32_t fw = 8u * (fs & 1u);
  uint32_t fa[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) fa[a] = frow * 256u + (((8u * wm + 4u * a + fin) ^ fx) << 4) + fw;

  float bins[4] = {};  // the thread's entries (dl_bins)

  // one chunk of up to 128 NBT columns from j0 on
  auto chunk = [&](int64_t j0, auto nbt) __attribute__((always_inline)) {
    constexpr int NBT = decltype(nbt)::value;
    constexpr int NF = NA + NBT;  // fragments of a half step: dY, X
    uint32_t fb[NBT];
#pragma unroll
    for (int b = 0; b < NBT; ++b)
      fb[b] = X0 + frow * 1024u + (((4u * NBT * wn + 4u * b + fin) ^ fx) << 4) + fw;
    // address of read r (0 .. 2 NF - 1) of a half step: fragment r / 2, first
    // or second four token rows
    auto rd = [&](uint32_t stage, int ks, int r) __attribute__((always_inline)) -> u32x2 {
      const int f = r >> 1;
      const uint32_t rs = f < NA ? 256u : 1024u;
      return ld_tr(stage + (f < NA ? fa[f & 1] + DD_TA * (uint32_t)(f >> 1) : fb[f < NA ? 0 : f - NA]) +
                   (16u * (uint32_t)ks + 4u * (r & 1)) * rs);
    };
    f32x16 acc[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < NBT; ++b) zero16(acc[a][b]);
    __syncthreads();  // the previous chunk's bins have been read
    const char* ys = reinterpret_cast<const char*>(ysrc);
    const char* xs[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int64_t col = j0 + 8 * (int64_t)(lane ^ ((uint32_t)h << 2));
      xs[h] = reinterpret_cast<const char*>(X + (int64_t)(4u * (uint32_t)wave + h) * d + (col <= d - 8 ? col : d - 8));
    }
    // the copies of step k, one at a time (dY, its second addend, 4 rows of X),
    // then the addresses of step k + 1, a step's worth of rows further
    auto copy = [&](int k, uint32_t stage, int c) __attribute__((always_inline)) {
      if (c == 0) {
        const void* yl = ys;
        if (!TWO && pa.zeros && k == KS - 1) yl = past ? pa.zeros : yl;
        dd_dma16_free(yl, stage + ydst);
      } else if (TWO && c == 1) {
        dd_dma16_free(ys + 2 * pa.lo_off, stage + DD_TA + ydst);
      } else if (NBT == 4 || lane < 16u * NBT) {
        dd_dma16_free(xs[c - NC + 4], stage + xdst + 1024u * (uint32_t)(c - NC + 4));
      }
    };
    auto advance = [&]() __attribute__((always_inline)) {
      ys += ystep * 2;
#pragma unroll
      for (int h = 0; h < 4; ++h) xs[h] += xstep * 2;
    };
#pragma unroll
    for (int c = 0; c < NC; ++c) copy(0, 0u, c);
    advance();
    if (KS > 1) {
#pragma unroll
      for (int c = 0; c < NC; ++c) copy(1, STAGE, c);
      advance();
      dd_wait_vmcnt<NC>();
    } else {
      dd_wait_vmcnt<0>();
    }
    dd_barrier();
    // Pipelined across the step barrier: step k's second half of reads runs
    // beside its first half of MFMAs, with the copies of step k + 2 between
    // them; then every read of stage k has landed (lgkmcnt 0) and this wave's
    // copies of step k + 1 (vmcnt), the barrier, and step k + 1's first half of
    // reads runs beside step k's second half of MFMAs. (Stage k + 2 is stage
    // k - 1: every wave finished reading it before the last barrier.)
    u32x2 p[2 * NF], q[2 * NF];  // the two halves' operands
    uint32_t st = 0u;            // stage of step k
    auto frag = [](const u32x2* v, int f) __attribute__((always_inline)) -> u32x4 {
      return u32x4{v[2 * f].x, v[2 * f].y, v[2 * f + 1].x, v[2 * f + 1].y};
    };
    // MFMAs of half v (NA NBT of them) with the reads of the next half into w
    // and, MORE, the copies of step k + 2: pinned group by group
    auto half = [&](const u32x2* v, u32x2* w, uint32_t rst, int ks, int k, uint32_t cst, auto more)
        __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value;
#pragma unroll
      for (int b = 0; b < NBT; ++b) {
#pragma unroll
        for (int r = 2 * NF * b / NBT; r < 2 * NF * (b + 1) / NBT; ++r) w[r] = rd(rst, ks, r);
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[a & 1][b] = MF::run(frag(v, NA + b), frag(v, a), acc[a & 1][b]);
        if constexpr (MORE) {
#pragma unroll
          for (int c = NC * b / NBT; c < NC * (b + 1) / NBT; ++c) copy(k + 2, cst, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto step = [&](int k, auto more) __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value;
      half(p, q, st, 1, k, st >= STAGE ? st - STAGE : st + 2u * STAGE, more);
      if constexpr (MORE) advance();
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): every read of stage k has landed
      if constexpr (MORE) dd_wait_vmcnt<NC>();
      else dd_wait_vmcnt<0>();
      dd_barrier();
      st = st + STAGE == 3u * STAGE ? 0u : st + STAGE;
      // (after the last step this reads a stale stage and the values go unused)
      half(q, p, st, 0, k, 0u, bool_tag<false>{});
    };
#pragma unroll
    for (int r = 0; r < 2 * NF; ++r) p[r] = rd(0u, 0, r);
    int k = 0;
    for (; k + 2 < KS; ++k) step(k, bool_tag<true>{});
    for (; k < KS; ++k) step(k, bool_tag<false>{});
    dd_wait_vmcnt<0>();  // (no copy is in flight here; the compiler does not count them)
    dl_bins<B, NBT>(acc, idx_packed, lane, wave, t, i0, n, d, j0, jend, bins);
  };

  for (int64_t j0 = jg0; j0 < jend && KS > 0; j0 += DL_BN) {
    const int64_t left = jend - j0;
    if (left > 384) chunk(j0, tiles_tag<4>{});
    else if (left > 256) chunk(j0, tiles_tag<3>{});
    else if (left > 128) chunk(j0, tiles_tag<2>{});
    else chunk(j0, tiles_tag<1>{});
  }
  dl_put_bins<B>(dLUT, i0, n, gpr, g, accumulate, t, bins, pa.inv_scale ? *pa.inv_scale : 1.0f);
}

template <int B, typename TX, bool TWO>
hipError_t dlut_piece_launch(const TX* dY, const TX* X, const uint8_t* idx, const Problem& p, float* dLUT,
                           int accumulate, float* part, const DlPiece& pa, hipStream_t s) {
  const auto kern = k_dlut_piece<B, TX, TWO>;
  static const hipError_t prep = prepare_kernel((const void*)kern, DpStage<TWO>::LDS);
  if (prep != hipSuccess) return prep;
  const int64_t rb = (p.n + DL_BM - 1) / DL_BM;
  // bands of 4 groups (or 2, or 1) in the XCD-local block order
  const int gband = p.gpr % 4 == 0 ? 4 : (p.gpr % 2 == 0 ? 2 : 1);
  const DlutSplit sp = dlut_split_of(p);
  const int64_t count = p.n * p.gpr * p.k();
  const bool split = sp.parts() > 1;
  hipLaunchKernelGGL(kern, dim3((unsigned)(rb * p.gpr * sp.parts())), dim3(512), DpStage<TWO>::LDS, s, dY, X, idx, p.m,
                     p.n, p.d, p.gpr, gband, split ? part : dLUT, split ? 0 : accumulate, sp.tsplits, sp.csplits,
                     sp.tokens, sp.cols, count, pa);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && split) e = dlut_reduce(part, sp.parts(), count, dLUT, accumulate, s);
  return e;
}

}  // namespace

}  // namespace skm
