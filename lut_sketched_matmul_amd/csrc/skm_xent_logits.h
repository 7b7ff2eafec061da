// Logit tiles of the cross entropy for b = 4 and groups of whole 64-column
// steps: the contraction of k_gemm_fwd64 (skm_gemm_fwd.h) with its activations
// and indices copied straight into LDS.
//
// k_gemm_fwd64 moves its activations through registers, because it converts
// them and puts them into the K order of mm::dequant8_b4. Here a pre-pass
// (k_xent_rows) has done both, for the listed tokens, so that every K-step's
// 256 x 64 activation tile goes from memory into LDS with global_load_lds, and
// so do the indices (each lane fetches the 16 bytes it will dequantise itself).
// What remains for a wave to do beside the MFMAs is the lookup of its weights.
// 2048 tokens x 32000 words of 4096 columns: 497 us through registers; the
// same kernel with the activations' stores left out 411 us, with no staging at
// all 383 us.
//
// Block tile 256 tokens x 256 words, 8 waves of 128 x 64, 64 columns per step;
// waves 0-3 multiply first and stage second, waves 4-7 the other way round.
// LDS (144 KB): A [2][256 tokens][64] and Bt [2][256 words][64] in 128-byte
// rows (mm::swz128), indices [2][512 lanes][16 bytes].
// Copies of step k + 1's activations and of step k + 2's indices are issued in
// step k and waited for (vmcnt) before the barrier that ends it; no other
// global load is in flight in the loop except a group's table, once per group.
#pragma once

#include "skm_gemm_dlut.h"
#include "skm_xent_tiles.h"

namespace skm {

namespace {

constexpr uint32_t XL_A = 0u;
constexpr uint32_t XL_B = 2u * A64_TILE;              // 65536
constexpr uint32_t XL_I = XL_B + 2u * B64_TILE;       // 131072
constexpr uint32_t XL_LDS = XL_I + 2u * 8192u;        // 147456

// Xp: [listed token][d] in TL, K order of dequant8_b4 in every 8 columns
template <typename TL, typename EP, bool SC>
__global__ void __launch_bounds__(512, 1)
k_xent_logits(const TL* __restrict__ Xp, const uint8_t* __restrict__ idx_packed, const TL* __restrict__ lut, int64_t n,
              int64_t d, int gpr, uint32_t ug_magic, typename EP::Args ep, const int32_t* __restrict__ rexp) {
  typedef mm::mfma32<TL> MF;
  extern __shared__ uint32_t smem[];  // dynamic LDS only: starts at address 0
  (void)smem;
  // the blocks that have tokens come first (see k_gemm_fwd64)
  const int64_t m = *ep.count;
  const int64_t mblocks = (m + 255) / 256;
  if (blockIdx.x >= mblocks * ((n + 255) / 256)) return;  // block-uniform

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t m0 = (int64_t)(blockIdx.x % mblocks) * 256, n0 = (int64_t)(blockIdx.x / mblocks) * 256;
  const int KS = (int)(d / 64);
  auto group_of = [&](int j) -> uint32_t { return mm::group_of((uint32_t)(2 * j), ug_magic); };

  // ---- copies. Activations: this wave's rows 32 wave + 8 i + lane / 8, i = 0
  // .. 3; the lane at slot lane % 8 fetches the chunk that belongs there.
  // Indices: the lane's own unit (word row t / 2, unit t % 2 of the step).
  const char* xs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * wave + 8 * i + (lane >> 3);
    const int64_t tok = m0 + r < m ? m0 + r : m - 1;
    xs[i] = reinterpret_cast<const char*>(Xp + tok * d) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  const int64_t grow = n0 + (t >> 1) < n ? n0 + (t >> 1) : n - 1;
  const char* is = reinterpret_cast<const char*>(idx_packed) + grow * (d / 2) + 16 * (t & 1);
  const uint32_t adst = XL_A + 4096u * (uint32_t)wave, idst = XL_I + 1024u * (uint32_t)wave;
  // copy c of a step (0 .. 3: activations of step k + 1, 4: indices of step k + 2)
  auto copy = [&](int k, uint32_t nxt, int c) __attribute__((always_inline)) {
    if (c < 4) dd_dma16_free(xs[c] + (int64_t)(k + 1) * 128, adst + nxt * A64_TILE + 1024u * c);
    else dd_dma16_free(is + (int64_t)(k + 2) * 32, idst + (1u - nxt) * 8192u);
  };

  // ---- staging: the thread's unit of tile j, from the LDS slot its own wave
  // filled; the group's table in registers as byte planes, the next one loaded
  const uint16_t* lutrow = reinterpret_cast<const uint16_t*>(lut) + grow * (int64_t)gpr * 16;
  mm::Planes16 P;
  uint32_t Ln[8];
  uint32_t cur_g = 0xFFFFFFFFu;
  auto load_tab = [&](uint32_t g) {
    const u32x4* tp = reinterpret_cast<const u32x4*>(lutrow + g * 16u);
    const u32x4 a = tp[0], b = tp[1];
    Ln[0] = a.x; Ln[1] = a.y; Ln[2] = a.z; Ln[3] = a.w;
    Ln[4] = b.x; Ln[5] = b.y; Ln[6] = b.z; Ln[7] = b.w;
  };
  uint32_t bst[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) bst[q] = XL_B + swz128((uint32_t)(t >> 1), 4u * (uint32_t)(t & 1) + q);
  const uint32_t isl = XL_I + 16u * (uint32_t)t;
  auto stage = [&](int j, uint32_t buf) __attribute__((always_inline)) {
    const u32x4 w = mm::ld_q(isl + buf * 8192u);
    const uint32_t g = group_of(j);
    if (g != cur_g) {
      mm::planes16(Ln, P);
      cur_g = g;
      load_tab(g + 1 < (uint32_t)gpr ? g + 1 : g);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) mm::st_q(bst[q] + buf * B64_TILE, mm::dequant8_b4(w[q], P));
  };

  // ---- matrix state (as in k_gemm_fwd64)
  const int wm = wave & 1, wn = wave >> 1;
  const uint32_t arow = (uint32_t)(128 * wm + (lane & 31));
  const uint32_t brow = (uint32_t)(64 * wn + (lane & 31));
  const uint32_t khalf = (uint32_t)(lane >> 5);
  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) mm::zero16(acc[i][jj]);
  uint32_t ard[4], brd[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    ard[ks] = XL_A + swz128(arow, (uint32_t)(2 * ks) + khalf);
    brd[ks] = XL_B + swz128(brow, (uint32_t)(2 * ks) + khalf);
  }
  // the four quarters of a step, each one's reads between the MFMAs of the one
  // before it
  auto mfma_step = [&](uint32_t buf) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
    u32x4 fa[4][4], fb[4][2];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[ks][i] = mm::ld_q(ard[ks] + buf * A64_TILE + 4096u * i);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) fb[ks][jj] = mm::ld_q(brd[ks] + buf * B64_TILE + 4096u * jj);
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
          acc[i][jj] = EP::SWAP ? MF::run(fb[ks][jj], fa[ks][i], acc[i][jj])
                                : MF::run(fa[ks][i], fb[ks][jj], acc[i][jj]);
    __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
    for (int ks = 1; ks < 4; ++ks) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };
  const bool mfma_first = wave < 4;

  // ---- prologue: tile 0's activations and indices, tile 1's indices
  load_tab(group_of(0));
#pragma unroll
  for (int c = 0; c < 4; ++c) dd_dma16_free(xs[c], adst + 1024u * c);
  dd_dma16_free(is, idst);
  if (KS > 1) dd_dma16_free(is + 32, idst + 8192u);
  dd_wait_vmcnt<0>();
  __syncthreads();
  stage(0, 0u);
  __syncthreads();

  // step k: multiplies buffer k & 1, stages tile k + 1 into the other. LAST:
  // fewer than two tiles follow
  auto step = [&](int k, uint32_t buf, auto last) __attribute__((always_inline)) {
    constexpr bool LAST = decltype(last)::value;
    const bool more = !LAST || k + 1 < KS;  // uniform
    if (more) {
#pragma unroll
      for (int c = 0; c < 4; ++c) copy(k, buf ^ 1u, c);
    }
    if constexpr (!LAST) copy(k, buf ^ 1u, 4);
    if (!mfma_first && more) stage(k + 1, buf ^ 1u);
    __builtin_amdgcn_sched_barrier(0);
    mfma_step(buf);
    if (mfma_first && more) stage(k + 1, buf ^ 1u);
    dd_wait_vmcnt<0>();  // this wave's copies of step k + 1 and indices of step k + 2 are in LDS
    __syncthreads();
  };
  int k = 0;
  for (; k + 3 < KS; k += 2) {
    step(k, 0u, bool_tag<false>{});
    step(k + 1, 1u, bool_tag<false>{});
  }
  if (k + 2 < KS) {
    step(k, 0u, bool_tag<false>{});
    ++k;
  }
  for (; k < KS; ++k) step(k, (uint32_t)(k & 1), bool_tag<true>{});
  EP::template run<SC>(acc, ep, rexp, m, n, m0, n0, wm, wn, lane, t);
}

template <typename TL, typename EP, bool SC>
hipError_t xent_logits_launch(const XentGemm& g, const typename EP::Args& ep, hipStream_t s) {
  const auto kern = k_xent_logits<TL, EP, SC>;
  static const hipError_t prep = prepare_kernel((const void*)kern, XL_LDS);
  if (prep != hipSuccess) return prep;
  const int64_t mb = (g.p.m + 255) / 256, nb = (g.p.n + 255) / 256;
  const uint32_t ug = (uint32_t)(g.p.group_cols() / 32);
  const uint32_t magic = ug == 1 ? 0u : (uint32_t)((((uint64_t)1) << 32) / ug + 1);
  hipLaunchKernelGGL(kern, dim3((unsigned)(mb * nb)), dim3(512), XL_LDS, s, (const TL*)g.Xp, g.idx, (const TL*)g.lut,
                     g.p.n, g.p.d, g.p.gpr, magic, ep, g.rexp);
  return hipGetLastError();
}

}  // namespace

}  // namespace skm
