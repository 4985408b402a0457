// Grouped product of E4M3 operands with one scale per block of 128 (fp8.hip).
#pragma once

#include "grouped.h"
#include "grouped_ops.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// C tile BM x BN by WM x WN waves; k tiles of one block (128 codes, one line of
// a row). The matrix instruction is 16x16x128: it sums a whole block into 4
// registers per lane (row l & 15 of the rows' fragment, columns 4 (l >> 4) .. +
// 3), which 4 FMAs then scale into the running sum; with 32x32x64 a block is two
// instructions and 16 registers, and a 128 x 64 wave tile's sums, fragments and
// those temporaries do not fit 256 registers.
//
// A wave holds the block's TN weight fragments and streams its TM row
// fragments: while fragment m is multiplied, m + 1 is read from LDS and the
// sums of m - 1 are scaled and added. The one barrier of a k tile sits before
// its last row fragment: past it the next tile has landed, nobody reads this
// tile's stage, and the tile after the next is loaded there.
template <int BM, int BN, int WM, int WN, int OCC>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_fp8_kernel(const Fp8Args P) {
  constexpr int NT = 64 * WM * WN;
  constexpr int WTN = BN / WN, TN = WTN / 16;
  static_assert(128 % WTN == 0, "a wave's columns lie in one weight block");
  __shared__ u32x4 sa0[BM * 8], sb0[BN * 8], sa1[BM * 8], sb1[BN * 8];
  __shared__ float sc0[BM], sc1[BM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave % WM, wave_n = wave / WM;

  int valid, t;
  TileRec rec;
  if (P.tiles != nullptr) {
    valid = *P.n_mtiles * P.ntiles;
    if ((int)blockIdx.x >= valid) return;
    t = xcd_remap(blockIdx.x, valid);
    rec = P.tiles[t / P.ntiles];
  } else {
    const OffsetScan scan(P.offsets, P.E, (int)P.R, lane);
    const int grid = (int)gridDim.x - P.rest_blocks;
    if ((int)blockIdx.x >= grid) {
      const int2 c = scan.covered();
      zero_rest(P.C, P.ldc, P.N, c.x, c.y, (int)P.R, (int)blockIdx.x - grid, P.rest_blocks, NT);
      return;
    }
    int incl;
    valid = scan.tiles(BM, incl) * P.ntiles;
    if ((int)blockIdx.x >= valid) return;
    t = xcd_remap(blockIdx.x, valid);
    rec = scan.find(BM, t / P.ntiles, incl);
  }
  const int e = __builtin_amdgcn_readfirstlane(rec.x), first = __builtin_amdgcn_readfirstlane(rec.y);
  const int lo = __builtin_amdgcn_readfirstlane(rec.z), hi = __builtin_amdgcn_readfirstlane(rec.w);
  int mt, nt;
  grouped_tile_order(t - first * P.ntiles, (hi - lo + BM - 1) / BM, (hi - lo) / BM, P.ntiles, 8, mt, nt);
  const int m0 = __builtin_amdgcn_readfirstlane(lo + mt * BM), n0 = __builtin_amdgcn_readfirstlane(nt * BN);
  const int K2 = P.K / 2;                              // the loads count pairs of codes

  // HQ: the tile's height in quarters of BM (an expert's short last tile)
  auto body = [&](auto height) __attribute__((always_inline)) {
    constexpr int HQ = decltype(height)::value;
    constexpr int H = BM * HQ / 4, WTM = H / WM, TM = WTM / 16;
    static_assert(TM >= 1 && H * 8 % NT == 0, "wave tile");
    OperandLoad<H, false, NT> la;
    OperandLoad<BN, false, NT> lb;
    la.init(reinterpret_cast<const uint16_t*>(P.A + (int64_t)m0 * P.K), K2, hi - m0, K2, wave, lane);
    lb.init(reinterpret_cast<const uint16_t*>(P.B + ((int64_t)e * P.N + n0) * P.K), K2, P.N - n0, K2, wave, lane);

    // a k tile's row scales: one dword per lane, 64 rows a wave (waves beyond
    // the tile's rows repeat others'); rows past the end repeat the last one
    constexpr int SW = H / 64;
    const int srow = (wave % SW) * 64;
    const uint32_t sofs = (uint32_t)min(srow + lane, hi - 1 - m0) * 4;
    auto issue_scales = [&](float* st, int kt) {
      const bool live = kt < P.kb;
      const __amdgpu_buffer_rsrc_t r =
          make_rsrc(uniform_ptr(reinterpret_cast<const uint16_t*>(P.sx + (live ? (int64_t)kt * P.R : 0) + m0)),
                    live ? kRsrc2G : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&st[srow], 4, (int)sofs, 0, 0, 0);
    };
    // the wave's weight scales, 64 blocks at a time in one register
    const float* sw = P.sw + ((int64_t)e * P.nb + min((n0 + wave_n * WTN) / 128, P.nb - 1)) * P.kb;
    float swv = sw[min(lane, P.kb - 1)];

    f32x4 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    // lane l's 32 codes of fragment row l & 15: chunks 4 (g >> 1) + (g & 1) and
    // that + 2 of the block, g = l >> 4 (both operands alike, so the order of k is
    // free; chunks 2 g and 2 g + 1 left the lanes a 16-byte read serves together
    // two to a bank: 46 % of the LDS cycles were conflicts). Fragments start at
    // multiples of 16 rows, so one swizzle serves them all and they differ by
    // constant offsets.
    const int r16 = lane & 15, swz = r16 >> 1, kc = 4 * (lane >> 5) + ((lane >> 4) & 1);
    const int c0 = r16 * 8 + (kc ^ swz), c1 = r16 * 8 + ((kc + 2) ^ swz);
    const int a0 = wave_m * WTM * 8, b0 = wave_n * WTN * 8;
    const int a_c0 = a0 + c0, a_c1 = a0 + c1, b_c0 = b0 + c0, b_c1 = b0 + c1;
    auto frag = [&](const u32x4* p0, const u32x4* p1, int row) {
      const u32x4 u = p0[row * 8], v = p1[row * 8];
      return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
    auto frag_a = [&](const u32x4* stage, int m) { return frag(stage + a_c0, stage + a_c1, m * 16); };
    auto frag_b = [&](const u32x4* stage, int n) { return frag(stage + b_c0, stage + b_c1, n * 16); };

    i32x8 fb[TN], fa;
    f32x4 z[TN];                      // the sums of the row fragment before, not yet scaled
    float zs = 0.f;
#pragma unroll
    for (int n = 0; n < TN; ++n) z[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int kt, u32x4* a, u32x4* b, float* sc, u32x4* a1, u32x4* b1) {
      if (kt > 0 && (kt & 63) == 0) swv = sw[min(kt + lane, P.kb - 1)];
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(swv), kt & 63));
      float s[TM];
#pragma unroll
      for (int m = 0; m < TM; ++m) s[m] = sc[wave_m * WTM + m * 16 + r16] * w;
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        i32x8 fn, fbn[TN];
        if (m + 1 < TM) {
          fn = frag_a(a, m + 1);
        } else {
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          la.issue(a, kt + 2, wave);
          lb.issue(b, kt + 2, wave);
          issue_scales(sc, kt + 2);
          fn = frag_a(a1, 0);
#pragma unroll
          for (int n = 0; n < TN; ++n) fbn[n] = frag_b(b1, n);
        }
        f32x4 zn[TN];
#pragma unroll
        for (int n = 0; n < TN; ++n)
          zn[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[n], fa, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                                  0x7F7F7F7F, 0, 0x7F7F7F7F);
        // (the first fragment adds the last one's of the tile before)
        f32x4(&dst)[TN] = acc[m == 0 ? TM - 1 : m - 1];
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) dst[n][q] = fmaf(z[n][q], zs, dst[n][q]);
        // (pinned here: the compiler otherwise keeps every fragment's z until
        // the end of the tile, and spills)
#pragma unroll
        for (int n = 0; n < TN; ++n) asm volatile("" : "+v"(dst[n]));
#pragma unroll
        for (int n = 0; n < TN; ++n) z[n] = zn[n];
        zs = s[m];
        fa = fn;
        if (m + 1 == TM) {
#pragma unroll
          for (int n = 0; n < TN; ++n) fb[n] = fbn[n];
        }
        __builtin_amdgcn_sched_barrier(0);   // (left to itself the scheduler reads every fragment first, and spills)
      }
    };
    constexpr int NL = OperandLoad<H, false, NT>::NL + OperandLoad<BN, false, NT>::NL + 1;
    la.issue(sa0, 0, wave);
    lb.issue(sb0, 0, wave);
    issue_scales(sc0, 0);
    la.issue(sa1, 1, wave);
    lb.issue(sb1, 1, wave);
    issue_scales(sc1, 1);
    MOE_WAIT_VMCNT(NL);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    fa = frag_a(sa0, 0);
#pragma unroll
    for (int n = 0; n < TN; ++n) fb[n] = frag_b(sb0, n);
    int kt = 0;
    for (; kt + 1 < P.kb; kt += 2) {
      step(kt, sa0, sb0, sc0, sa1, sb1);
      step(kt + 1, sa1, sb1, sc1, sa0, sb0);
    }
    if (kt < P.kb) step(kt, sa0, sb0, sc0, sa1, sb1);
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[TM - 1][n][q] = fmaf(z[n][q], zs, acc[TM - 1][n][q]);
    MOE_WAIT_VMCNT(0);
    __syncthreads();

    // through LDS to whole rows of the wave tile, as store_wave_tile
    constexpr int per = BM * 8 * 16 / 16384, CPW = WTN / 8, RPI = 64 / CPW, NRB = WTM / RPI;
    static_assert(WM * WN <= 4 * per && WTM * WTN * 2 <= 16384, "staging areas");
    const int h = wave / per;
    char* stg = reinterpret_cast<char*>(h == 0 ? sa0 : h == 1 ? sb0 : h == 2 ? sa1 : sb1) + (wave % per) * 16384;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int r = m * 16 + r16;
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const int c = n * 2 + (lane >> 5);
        *reinterpret_cast<u32x2*>(stg + r * (CPW * 16) + ((c ^ (r % CPW)) * 16) + ((lane >> 4) & 1) * 8) =
            u32x2{cvt_pk_bf16(acc[m][n][0], acc[m][n][1]), cvt_pk_bf16(acc[m][n][2], acc[m][n][3])};
      }
    }
    const int r0 = lane / CPW, c = lane % CPW;
    u32x4 rb[NRB];
#pragma unroll
    for (int i = 0; i < NRB; ++i) {
      const int r = i * RPI + r0;
      rb[i] = *reinterpret_cast<const u32x4*>(stg + r * (CPW * 16) + ((c ^ (r % CPW)) * 16));
    }
    const int mw = m0 + wave_m * WTM, nw = n0 + wave_n * WTN;
    if (nw + c * 8 < P.N) {
      uint16_t* out = P.C + (int64_t)(mw + r0) * P.ldc + nw + c * 8;
#pragma unroll
      for (int i = 0; i < NRB; ++i, out += RPI * P.ldc)
        if (mw + i * RPI + r0 < hi) *reinterpret_cast<u32x4*>(out) = rb[i];
    }
  };
  if constexpr (BM == 256) {
    const int rows = hi - m0;
    if (rows <= 64) { body(Stage<1>{}); return; }
    if (rows <= 128) { body(Stage<2>{}); return; }
    if (rows <= 192) { body(Stage<3>{}); return; }
  }
  body(Stage<4>{});
}

}  // namespace moe
