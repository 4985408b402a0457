// Grouped product of E4M3 operands with one scale per block of 128 (fp8.hip).
#pragma once

#include "grouped.h"
#include "grouped_ops.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// exponent e of the block scale 2^e: the least with amax <= 448 * 2^e, not below
// -126 (the scale stays a normal number). 448 = 0.875 * 2^9. A power of two loses
// nothing against amax / 448 (E4M3's precision is relative; a block gives up at
// most one bit of its range), and scaling by it is exact, so the codes are the
// definition's own, with one rounding each.
__device__ __forceinline__ int fp8_block_exponent(float amax) {
  if (!(amax > 0.f)) return -126;
  const int ex = __builtin_amdgcn_frexp_expf(amax);
  const float mant = __builtin_amdgcn_frexp_mantf(amax);
  return max(mant > 0.875f ? ex - 8 : ex - 9, -126);
}

// Four values of magnitude at most 448 as E4M3 codes (round to nearest even);
// a value that is not finite becomes the NaN code.
__device__ __forceinline__ uint32_t fp8_pack4(const float (&v)[4]) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  uint32_t u = (uint32_t)w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(fabsf(v[i]) <= 448.f)) u |= 0x7Fu << (8 * i);
  return u;
}

__device__ __forceinline__ float finite_abs(uint32_t bf16_bits) {
  const uint32_t a = bf16_bits & 0x7FFFu;
  return a < 0x7F80u ? __uint_as_float(a << 16) : 0.f;
}

// max |v| over the finite values of 8 bf16
__device__ __forceinline__ float amax8(const u32x4 w) {
  float a = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) a = fmaxf(a, fmaxf(finite_abs(w[q] & 0xFFFFu), finite_abs(w[q] >> 16)));
  return a;
}

__device__ __forceinline__ u32x2 codes8(const u32x4 w, float inv) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float v[4] = {bf16_bits_to_f32(w[2 * h] & 0xFFFFu) * inv, bf16_bits_to_f32(w[2 * h] >> 16) * inv,
                        bf16_bits_to_f32(w[2 * h + 1] & 0xFFFFu) * inv, bf16_bits_to_f32(w[2 * h + 1] >> 16) * inv};
    o[h] = fp8_pack4(v);
  }
  return o;
}

// Block b of a row, 16 lanes with 8 values each.
__device__ __forceinline__ u32x4 load_block(const uint16_t* row, int b, int K) {
  const int k = b * 128 + (threadIdx.x & 15) * 8;
  return k < K ? *reinterpret_cast<const u32x4*>(row + k) : u32x4{0u, 0u, 0u, 0u};
}
// Its codes and its scale. The 16 lanes are together.
__device__ __forceinline__ void quantise_block(const u32x4 w, uint8_t* row, int b, int K, float* scale) {
  const int k = b * 128 + (threadIdx.x & 15) * 8;
  float a = amax8(w);
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) a = fmaxf(a, __shfl_xor(a, m, kWave));
  const int e = fp8_block_exponent(a);
  if (k < K) *reinterpret_cast<u32x2*>(row + k) = codes8(w, __builtin_ldexpf(1.f, -e));
  if ((threadIdx.x & 15) == 0) *scale = __builtin_ldexpf(1.f, e);
}

// s_waitcnt vmcnt(n) lgkmcnt(0), and lgkmcnt(0) alone
constexpr int wait_lgkm0(int n) { return (n & 0xF) | (0x7 << 4) | (((n >> 4) & 3) << 14); }
constexpr int kWaitLgkm0 = 0xF | (0x7 << 4) | (3 << 14);

// C tile BM x BN by WM x WN waves; k tiles of one block (128 codes, one line of
// a row). The matrix instruction is 16x16x128: it sums a whole block into 4
// registers per lane (row l & 15 of the rows' fragment, columns 4 (l >> 4) .. +
// 3), which 4 FMAs then scale into the running sum; with 32x32x64 a block is two
// instructions and 16 registers, and a 128 x 64 wave tile's sums, fragments and
// those temporaries do not fit 256 registers.
//
// A wave holds the block's TN weight fragments and streams its TM row
// fragments: while fragment m is multiplied, m + 1 is read from LDS and the
// sums of m - 1 are scaled and added.
//
// What bounds it is the loads' latency (without them, on stale data, a k tile
// took 1.29 us against 1.96): two stages of 64 KB fill the LDS, so each part of
// a stage is loaded again as soon as it is free, not a whole stage at a time. A
// k tile has two barriers. By the first, half way, its weight fragments (read
// into registers before the tile began) and the first half of every wave's row
// fragments are done with: those parts of the tile after the next are loaded.
// Past the second, before the last row fragment, the second halves and the
// scales follow, and the next tile's first fragments are read. Every load of
// codes then has one and a half k tiles to land, and each barrier waits only
// for what is read next.
template <int BM, int BN, int WM, int WN, int OCC, int OUT>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_fp8_kernel(const Fp8Args P) {
  constexpr int NT = 64 * WM * WN;
  constexpr int WTN = BN / WN, TN = WTN / 16;
  static_assert(128 % WTN == 0, "a wave's columns lie in one weight block");
  // (the halves of the row stages are arrays of their own: the compiler waits for
  // every load into an array before it reads from it)
  constexpr int AH = BM * 8 / NT > 1 ? BM * 4 : BM * 8;   // chunks of a row stage's array: half, or all of it
  constexpr int AHH = BM * 8 / NT > 1 ? BM * 4 : 1;
  __shared__ u32x4 sa0[AH], sa0h[AHH], sb0[BN * 8], sa1[AH], sa1h[AHH], sb1[BN * 8];
  __shared__ float sc0[BM < 64 ? 64 : BM], sc1[BM < 64 ? 64 : BM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave % WM, wave_n = wave / WM;

  // a split reduction: piece s of ksplit sums klen codes (blocks of 128) into C + s * c_stride (fp32)
  int block = blockIdx.x, nblocks = gridDim.x, kt0 = 0, kb = P.kb;
  int64_t c_base = 0;
  if (P.ksplit > 1) {
    nblocks /= P.ksplit;
    const int piece = block / nblocks;
    block -= piece * nblocks;
    kt0 = piece * P.klen;
    kb = min(P.klen, P.kb - kt0);
    c_base = piece * P.c_stride;
  }
  TilePart tp;
  TileRec rec;
  if (P.tiles != nullptr) {
    if (!tp.pick<BM>(block, *P.n_mtiles * P.ntiles, nblocks, 0)) return;
    rec = P.tiles[tp.t / P.ntiles];
  } else {
    const bool mine = with_scan(P.offsets, P.E, (int)P.R, lane, [&](const auto& scan) {
      const int grid = nblocks - P.rest_blocks;
      if (block >= grid) {
        const int2 c = scan.covered();
        zero_rest(static_cast<uint16_t*>(P.C), P.ldc, P.N, c.x, c.y, (int)P.R, block - grid, P.rest_blocks, NT);
        return false;
      }
      int incl;
      if (!tp.pick<BM>(block, scan.tiles(BM, incl) * P.ntiles, grid, 0)) return false;
      rec = scan.find(BM, tp.t / P.ntiles, incl);
      return true;
    });
    if (!mine) return;
  }
  const int e = __builtin_amdgcn_readfirstlane(rec.x), first = __builtin_amdgcn_readfirstlane(rec.y);
  const int lo = __builtin_amdgcn_readfirstlane(rec.z);
  int hi = __builtin_amdgcn_readfirstlane(rec.w), mt, nt;
  grouped_tile_order(tp.t - first * P.ntiles, (hi - lo + BM - 1) / BM, (hi - lo) / BM, P.ntiles, 8, mt, nt);
  const int n0 = __builtin_amdgcn_readfirstlane(nt * BN);
  int m0 = __builtin_amdgcn_readfirstlane(lo + mt * BM);
  if constexpr (BM == 256) {
    if (!tp.rows(BM, m0, hi)) return;
  }
  if constexpr (BM == 32) {
    if (P.x != nullptr) {
      // Few rows, quantised here: every workgroup makes the codes and scales that
      // it reads itself (those of other column tiles store the same bytes), and
      // no launch comes before this one. Four blocks a 16 lanes at a time, their
      // loads together.
      constexpr int NG = NT / 16;
      const int n = min(hi - m0, BM) * kb;
      for (int i = tid / 16; i < n; i += 4 * NG) {
        u32x4 w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = min(i + q * NG, n - 1), r = j / kb;
          w[q] = load_block(P.x + (int64_t)(m0 + r) * P.ldx, kt0 + j - r * kb, P.K);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = min(i + q * NG, n - 1), r = j / kb, b = kt0 + j - r * kb;
          quantise_block(w[q], const_cast<uint8_t*>(P.A) + (int64_t)(m0 + r) * P.K, b, P.K,
                         const_cast<float*>(P.sx) + (int64_t)b * P.R + m0 + r);
        }
      }
      __threadfence_block();
      __syncthreads();
    }
  }
  const int ld2 = P.K / 2, K2 = min(P.K - kt0 * 128, kb * 128) / 2;   // the loads count pairs of codes

  // HQ: the tile's height in quarters of BM (1, 2 or 4: an expert's last tile may be short)
  auto body = [&](auto height) __attribute__((always_inline)) {
    constexpr int HQ = decltype(height)::value;
    constexpr int H = BM * HQ / 4, WTM = H / WM, TM = WTM / 16;
    static_assert(TM >= 2 && TM % 2 == 0 && H * 8 % NT == 0, "wave tile");
    // (few rows are one load a thread: they go whole, at the second barrier)
    constexpr bool HALVES = H * 8 / NT > 1;
    constexpr int HR = HALVES ? H / 2 : H;            // rows of a row stage array
    typedef OperandLoad<HR, false, NT, HALVES ? WTM / 2 : 0> LoadA;
    constexpr int NA = LoadA::NL, NB = BN * 8 / NT;
    LoadA la, lah;
    OperandLoad<BN, false, NT> lb;
    const uint16_t* rows8 = reinterpret_cast<const uint16_t*>(P.A + (int64_t)m0 * P.K + kt0 * 128);
    la.init(rows8, ld2, hi - m0, K2, wave, lane);
    if constexpr (HALVES) lah.init(rows8, ld2, hi - m0, K2, wave, lane, WTM / 2);
    lb.init(reinterpret_cast<const uint16_t*>(P.B + ((int64_t)e * P.N + n0) * P.K + kt0 * 128), ld2, P.N - n0, K2, wave,
            lane);

    // a k tile's row scales: one dword per lane, 64 rows a wave (waves beyond
    // the tile's rows repeat others'); rows past the end repeat the last one
    constexpr int SW = H < 64 ? 1 : H / 64;
    const int srow = (wave % SW) * 64;
    const uint32_t sofs = (uint32_t)min(srow + lane, hi - 1 - m0) * 4;
    auto issue_scales = [&](float* st, int kt) {
      const bool live = kt < kb;
      const __amdgpu_buffer_rsrc_t r =
          make_rsrc(uniform_ptr(reinterpret_cast<const uint16_t*>(P.sx + (int64_t)(kt0 + (live ? kt : 0)) * P.R + m0)),
                    live ? kRsrc2G : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&st[srow], 4, (int)sofs, 0, 0, 0);
    };
    // the wave's weight scales, one a k tile (scalar loads, through the constant address space)
    typedef const __attribute__((address_space(4))) float* scale_ptr;
    const scale_ptr sw = (scale_ptr)(uintptr_t)uniform_ptr(reinterpret_cast<const uint16_t*>(
        P.sw + ((int64_t)e * P.nb + min((n0 + wave_n * WTN) / 128, P.nb - 1)) * P.kb + kt0));

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
    const int a0 = wave_m * (HALVES ? WTM / 2 : WTM) * 8, b0 = wave_n * WTN * 8;
    const int a_c0 = a0 + c0, a_c1 = a0 + c1, b_c0 = b0 + c0, b_c1 = b0 + c1;
    auto frag = [&](const u32x4* p0, const u32x4* p1, int row) {
      const u32x4 u = p0[row * 8], v = p1[row * 8];
      return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
    auto frag_a = [&](const u32x4* lo, const u32x4* hi, int m) {
      const u32x4* p = HALVES && m >= TM / 2 ? hi : lo;
      return frag(p + a_c0, p + a_c1, (HALVES && m >= TM / 2 ? m - TM / 2 : m) * 16);
    };
    auto frag_b = [&](const u32x4* stage, int n) { return frag(stage + b_c0, stage + b_c1, n * 16); };

    i32x8 fb[TN], fa;
    f32x4 z[TN];                      // the sums of the row fragment before, not yet scaled
    float w = sw[0];
    float zs = 0.f, sv;               // their rows' scale times the weights'; the current fragment's row scale
#pragma unroll
    for (int n = 0; n < TN; ++n) z[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int srow0 = wave_m * WTM + r16;
    auto step = [&](int kt, u32x4* a, u32x4* ah, u32x4* b, float* sc, u32x4* a1, u32x4* b1, float* sc1) {
      float wn;
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        i32x8 fn;
        float sn;
        if (m == TM / 2) wn = sw[min(kt + 1, kb - 1)];
        if (m + 1 == TM / 2) {
          // (unsplit rows: the last barrier waited for the whole tile)
          __builtin_amdgcn_s_waitcnt(HALVES ? wait_lgkm0(NB + 2 * NA + 1) : kWaitLgkm0);
          asm volatile("s_barrier" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          lb.issue(b, kt + 2, wave);
          if constexpr (HALVES) la.issue(a, kt + 2, wave);
        }
        if (m + 1 < TM) {
          fn = frag_a(a, ah, m + 1);
          sn = sc[srow0 + (m + 1) * 16];
        } else {
          __builtin_amdgcn_s_waitcnt(wait_lgkm0(NB + (HALVES ? 2 * NA : 0)));
          asm volatile("s_barrier" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          issue_scales(sc, kt + 2);
          if constexpr (HALVES) lah.issue(ah, kt + 2, wave);
          else la.issue(a, kt + 2, wave);
          fn = frag_a(a1, a1, 0);
          sn = sc1[srow0];
        }
        // one matrix instruction, then the scaling of the sums it replaces (of the
        // row fragment before; the tile's first fragment finishes the last one of
        // the tile before). Pinned in this order: left to itself the compiler
        // keeps more sums and fragments alive than there are registers.
        f32x4(&dst)[TN] = acc[m == 0 ? TM - 1 : m - 1];
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          const f32x4 zn = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fb[n], fa, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
          if (m + 1 == TM) fb[n] = frag_b(b1, n);      // the next tile's, in the place of the one just used
#pragma unroll
          for (int q = 0; q < 4; ++q) dst[n][q] = fmaf(z[n][q], zs, dst[n][q]);
          asm volatile("" : "+v"(dst[n]));
          z[n] = zn;
          __builtin_amdgcn_sched_barrier(0);
        }
        zs = sv * w;
        sv = sn;
        if (m + 1 == TM) w = wn;
        fa = fn;
      }
    };
    // in the order of the steps: what the second barrier of the step before waits
    // for, then what later ones do
    auto start = [&](int kt, u32x4* a, u32x4* ah, u32x4* b, float* sc) {
      lb.issue(b, kt, wave);
      if constexpr (HALVES) la.issue(a, kt, wave);
      issue_scales(sc, kt);
      if constexpr (HALVES) lah.issue(ah, kt, wave);
      else la.issue(a, kt, wave);
    };
    start(0, sa0, sa0h, sb0, sc0);
    start(1, sa1, sa1h, sb1, sc1);
    MOE_WAIT_VMCNT(NB + 1 + (HALVES ? 3 * NA : NA));
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    fa = frag_a(sa0, sa0, 0);
    sv = sc0[srow0];
#pragma unroll
    for (int n = 0; n < TN; ++n) fb[n] = frag_b(sb0, n);
    int kt = 0;
    for (; kt + 1 < kb; kt += 2) {
      step(kt, sa0, sa0h, sb0, sc0, sa1, sb1, sc1);
      step(kt + 1, sa1, sa1h, sb1, sc1, sa0, sb0, sc0);
    }
    if (kt < kb) step(kt, sa0, sa0h, sb0, sc0, sa1, sb1, sc1);
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[TM - 1][n][q] = fmaf(z[n][q], zs, acc[TM - 1][n][q]);
    MOE_WAIT_VMCNT(0);
    __syncthreads();

    if constexpr (OUT == EPI_F32) {
      // pieces: straight from the registers (16 bytes of 16 rows a store; few and small)
      float* out = static_cast<float*>(P.C) + c_base;
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int row = m0 + wave_m * WTM + m * 16 + r16;
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          const int col = n0 + wave_n * WTN + n * 16 + 4 * (lane >> 4);
          if (row < hi && col < P.N) *reinterpret_cast<f32x4*>(out + (int64_t)row * P.ldc + col) = acc[m][n];
        }
      }
      return;
    }
    // through LDS to whole rows of the wave tile, as store_wave_tile
    constexpr int CPW = WTN / 8, RPI = 64 / CPW, NRB = WTM / RPI, SB = WTM * WTN * 2;
    constexpr int APER = std::max(1, AH * 16 / SB), BPER = BN * 128 / SB;   // wave tiles in a row array, in a weight stage
    static_assert(WM * WN <= 2 * BPER || (AH * 16 >= SB && WM * WN <= 4 * APER + 2 * BPER), "staging areas");
    u32x4* const area = wave < BPER                 ? sb0
                        : wave < 2 * BPER            ? sb1
                        : wave < 2 * BPER + APER     ? sa0
                        : wave < 2 * BPER + 2 * APER ? sa0h
                        : wave < 2 * BPER + 3 * APER ? sa1
                                                     : sa1h;
    char* stg = reinterpret_cast<char*>(area) +
                (wave < 2 * BPER ? wave % BPER : (wave - 2 * BPER) % APER) * SB;
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
      uint16_t* out = static_cast<uint16_t*>(P.C) + (int64_t)(mw + r0) * P.ldc + nw + c * 8;
#pragma unroll
      for (int i = 0; i < NRB; ++i, out += RPI * P.ldc)
        if (mw + i * RPI + r0 < hi) *reinterpret_cast<u32x4*>(out) = rb[i];
    }
  };
  if constexpr (BM == 256) {
    const int rows = hi - m0;
    if (rows <= 64) { body(Stage<1>{}); return; }
    if (rows <= 128) { body(Stage<2>{}); return; }
  }
  body(Stage<4>{});
}

}  // namespace moe
