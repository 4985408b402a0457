// Grouped product of E4M3 operands with one scale per block of 128 (fp8.hip).
#pragma once

#include "grouped.h"
#include "grouped_ops.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int BM, int BN, int WM, int WN, int OCC>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_fp8_kernel(const Fp8Args P) {
  constexpr int NT = 64 * WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  static_assert(TM >= 1 && TN >= 1 && 128 % WTN == 0, "tile shape");
  __shared__ u32x4 sa0[BM * 8], sb0[BN * 8], sa1[BM * 8], sb1[BN * 8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave % WM, wave_n = wave / WM;

  const int valid = *P.n_mtiles * P.ntiles;
  if ((int)blockIdx.x >= valid) return;
  const int t = xcd_remap(blockIdx.x, valid);
  const TileRec rec = P.tiles[t / P.ntiles];
  const int e = __builtin_amdgcn_readfirstlane(rec.x), first = __builtin_amdgcn_readfirstlane(rec.y);
  const int lo = __builtin_amdgcn_readfirstlane(rec.z), hi = __builtin_amdgcn_readfirstlane(rec.w);
  int mt, nt;
  grouped_tile_order(t - first * P.ntiles, (hi - lo + BM - 1) / BM, (hi - lo) / BM, P.ntiles, 1 << 20, mt, nt);
  const int m0 = __builtin_amdgcn_readfirstlane(lo + mt * BM), n0 = __builtin_amdgcn_readfirstlane(nt * BN);
  const int K2 = P.K / 2;                              // the loads count pairs of codes
  OperandLoad<BM, false, NT> la;
  OperandLoad<BN, false, NT> lb;
  la.init(reinterpret_cast<const uint16_t*>(P.A + (int64_t)m0 * P.K), K2, hi - m0, K2, wave, lane);
  lb.init(reinterpret_cast<const uint16_t*>(P.B + ((int64_t)e * P.N + n0) * P.K), K2, P.N - n0, K2, wave, lane);

  // the row scales of the lane's rows (rows past the end repeat the last one)
  const float* sx[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) sx[tm] = P.sx + min(m0 + wave_m * WTM + tm * 32 + (lane & 31), hi - 1);
  // the wave's columns lie in one block of 128
  const int nblk = min((n0 + wave_n * WTN) / 128, P.nb - 1);
  const float* sw = P.sw + ((int64_t)e * P.nb + nblk) * P.kb;

  f32x16 acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[a][b][q] = 0.f;

  const int swz = ((lane & 31) >> 1) & 7, half = lane >> 5;
  auto frag = [&](const u32x4* stage, int row, int s) {
    // k order inside the block is the same for both operands: chunks 4 s + 2 half, + 1
    const u32x4 c0 = stage[row * 8 + ((4 * s + 2 * half) ^ swz)], c1 = stage[row * 8 + ((4 * s + 2 * half + 1) ^ swz)];
    return i32x8{(int)c0.x, (int)c0.y, (int)c0.z, (int)c0.w, (int)c1.x, (int)c1.y, (int)c1.z, (int)c1.w};
  };
  auto step = [&](int kt, const u32x4* a, const u32x4* b, u32x4* an, u32x4* bn) {
    float s[TM];
    const float w = sw[kt];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) s[tm] = sx[tm][(int64_t)kt * P.R] * w;
    la.issue(an, kt + 1, wave);
    lb.issue(bn, kt + 1, wave);
    i32x8 fa[2][TM], fb[2][TN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) fa[h][tm] = frag(a, wave_m * WTM + tm * 32 + (lane & 31), h);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) fb[h][tn] = frag(b, wave_n * WTN + tn * 32 + (lane & 31), h);
    }
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        f32x16 z = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[0][tn], fa[0][tm], z, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
        z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[1][tn], fa[1][tm], z, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[tn][tm][q] = fmaf(z[q], s[tm], acc[tn][tm][q]);
      }
    MOE_WAIT_VMCNT(0);
    __syncthreads();
  };
  la.issue(sa0, 0, wave);
  lb.issue(sb0, 0, wave);
  MOE_WAIT_VMCNT(0);
  __syncthreads();
  for (int kt = 0; kt < P.kb; kt += 2) {
    step(kt, sa0, sb0, sa1, sb1);
    if (kt + 1 < P.kb) step(kt + 1, sa1, sb1, sa0, sb0);
  }

#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int m = m0 + wave_m * WTM + tm * 32 + (lane & 31);
    if (m >= hi) continue;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wave_n * WTN + tn * 32 + 8 * g + 4 * half;
        if (n >= P.N) continue;
        *reinterpret_cast<u32x2*>(P.C + (int64_t)m * P.ldc + n) =
            u32x2{cvt_pk_bf16(acc[tn][tm][4 * g], acc[tn][tm][4 * g + 1]),
                  cvt_pk_bf16(acc[tn][tm][4 * g + 2], acc[tn][tm][4 * g + 3])};
      }
  }
}

}  // namespace moe
