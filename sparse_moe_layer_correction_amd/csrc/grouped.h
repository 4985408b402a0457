// Products over rows grouped by expert, and their gradients (bf16 MFMA, gfx950).
//
// With rows r of expert e(r) in [lo_e, hi_e) and W[e] an [N, K] weight:
//   forward  y[r, n]     = sum_k x[r, k] W[e][n, k]     rows x k      . cols x k
//   dgrad    dx[r, k]    = sum_n dy[r, n] W[e][n, k]    rows x n      . n x cols
//   wgrad    dW[e][n, k] = sum_{r in e} dy[r, n] x[r, k]   r x rows   . r x cols
// One kernel template serves the three: an operand either has the reduction
// index contiguous (stored [tile row][k]) or the tile's own index contiguous
// (stored [k][tile row], "transposed"). Both come global -> LDS directly in
// 16-byte chunks. A transposed operand's MFMA fragments are read from LDS by
// ds_read_b64_tr_b16, which hands each lane four consecutive k of its column, so
// no tensor is transposed in memory and both layouts move the same bytes.
//
// What lies outside a tensor (rows past an expert's end, columns past N or K,
// the reduction's tail) is put out of the buffer's range: the load then writes
// zeros to LDS and reads no memory, so neighbours' infinities or NaN never
// enter a sum.
#pragma once

#include "gemm.h"

namespace moe {

// One tile row block of a grouped product: expert, first M tile of the expert, rows [lo, hi).
typedef int4 TileRec;

struct GroupedArgs {
  const uint16_t* A;
  const uint16_t* B;
  void* C;
  int64_t lda, ldb, ldc;       // row strides in elements
  int64_t b_estride, c_estride;// elements between experts (B of forward / dgrad, C of wgrad)
  int M, N;                    // wgrad: rows / columns of C; else N = columns of C
  int Kd;                      // forward, dgrad: reduction length
  const TileRec* tiles;        // forward, dgrad: M tile table
  const int32_t* n_mtiles;     //   valid entries
  const int2* ranges;          // wgrad: rows of each expert
  int mtiles, ntiles;          // wgrad: tiles of one expert's C; else ntiles = column tiles
  int accumulate;              // wgrad: add to what C holds
};

enum GroupedForm : int { FORM_NT = 0, FORM_NN = 1, FORM_TN = 2 };   // forward, dgrad, wgrad

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

constexpr uint32_t kOutOfRange = 0x80000000u;   // past every buffer range used here

// Slot of 16-byte chunk c of reduction row k of a transposed stage of W
// columns. A transposing read's 32 lanes take 64 bytes of each of 4 consecutive
// rows: the four pieces have to lie in different quarters of the 256-byte bank
// window.
template <int W>
__device__ __forceinline__ int swz_tr(int k, int c) {
  if constexpr (W >= 128) return c ^ ((k & 3) << 2);
  else return c ^ (((k >> 1) & 1) << 2);
}

// Loads of one operand's [64-deep k tile] stage: W tile rows (columns of C or
// rows of C), TR: stored reduction-major.
template <int W, bool TR, int NT>
struct OperandLoad {
  static constexpr int NL = W * 8 / NT;      // 16-byte loads per thread
  const uint16_t* base;                      // tile's first element (not TR), or first column (TR)
  int64_t ld;
  int klen;
  uint32_t ofs[NL];
  int kc[NL];                                // not TR: first k of the lane's chunk inside the tile
  // width: valid tile rows
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int width, int klen_, int wave, int lane) {
    base = p;
    ld = ld_;
    klen = klen_;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = (wave * NL + i) * 64 + lane;
      if constexpr (TR) {
        const int k = q / (W / 8), c = swz_tr<W>(k, q % (W / 8));
        ofs[i] = c * 8 < width ? (uint32_t)(k * ld * 2 + c * 16) : kOutOfRange;
        kc[i] = 0;
      } else {
        const int r = q / 8, c = swz_slot(r, q % 8);
        ofs[i] = r < width ? (uint32_t)(r * ld * 2 + c * 16) : kOutOfRange;
        kc[i] = c * 8;
      }
    }
  }
  __device__ __forceinline__ void issue(u32x4* stage, int kt, int wave) const {
    const int left = klen - kt * 64;
    if constexpr (TR) {
      // (a scalar again: the clamp is a vector instruction, and a resource in
      // vector registers costs a loop over the lanes at every load)
      const int rows = __builtin_amdgcn_readfirstlane(min(max(left, 0), 64));
      const __amdgpu_buffer_rsrc_t r = make_rsrc(base + (int64_t)(rows > 0 ? kt : 0) * 64 * ld, (int)(rows * ld * 2));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&stage[(wave * NL + i) * 64], 16, (int)ofs[i], 0, 0,
                                                 0);
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(base, left > 0 ? kRsrc2G : 0);
      const int so = left > 0 ? kt * 128 : 0;
#pragma unroll
      for (int i = 0; i < NL; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&stage[(wave * NL + i) * 64], 16,
                                                 (int)(kc[i] < left ? ofs[i] : kOutOfRange), so, 0, 0);
    }
  }
};

// MFMA fragments of an operand's wave tile (T 32-row tiles from tile row row0):
// lane l holds tile row (l & 31), k = 16 ks + 8 (l >> 5) .. + 7.
template <int W, bool TR, int T>
struct OperandRead {
  int at[T];                                 // TR: byte address; else the row's first chunk
  int sw;
  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (TR) {
      const int i = lane & 15, g = lane >> 4;
      const int k = (g >> 1) * 8 + (i >> 2);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int col = row0 + t * 32 + (g & 1) * 16 + (i & 3) * 4;
        at[t] = k * (W * 2) + swz_tr<W>(k, col / 8) * 16 + (i & 1) * 8;
      }
      sw = 0;
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) at[t] = (row0 + t * 32 + (lane & 31)) * 8;
      sw = ((lane & 31) >> 1) & 7;
    }
  }
  __device__ __forceinline__ void read(bf16x8 (&f)[T], const u32x4* stage, int ks, int lane) const {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if constexpr (TR) {
        const char* p = reinterpret_cast<const char*>(stage) + at[t] + ks * 16 * (W * 2);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(const_cast<char*>(p)));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(const_cast<char*>(p) + 4 * (W * 2)));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        f[t] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        f[t] = __builtin_bit_cast(bf16x8, stage[at[t] + ((ks * 2 + (lane >> 5)) ^ sw)]);
      }
    }
  }
};

// C tile BM x BN by WM x WN waves. OUT: EPI_BF16 or EPI_F32.
template <int FORM, int BM, int BN, int WM, int WN, int OCC, int OUT>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_kernel(const GroupedArgs P) {
  constexpr int NT = 64 * WM * WN;
  constexpr bool AT = FORM == FORM_TN, BT = FORM != FORM_NT;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  static_assert(TM >= 1 && TN >= 1 && BM * 8 % NT == 0 && BN * 8 % NT == 0, "tile shape");
  __shared__ u32x4 sa0[BM * 8], sb0[BN * 8], sa1[BM * 8], sb1[BN * 8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave % WM, wave_n = wave / WM;

  int m0, mend, n0, Kd;
  const uint16_t *Ap, *Bp;
  int64_t c_base = 0;
  if constexpr (FORM == FORM_TN) {
    const int per = P.mtiles * P.ntiles;
    const int t = xcd_remap(blockIdx.x, gridDim.x);
    const int e = __builtin_amdgcn_readfirstlane(t / per);
    int mt, nt;
    tile_order(t - e * per, P.mtiles, P.ntiles, 4, mt, nt);
    m0 = mt * BM;
    mend = P.M;
    n0 = nt * BN;
    m0 = __builtin_amdgcn_readfirstlane(m0);
    n0 = __builtin_amdgcn_readfirstlane(n0);
    const int lo = __builtin_amdgcn_readfirstlane(P.ranges[e].x);
    Kd = __builtin_amdgcn_readfirstlane(P.ranges[e].y) - lo;
    if (Kd <= 0 && P.accumulate) return;
    Ap = P.A + (int64_t)lo * P.lda + m0;
    Bp = P.B + (int64_t)lo * P.ldb + n0;
    c_base = (int64_t)e * P.c_estride;
  } else {
    const int valid = *P.n_mtiles * P.ntiles;
    if ((int)blockIdx.x >= valid) return;
    const int t = xcd_remap(blockIdx.x, valid);
    const TileRec rec = P.tiles[t / P.ntiles];
    const int e = __builtin_amdgcn_readfirstlane(rec.x), first = __builtin_amdgcn_readfirstlane(rec.y);
    const int lo = __builtin_amdgcn_readfirstlane(rec.z), hi = __builtin_amdgcn_readfirstlane(rec.w);
    int mt, nt;
    grouped_tile_order(t - first * P.ntiles, (hi - lo + BM - 1) / BM, (hi - lo) / BM, P.ntiles, 1 << 20, mt, nt);
    m0 = lo + mt * BM;
    mend = hi;
    n0 = nt * BN;
    m0 = __builtin_amdgcn_readfirstlane(m0);
    n0 = __builtin_amdgcn_readfirstlane(n0);
    Kd = P.Kd;
    Ap = P.A + (int64_t)m0 * P.lda;
    Bp = P.B + (int64_t)e * P.b_estride + (BT ? (int64_t)n0 : (int64_t)n0 * P.ldb);
  }

  OperandLoad<BM, AT, NT> la;
  OperandLoad<BN, BT, NT> lb;
  la.init(Ap, P.lda, mend - m0, Kd, wave, lane);
  lb.init(Bp, P.ldb, P.N - n0, Kd, wave, lane);
  OperandRead<BM, AT, TM> ra;
  OperandRead<BN, BT, TN> rb;
  ra.init(wave_m * WTM, lane);
  rb.init(wave_n * WTN, lane);

  f32x16 acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[a][b][q] = 0.f;

  const int nk = (Kd + 63) / 64;
  auto step = [&](int kt, const u32x4* a, const u32x4* b, u32x4* an, u32x4* bn) {
    la.issue(an, kt + 1, wave);
    lb.issue(bn, kt + 1, wave);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8 fa[TM], fb[TN];
      ra.read(fa, a, ks, lane);
      rb.read(fb, b, ks, lane);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
          acc[tn][tm] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[tn], fa[tm], acc[tn][tm], 0, 0, 0);
    }
    MOE_WAIT_VMCNT(0);
    __syncthreads();
  };
  if (nk > 0) {
    la.issue(sa0, 0, wave);
    lb.issue(sb0, 0, wave);
    MOE_WAIT_VMCNT(0);
    __syncthreads();
    for (int kt = 0; kt < nk; kt += 2) {
      step(kt, sa0, sb0, sa1, sb1);
      if (kt + 1 < nk) step(kt + 1, sa1, sb1, sa0, sb0);
    }
  }

  // lane l owns row (l & 31) of each 32 x 32 tile and columns 8 g + 4 (l >> 5) .. + 3
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int m = m0 + wave_m * WTM + tm * 32 + (lane & 31);
    if (m >= mend) continue;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wave_n * WTN + tn * 32 + 8 * g + 4 * (lane >> 5);
        if (n >= P.N) continue;
        f32x4 v{acc[tn][tm][4 * g], acc[tn][tm][4 * g + 1], acc[tn][tm][4 * g + 2], acc[tn][tm][4 * g + 3]};
        const int64_t at = c_base + (int64_t)m * P.ldc + n;
        if constexpr (OUT == EPI_F32) {
          f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(P.C) + at);
          if (FORM == FORM_TN && P.accumulate) v += *dst;
          *dst = v;
        } else {
          u32x2* dst = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(P.C) + at);
          if (FORM == FORM_TN && P.accumulate) {
            const u32x2 o = *dst;
            v[0] += bf16_bits_to_f32(o.x & 0xFFFFu);
            v[1] += bf16_bits_to_f32(o.x >> 16);
            v[2] += bf16_bits_to_f32(o.y & 0xFFFFu);
            v[3] += bf16_bits_to_f32(o.y >> 16);
          }
          *dst = u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
        }
      }
  }
}

}  // namespace moe
