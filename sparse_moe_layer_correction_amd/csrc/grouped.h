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

constexpr int kCus = 256;
// Workgroups beyond the most tiles there can be, for the parts of cut tiles
// (grouped_body). Those that find nothing to do are not free: with 192, 500 rows
// for each of 10 experts, [1504, 1504], took 78 us for both gradients instead of 58.
constexpr int kTailBlocks = 32;

struct GroupedArgs {
  const uint16_t* A;
  const uint16_t* B;
  void* C;
  int64_t lda, ldb, ldc;       // row strides in elements
  int64_t b_estride, c_estride;// elements between experts (B of forward / dgrad, C of wgrad)
  int M, N;                    // wgrad: rows / columns of C; else N = columns of C
  int Kd;                      // forward, dgrad: reduction length
  const TileRec* tiles;        // forward, dgrad: M tile table; null: each wave finds its tile in the offsets
  const int32_t* n_mtiles;     //   valid entries
  const int2* ranges;          // wgrad: rows of each expert; null as above
  const int32_t* offsets;      // [E + 1]
  int E, R;
  int rest_blocks;             // without a table: the grid's last workgroups zero the rows of no expert
  int mtiles, ntiles;          // wgrad: tiles of one expert's C; else ntiles = column tiles
  int accumulate;              // wgrad: add to what C holds
  int ksplit, klen;            // forward, dgrad: pieces of the reduction (0 or 1: none) and their length; piece
                               //   s's fp32 sums go to C + s * c_estride
  int before;                  // forward, dgrad: workgroups of the launch that come first
  int split;                   // wgrad: rows of a piece (0: an expert's rows are one sum); piece i's
                               //   fp32 sums go to C + i * c_estride
};

// Finds, in one wave and from the offsets alone, what the tile table holds: lane
// l has the Q experts from Q l on (Q = 2 for up to 128 experts, 16 for 1024). One
// round of loads and two scans over the lanes, against a launch of its own for
// the table: taken for the grids of few workgroups (grouped.hip).
template <int Q>
struct OffsetScan {
  int e0;
  int s[Q + 1];        // expert e0 + j has the rows [s[j], s[j + 1]); none past the last expert
  __device__ __forceinline__ OffsetScan(const int32_t* offsets, int E, int R, int lane) : e0(Q * lane) {
#pragma unroll
    for (int j = 0; j <= Q; ++j) s[j] = min(max(offsets[min(e0 + j, E)], 0), R);
#pragma unroll
    for (int j = 1; j <= Q; ++j) s[j] = max(s[j], s[j - 1]);
    int v = s[Q - 1];                                // the running maximum up to the lane's last start
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(v, d, kWave);
      if (lane >= d) v = max(v, o);
    }
    const int before = __shfl_up(v, 1, kWave);
    if (lane > 0) {
#pragma unroll
      for (int j = 0; j <= Q; ++j) s[j] = max(s[j], before);
    }
  }
  __device__ __forceinline__ int tiles_at(int j, int BM) const { return (s[j + 1] - s[j] + BM - 1) / BM; }
  // rows of expert e, the same in every lane
  __device__ __forceinline__ int2 rows(int e) const {
    int a = 0, b = 0;
#pragma unroll
    for (int j = 0; j < Q; ++j)
      if (e % Q == j) { a = s[j]; b = s[j + 1]; }
    return make_int2(__builtin_amdgcn_readlane(a, e / Q), __builtin_amdgcn_readlane(b, e / Q));
  }
  // M tiles of BM rows over all experts (incl: up to and with the lane's)
  __device__ __forceinline__ int tiles(int BM, int& incl) const {
    int n = 0;
#pragma unroll
    for (int j = 0; j < Q; ++j) n += tiles_at(j, BM);
    incl = wave_inclusive_scan_i32(n);
    return __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  // the lane's first M tile
  __device__ __forceinline__ int first_tile(int BM, int incl) const {
#pragma unroll
    for (int j = 0; j < Q; ++j) incl -= tiles_at(j, BM);
    return incl;
  }
  // the record of the expert that holds M tile mtile
  __device__ __forceinline__ TileRec find(int BM, int mtile, int incl) const {
    int first = first_tile(BM, incl);
    const int src = __builtin_ctzll(__ballot(first <= mtile && mtile < incl));
    int e = 0, f = 0, lo = 0, hi = 0;                // (looked at in lane src only)
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int n = tiles_at(j, BM);
      if (first <= mtile && mtile < first + n) { e = e0 + j; f = first; lo = s[j]; hi = s[j + 1]; }
      first += n;
    }
    return make_int4(__builtin_amdgcn_readlane(e, src), __builtin_amdgcn_readlane(f, src),
                     __builtin_amdgcn_readlane(lo, src), __builtin_amdgcn_readlane(hi, src));
  }
  // first M tile and number of M tiles of expert e
  __device__ __forceinline__ int2 tiles_of(int e, int BM, int incl) const {
    int first = first_tile(BM, incl), f = 0, c = 0;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int n = tiles_at(j, BM);
      if (e % Q == j) { f = first; c = n; }
      first += n;
    }
    return make_int2(__builtin_amdgcn_readlane(f, e / Q), __builtin_amdgcn_readlane(c, e / Q));
  }
  // the rows of no expert: [0, x) and [y, R)
  __device__ __forceinline__ int2 covered() const {
    return make_int2(__builtin_amdgcn_readlane(s[0], 0), __builtin_amdgcn_readlane(s[Q], kWave - 1));
  }
};

// f(the scan), returned
template <typename F>
__device__ __forceinline__ auto with_scan(const int32_t* offsets, int E, int R, int lane, F&& f) {
  if (E <= 2 * kWave) return f(OffsetScan<2>(offsets, E, R, lane));
  return f(OffsetScan<16>(offsets, E, R, lane));
}

// zeroes the rows of no expert, by workgroup i of n with nt threads
__device__ __forceinline__ void zero_rest(uint16_t* C, int64_t ldc, int N, int begin, int end, int R, int i, int n,
                                          int nt) {
  const int cpr = N / 8;
  const int64_t total = (int64_t)(begin + R - end) * cpr;
  for (int64_t j = (int64_t)i * nt + threadIdx.x; j < total; j += (int64_t)n * nt) {
    const int64_t q = j / cpr, r = q < begin ? q : end + (q - begin);
    *reinterpret_cast<u32x4*>(C + r * ldc + (j - q * cpr) * 8) = u32x4{0u, 0u, 0u, 0u};
  }
}

enum GroupedForm : int { FORM_NT = 0, FORM_NN = 1, FORM_TN = 2 };   // forward, dgrad, wgrad

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

constexpr uint32_t kOutOfRange = 0x80000000u;   // past every buffer range used here

// The pointer as scalar registers: the compiler otherwise may keep a uniform
// address in vector registers, and a buffer resource made of those costs a loop
// over the lanes at every load.
__device__ __forceinline__ const uint16_t* uniform_ptr(const uint16_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint16_t*>(((uint64_t)hi << 32) | lo);
}

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
// HS (not TR): not 0, the stage holds half of the tile: of every strip of 2 HS
// rows the HS rows from `half` on.
template <int W, bool TR, int NT, int HS = 0>
struct OperandLoad {
  static constexpr int NL = W * 8 / NT;      // 16-byte loads per thread
  static_assert(HS == 0 || (!TR && HS % 8 == 0), "halves");
  const uint16_t* base;                      // tile's first element (not TR), or first column (TR)
  int64_t ld;
  int klen;
  uint32_t ofs[NL];
  uint64_t tail0, tail1;                     // not TR: the lanes whose chunk lies inside the last k tile,
                                             //   for the loads of even and of odd 8-row blocks
  // load i of a wave fills the 64 chunks (8 rows) from here on
  static __device__ __forceinline__ int chunk(int wave, int i) { return (wave * NL + i) * 64; }
  // width: valid tile rows
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int width, int klen_, int wave, int lane,
                                       int half = 0) {
    base = p;
    ld = ld_;
    klen = klen_;
    if constexpr (!TR) {
      const int left = klen - (klen - 1) / 64 * 64;
      tail0 = __ballot(swz_slot(lane / 8, lane % 8) * 8 < left);
      tail1 = __ballot(swz_slot(8 + lane / 8, lane % 8) * 8 < left);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = chunk(wave, i) + lane;
      if constexpr (TR) {
        const int k = q / (W / 8), c = swz_tr<W>(k, q % (W / 8));
        ofs[i] = c * 8 < width ? (uint32_t)(k * ld * 2 + c * 16) : kOutOfRange;
      } else {
        int r = q / 8;
        const int c = swz_slot(r, q % 8);
        if constexpr (HS > 0) r = r / HS * (2 * HS) + half + r % HS;
        ofs[i] = r < width ? (uint32_t)(r * ld * 2 + c * 16) : kOutOfRange;
      }
    }
  }
  __device__ __forceinline__ void issue(u32x4* stage, int kt, int wave) const {
    const int left = klen - kt * 64;
    if constexpr (TR) {
      const int rows = min(max(left, 0), 64);
      const __amdgpu_buffer_rsrc_t r = make_rsrc(uniform_ptr(base + (int64_t)(rows > 0 ? kt : 0) * 64 * ld),
                                                 __builtin_amdgcn_readfirstlane((int)(rows * ld * 2)));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&stage[chunk(wave, i)], 16, (int)ofs[i], 0, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(base, left > 0 ? kRsrc2G : 0);
      const int so = left > 0 ? kt * 128 : 0;
      const bool whole = left >= 64;
#pragma unroll
      for (int i = 0; i < NL; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)&stage[chunk(wave, i)], 16,
                                                 (int)(__builtin_amdgcn_inverse_ballot_w64(
                                                           whole ? ~0ull : (chunk(wave, i) >> 6) & 1 ? tail1 : tail0)
                                                           ? ofs[i]
                                                           : kOutOfRange),
                                                 so, 0, 0);
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

// MFMA fragments of one 16-deep substep of a wave tile.
template <int TM, int TN>
struct GroupedFrag {
  bf16x8 a[TM], b[TN];
};

// Epilogue of one wave's WTM x WTN tile through its staging area stg (16 KB of
// the idle stages): a lane owns 4 consecutive columns of a row, which stored
// directly would be 8- or 16-byte pieces of 32 rows (measured: the store
// requests then bound the short sums of the weight gradient, 20 us a 256 x 256
// tile); staged, every store writes whole rows of the wave tile. 16-byte chunk c
// of row r sits at chunk c ^ (r % CPW), which spreads the 32 rows of a write
// over the banks. dst: the wave tile's first element; rows / cols: how many of its rows
// and columns (a multiple of 8) exist.
template <int WTM, int WTN, int OUT>
__device__ __forceinline__ void store_wave_tile(const f32x16 (&acc)[WTN / 32][WTM / 32], char* stg, void* dst,
                                                int64_t ldc, int rows, int cols, bool accumulate, int lane) {
  constexpr int ES = OUT == EPI_F32 ? 4 : 2, EPC = 16 / ES;     // bytes of an element, elements of a chunk
  constexpr int CPW = WTN / EPC;                                // chunks of a row
  constexpr int RP = WTM * WTN * ES <= 16384 ? WTM : 16384 / (WTN * ES);   // rows staged at a time
  static_assert(RP % 32 == 0 && WTM % RP == 0 && 64 % CPW == 0, "staging");
  constexpr int RPI = 64 / CPW, NRB = RP / RPI;
#pragma unroll
  for (int p = 0; p < WTM / RP; ++p) {
#pragma unroll
    for (int tm = 0; tm < RP / 32; ++tm) {
      const int r = tm * 32 + (lane & 31);
#pragma unroll
      for (int tn = 0; tn < WTN / 32; ++tn)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& v = acc[tn][p * (RP / 32) + tm];
          if constexpr (OUT == EPI_F32) {
            const int c = tn * 8 + g * 2 + (lane >> 5);
            *reinterpret_cast<f32x4*>(stg + r * (CPW * 16) + ((c ^ (r % CPW)) * 16)) =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          } else {
            const int c = tn * 4 + g;
            *reinterpret_cast<u32x2*>(stg + r * (CPW * 16) + ((c ^ (r % CPW)) * 16) + (lane >> 5) * 8) =
                u32x2{cvt_pk_bf16(v[4 * g], v[4 * g + 1]), cvt_pk_bf16(v[4 * g + 2], v[4 * g + 3])};
          }
        }
    }
    const int r0 = lane / CPW, c = lane % CPW;
    u32x4 rb[NRB];
#pragma unroll
    for (int i = 0; i < NRB; ++i) {
      const int r = i * RPI + r0;
      rb[i] = *reinterpret_cast<const u32x4*>(stg + r * (CPW * 16) + ((c ^ (r % CPW)) * 16));
    }
    const int left = rows - p * RP;
    char* out = static_cast<char*>(dst) + ((int64_t)(p * RP + r0) * ldc + c * EPC) * ES;
    const int64_t step = (int64_t)RPI * ldc * ES;
    if (c * EPC < cols) {
#pragma unroll
      for (int i = 0; i < NRB; ++i, out += step)
        if (i * RPI + r0 < left) {
          u32x4 v = rb[i];
          if constexpr (OUT == EPI_F32) {
            if (accumulate) v = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, v) + *reinterpret_cast<f32x4*>(out));
          }
          *reinterpret_cast<u32x4*>(out) = v;
        }
    }
  }
}

// Tile and part of a workgroup, of valid tiles in a grid that has room for more
// (before: workgroups of the launch that come first). The tiles behind the last
// full round over the CUs are cut into parts of a half or a quarter of their
// height, as far as the grid's spare workgroups go: they end sooner on CUs that
// would idle. us, whole / cut: 544 tiles of 1024 deep sums 84 / 76, 272 of 2048
// 91 / 74, R 65536 over 64, [2048, 2048] 558 / 545; codes, 272 of 2048 59 / 48.
// (Not in a first round: half-height tiles on all CUs load half again as much,
// 126 tiles 31 / 39.)
struct TilePart {
  int t, part = 0, parts = 1;
  template <int BM>
  __device__ __forceinline__ bool pick(int block, int valid, int grid, int before) {
    int tail = 0, n = 1;
    if constexpr (BM == 256) {
      tail = min((before + valid) % kCus, valid);
      const int spare = before + valid > kCus ? min(grid - valid, kCus / 2) : 0;   // (half a round at most)
      n = tail * 3 <= spare ? 4 : tail <= spare ? 2 : 1;
      if (n == 1) tail = 0;
    }
    const int main = valid - tail;
    if (block >= valid + tail * (n - 1)) return false;
    if (block < main) {
      t = xcd_remap(block, main);
    } else {
      part = (block - main) / tail;
      parts = n;
      t = block - part * tail;
    }
    return true;
  }
  // the part's rows [m0, mend); false if the tile has none there
  __device__ __forceinline__ bool rows(int BM, int& m0, int& mend) const {
    if (parts == 1) return true;
    const int h = BM / parts;
    m0 = __builtin_amdgcn_readfirstlane(m0 + part * h);
    mend = __builtin_amdgcn_readfirstlane(min(mend, m0 + h));
    return m0 < mend;
  }
};

// LDS of a workgroup: AST stages of the rows operand, BST of the other, each an
// array of its own, so that the compiler can tell the stage being filled from
// the one being read.
struct GroupedLds {
  u32x4 *a0, *a1, *a2, *a3, *b0, *b1, *b2, *b3;
};
#define MOE_GROUPED_LDS(BM, BN, AST, BST)                                                            \
  static_assert((AST == 2 && (BST == 2 || BST == 3)) || (AST == 4 && BST == 4), "stages");           \
  __shared__ u32x4 sa0[BM * 8], sb0[BN * 8], sa1[BM * 8], sb1[BN * 8], sb2[BST >= 3 ? BN * 8 : 1];   \
  __shared__ u32x4 sa2[AST == 4 ? BM * 8 : 1], sa3[AST == 4 ? BM * 8 : 1], sb3[AST == 4 ? BN * 8 : 1]; \
  const GroupedLds lds{sa0, sa1, sa2, sa3, sb0, sb1, sb2, sb3}

// Tile of workgroup `block` of a weight gradient: runs of g tiles go to the XCDs
// in turn (xcd_remap's one run an XCD shares more rows in an L2, but experts
// differ in length, and the XCD with the longest ones ends the launch alone).
// us, dx and fp32 dW, one run / runs of 8 / of 16 tiles: R 65536 over 64 experts as
// 1/rank^1.1, [2048, 2048] 1711 / 1144 / 1245, R 16384 over 8, [2048, 1024] 205 /
// 146 / 185; even, R 65536 1171 / 1182 / 1172, R 32768 over 128, [2048, 5120] 2360 /
// 2307 / 2334.
constexpr int kWgradRun = 8;
__device__ __forceinline__ int xcd_runs(int block, int nblocks, int g) {
  if (block >= nblocks / (8 * g) * (8 * g)) return block;
  const int x = block % 8, j = block / 8;
  return (j / g * 8 + x) * g + j % g;
}

// Workgroup `block` of the `nblocks` of one product: a C tile BM x BN by WM x WN
// waves. OUT: EPI_BF16 or EPI_F32.
template <int FORM, int BM, int BN, int WM, int WN, int OUT, int AST, int BST>
__device__ __forceinline__ void grouped_body(const GroupedArgs& P, int block, int nblocks, const GroupedLds& lds) {
  constexpr int NT = 64 * WM * WN;
  constexpr bool AT = FORM == FORM_TN, BT = FORM != FORM_NT;
  constexpr bool DEEP = AST == 4;
  static_assert(BM * 8 % NT == 0 && BN * 8 % NT == 0, "tile shape");
  u32x4 *const sa0 = lds.a0, *const sa1 = lds.a1, *const sa2 = lds.a2, *const sa3 = lds.a3;
  u32x4 *const sb0 = lds.b0, *const sb1 = lds.b1, *const sb2 = lds.b2, *const sb3 = lds.b3;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave % WM, wave_n = wave / WM;

  int m0, mend, n0, Kd;
  const uint16_t *Ap, *Bp;
  int64_t c_base = 0;
  if constexpr (FORM == FORM_TN) {
    const int per = P.mtiles * P.ntiles;
    int t, e;
    int2 rg;
    if (P.split > 0) {
      // pieces of an expert's rows are laid out as the M tiles of a rows product are
      TileRec rec;
      const bool mine = with_scan(P.offsets, P.E, P.R, lane, [&](const auto& scan) {
        int incl;
        const int valid = scan.tiles(P.split, incl) * per;
        if (block >= valid) return false;
        t = xcd_remap(block, valid);
        e = __builtin_amdgcn_readfirstlane(t / per);     // the piece: C's index
        rec = scan.find(P.split, e, incl);
        return true;
      });
      if (!mine) return;
      rg.x = rec.z + (e - rec.y) * P.split;
      rg.y = min(rg.x + P.split, rec.w);
    } else {
      t = xcd_runs(block, nblocks, min(per, kWgradRun));
      e = __builtin_amdgcn_readfirstlane(t / per);
      if (P.ranges != nullptr) rg = P.ranges[e];
      else rg = with_scan(P.offsets, P.E, P.R, lane, [&](const auto& scan) { return scan.rows(e); });
    }
    int mt, nt;
    tile_order(t - e * per, P.mtiles, P.ntiles, 4, mt, nt);
    m0 = __builtin_amdgcn_readfirstlane(mt * BM);
    n0 = __builtin_amdgcn_readfirstlane(nt * BN);
    mend = P.M;
    const int lo = __builtin_amdgcn_readfirstlane(rg.x);
    Kd = __builtin_amdgcn_readfirstlane(rg.y) - lo;
    if (Kd <= 0) {
      // no rows: zeros, straight to memory (through the sums and LDS a tile of
      // them took 10 us; 500 MB of empty experts 163 us)
      if (P.accumulate) return;
      constexpr int ES = OUT == EPI_F32 ? 4 : 2, EPC = 16 / ES, CPR = BN / EPC;
      char* dst = static_cast<char*>(P.C) + ((int64_t)e * P.c_estride + (int64_t)m0 * P.ldc + n0) * ES;
      const int rows = min(BM, mend - m0), cols = P.N - n0;
      for (int i = tid; i < rows * CPR; i += NT) {
        const int r = i / CPR, c = i % CPR * EPC;
        if (c < cols) *reinterpret_cast<u32x4*>(dst + ((int64_t)r * P.ldc + c) * ES) = u32x4{0u, 0u, 0u, 0u};
      }
      return;
    }
    Ap = P.A + (int64_t)lo * P.lda + m0;
    Bp = P.B + (int64_t)lo * P.ldb + n0;
    c_base = (int64_t)e * P.c_estride;
  } else {
    int k0 = 0;
    TilePart tp;
    TileRec rec;
    if (P.ksplit > 1) {
      nblocks /= P.ksplit;
      const int piece = block / nblocks;
      block -= piece * nblocks;
      k0 = piece * P.klen;
      c_base = piece * P.c_estride;
    }
    if (P.tiles != nullptr) {
      if (!tp.pick<BM>(block, *P.n_mtiles * P.ntiles, nblocks, P.before)) return;
      rec = P.tiles[tp.t / P.ntiles];
    } else {
      const bool mine = with_scan(P.offsets, P.E, P.R, lane, [&](const auto& scan) {
        const int grid = nblocks - P.rest_blocks;
        if (block >= grid) {
          const int2 c = scan.covered();
          zero_rest(static_cast<uint16_t*>(P.C), P.ldc, P.N, c.x, c.y, P.R, block - grid, P.rest_blocks, NT);
          return false;
        }
        int incl;
        if (!tp.pick<BM>(block, scan.tiles(BM, incl) * P.ntiles, grid, P.before)) return false;
        rec = scan.find(BM, tp.t / P.ntiles, incl);
        return true;
      });
      if (!mine) return;
    }
    const int e = __builtin_amdgcn_readfirstlane(rec.x), first = __builtin_amdgcn_readfirstlane(rec.y);
    const int lo = __builtin_amdgcn_readfirstlane(rec.z), hi = __builtin_amdgcn_readfirstlane(rec.w);
    int mt, nt;
    grouped_tile_order(tp.t - first * P.ntiles, (hi - lo + BM - 1) / BM, (hi - lo) / BM, P.ntiles, 8, mt, nt);
    m0 = __builtin_amdgcn_readfirstlane(lo + mt * BM);
    n0 = __builtin_amdgcn_readfirstlane(nt * BN);
    mend = hi;
    if constexpr (BM == 256) {
      if (!tp.rows(BM, m0, mend)) return;
    }
    Kd = P.ksplit > 1 ? min(P.klen, P.Kd - k0) : P.Kd;
    Ap = P.A + (int64_t)m0 * P.lda + k0;
    Bp = P.B + (int64_t)e * P.b_estride + (BT ? (int64_t)k0 * P.ldb + n0 : (int64_t)n0 * P.ldb + k0);
  }

  // HQ: the tile's height in quarters of BM (an expert's short last tile; the
  // weight gradient's tiles are always whole)
  auto body = [&](auto height) __attribute__((always_inline)) {
    constexpr int HQ = decltype(height)::value;
    constexpr int H = BM * HQ / 4;
    constexpr int WTM = H / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
    static_assert(TM >= 1 && TN >= 1 && WTM % 32 == 0 && H * 8 % NT == 0, "wave tile");
    OperandLoad<H, AT, NT> la;
    OperandLoad<BN, BT, NT> lb;
    la.init(Ap, P.lda, mend - m0, Kd, wave, lane);
    lb.init(Bp, P.ldb, P.N - n0, Kd, wave, lane);
    OperandRead<H, AT, TM> ra;
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
    typedef GroupedFrag<TM, TN> Frag;
    Frag f0, f1;
    auto read = [&](Frag& f, const u32x4* a, const u32x4* b, int ks) {
      ra.read(f.a, a, ks, lane);
      rb.read(f.b, b, ks, lane);
    };
    auto mma = [&](const Frag& f) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
          acc[tn][tm] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[tn], f.a[tm], acc[tn][tm], 0, 0, 0);
    };
    // AST LDS stages of A, BST of B. The reads of a 16-deep substep run beside
    // the MFMAs of the one before; the one barrier of a k tile sits before its
    // last substep, whose fragments are in registers by then: past it the next
    // tile has landed and nobody reads this tile's stages. With three stages B
    // is loaded two tiles ahead (the weights, which come from HBM while the
    // rows stay in the caches), in the second substep of the tile before. Four
    // stages of both (128 x 128 tiles, one workgroup to a CU) are for grids that
    // leave CUs idle: a k tile's time is then the loads' latency over the tiles in flight.
    constexpr int NM = TM * TN, NR = TM * (AT ? 2 : 1) + TN * (BT ? 2 : 1);
    constexpr int NA = OperandLoad<H, AT, NT>::NL, NB = OperandLoad<BN, BT, NT>::NL;
    auto stA = [&](auto v) -> u32x4* {
      if constexpr (decltype(v)::value == 0) return sa0;
      else if constexpr (decltype(v)::value == 1) return sa1;
      else if constexpr (decltype(v)::value == 2) return sa2;
      else return sa3;
    };
    auto stB = [&](auto v) -> u32x4* {
      if constexpr (decltype(v)::value == 0) return sb0;
      else if constexpr (decltype(v)::value == 1) return sb1;
      else if constexpr (decltype(v)::value == 2) return sb2;
      else return sb3;
    };
    // s_waitcnt vmcnt(VM) lgkmcnt(0): the loads that stay in flight over a barrier are,
    // with three stages of B, those of its tile kt + 2, with four those of the tiles kt + 2 and kt + 3
    constexpr int VM = DEEP ? 2 * (NA + NB) : BST == 3 ? NB : 0;
    constexpr int kWait = (VM & 0xF) | (0x7 << 4) | (0x0 << 8) | (((VM >> 4) & 3) << 14);
    auto step = [&](int kt, auto sa, auto sb, auto first) {
      constexpr int SA = decltype(sa)::value, SB = decltype(sb)::value;
      constexpr bool MID = BST == 3 &&  decltype(first)::value == 0;   // tile 2 was loaded before step 0
      read(f1, stA(sa), stB(sb), 1);
      mma(f0);
      interleave<NM, NR, 0>();
      read(f0, stA(sa), stB(sb), 2);
      if constexpr (MID) lb.issue(stB(Stage<(SB + 2) % 3>{}), kt + 2, wave);
      mma(f1);
      interleave<NM, NR, MID ? NB : 0>();
      read(f1, stA(sa), stB(sb), 3);
      mma(f0);
      interleave<NM, NR, 0>();
      __builtin_amdgcn_s_waitcnt(kWait);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      la.issue(stA(sa), kt + AST, wave);
      if constexpr (BST != 3) lb.issue(stB(sb), kt + BST, wave);
      read(f0, stA(Stage<(SA + 1) % AST>{}), stB(Stage<(SB + 1) % BST>{}), 0);
      mma(f1);
      interleave<NM, NR, NA + (BST != 3 ? NB : 0)>();
    };
    if (nk > 0) {
      la.issue(sa0, 0, wave);
      lb.issue(sb0, 0, wave);
      la.issue(sa1, 1, wave);
      lb.issue(sb1, 1, wave);
      if constexpr (BST == 3) lb.issue(sb2, 2, wave);
      if constexpr (DEEP) {
        la.issue(sa2, 2, wave);
        lb.issue(sb2, 2, wave);
        la.issue(sa3, 3, wave);
        lb.issue(sb3, 3, wave);
      }
      MOE_WAIT_VMCNT((AST - 1) * NA + (BST - 1) * NB);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      read(f0, sa0, sb0, 0);
      const Stage<0> S0{};
      const Stage<1> S1{};
      const Stage<2> S2{};
      if constexpr (BST == 2) {
        int kt = 0;
        for (; kt + 1 < nk; kt += 2) {
          step(kt, S0, S0, S0);
          step(kt + 1, S1, S1, S0);
        }
        if (kt < nk) step(kt, S0, S0, S0);
      } else if constexpr (DEEP) {
        const Stage<3> S3{};
        int kt = 0;
        for (; kt + 4 <= nk; kt += 4) {
          step(kt, S0, S0, S0);
          step(kt + 1, S1, S1, S0);
          step(kt + 2, S2, S2, S0);
          step(kt + 3, S3, S3, S0);
        }
        if (kt < nk) {
          step(kt, S0, S0, S0);
          if (kt + 1 < nk) {
            step(kt + 1, S1, S1, S0);
            if (kt + 2 < nk) step(kt + 2, S2, S2, S0);
          }
        }
      } else {
        step(0, S0, S0, S1);
        // step kt reads A stage kt % 2 and B stage kt % 3
        int kt = 1;
        for (; kt + 6 <= nk; kt += 6) {
          step(kt, S1, S1, S0);
          step(kt + 1, S0, S2, S0);
          step(kt + 2, S1, S0, S0);
          step(kt + 3, S0, S1, S0);
          step(kt + 4, S1, S2, S0);
          step(kt + 5, S0, S0, S0);
        }
        if (kt < nk) {
          step(kt, S1, S1, S0);
          if (kt + 1 < nk) {
            step(kt + 1, S0, S2, S0);
            if (kt + 2 < nk) {
              step(kt + 2, S1, S0, S0);
              if (kt + 3 < nk) {
                step(kt + 3, S0, S1, S0);
                if (kt + 4 < nk) step(kt + 4, S1, S2, S0);
              }
            }
          }
        }
      }
    }
    MOE_WAIT_VMCNT(0);   // no load may write a stage that the epilogue uses, or that the next workgroup gets
    __syncthreads();
    // staging: all of it in one array, or 16 KB a wave in an array each or half of one
    constexpr int ES = OUT == EPI_F32 ? 4 : 2, SB = WTM * WTN * ES;
    char* stg;
    if constexpr (WM * WN * SB <= BN * 128) {
      stg = reinterpret_cast<char*>(sb0) + wave * SB;
    } else {
      constexpr int per = BM * 8 * 16 / 16384;
      static_assert(WM * WN <= 4 * per, "staging areas");
      const int h = wave / per;
      stg = reinterpret_cast<char*>(h == 0 ? sa0 : h == 1 ? sb0 : h == 2 ? sa1 : sb1) + (wave % per) * 16384;
    }
    const int mw = m0 + wave_m * WTM, nw = n0 + wave_n * WTN;
    void* dst = static_cast<char*>(P.C) + (c_base + (int64_t)mw * P.ldc + nw) * ES;
    bool add = false;
    if constexpr (FORM == FORM_TN) {
      add = P.accumulate != 0;
      if constexpr (OUT == EPI_BF16) {
        // bf16 sums are added in fp32, before the one rounding
        if (add) {
#pragma unroll
          for (int tm = 0; tm < TM; ++tm) {
            const int r = tm * 32 + (lane & 31);
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const int c = tn * 32 + 8 * g + 4 * (lane >> 5);
                if (mw + r >= mend || nw + c >= P.N) continue;
                const u32x2 o = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(dst) + (int64_t)r * P.ldc + c);
                acc[tn][tm][4 * g] += bf16_bits_to_f32(o.x & 0xFFFFu);
                acc[tn][tm][4 * g + 1] += bf16_bits_to_f32(o.x >> 16);
                acc[tn][tm][4 * g + 2] += bf16_bits_to_f32(o.y & 0xFFFFu);
                acc[tn][tm][4 * g + 3] += bf16_bits_to_f32(o.y >> 16);
              }
          }
        }
      }
    }
    store_wave_tile<WTM, WTN, OUT>(acc, stg, dst, P.ldc, mend - mw, P.N - nw, add, lane);
  };
  if constexpr (FORM != FORM_TN && BM == 256) {
    // an expert's short last tile at a quarter, half or three quarters of the height
    const int rows = mend - m0;
    if (rows <= 64) { body(Stage<1>{}); return; }
    if (rows <= 128) { body(Stage<2>{}); return; }
    if (rows <= 192) { body(Stage<3>{}); return; }
  }
  body(Stage<4>{});
}

// OCC: waves per SIMD the registers are sized for.
template <int FORM, int BM, int BN, int WM, int WN, int OCC, int OUT, int AST, int BST>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_kernel(const GroupedArgs P) {
  MOE_GROUPED_LDS(BM, BN, AST, BST);
  grouped_body<FORM, BM, BN, WM, WN, OUT, AST, BST>(P, blockIdx.x, gridDim.x, lds);
}

// Both gradients in one launch: the first g0 workgroups take dW, the others dx.
// The two are independent, and what one leaves idle the other fills: the CUs
// beside a long expert's dW, whose tiles start first, and those of dx's last
// tiles.
// (DXO: of dx; EPI_F32 for the pieces of a split reduction)
template <int BM, int BN, int WM, int WN, int OCC, int DXO, int OUT, int AST, int BST>
__global__ void __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
grouped_grad_kernel(const GroupedArgs DX, const GroupedArgs DW, int g0) {
  MOE_GROUPED_LDS(BM, BN, AST, BST);
  if ((int)blockIdx.x < g0)
    grouped_body<FORM_TN, BM, BN, WM, WN, OUT, AST, BST>(DW, blockIdx.x, g0, lds);
  else
    grouped_body<FORM_NN, BM, BN, WM, WN, DXO, AST, BST>(DX, (int)blockIdx.x - g0, (int)gridDim.x - g0, lds);
}

}  // namespace moe
