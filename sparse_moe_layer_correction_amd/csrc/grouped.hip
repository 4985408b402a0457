// Tile table and launchers of the grouped products (grouped.h).
#include "grouped.h"
#include "grouped_ops.h"

namespace moe {

// Rows of each expert from its offsets, and the M tile table of a product with
// BM-row tiles. offsets that fall, or lie outside [0, R], are read as their
// running maximum clamped to [0, R]: ranges then never overlap, their tiles
// never pass R / BM + E, and no kernel touches a row outside [0, R). One
// workgroup, thread e for expert e (E <= 1024): two scans over the waves. The
// workgroups after it (kRestBlocks, launched where rest is asked for) zero the
// output's rows before the first expert's and after the last one's.
constexpr int kRestBlocks = 64;
__global__ void __launch_bounds__(1024) grouped_tiles_kernel(const int32_t* __restrict__ offsets, int E, int R, int BM,
                                                             int2* __restrict__ ranges, TileRec* __restrict__ tiles,
                                                             int32_t* __restrict__ n_mtiles, const RestRows rest) {
  __shared__ int wmax[16], wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto clamped = [&](int i) { return min(max(offsets[min(i, E)], 0), R); };
  int v = clamped(tid);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(v, d, kWave);
    if (lane >= d) v = max(v, o);
  }
  if (lane == 63) wmax[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = max(v, wmax[w]);
  if (blockIdx.x > 0) {
    __shared__ int end;                                      // the highest offset
    if (tid == E - 1) end = max(v, clamped(E));
    __syncthreads();
    zero_rest(rest.C, rest.ldc, rest.N, clamped(0), end, R, (int)blockIdx.x - 1, kRestBlocks, 1024);
    return;
  }
  const int lo = v;
  const int hi = tid < E ? max(lo, clamped(tid + 1)) : lo;   // the next expert's start: max with all before it
  const int nt = (hi - lo + BM - 1) / BM;
  const int it = wave_inclusive_scan_i32(nt);
  if (lane == 63) wsum[wave] = it;
  __syncthreads();
  int first = it - nt;
  for (int w = 0; w < wave; ++w) first += wsum[w];
  if (tid < E) ranges[tid] = make_int2(lo, hi);
  if (tid == E - 1) *n_mtiles = first + nt;
  // the records, a thread for every 1024th of them (an expert with all rows has
  // thousands): the last expert that starts at or before the tile, empty ones
  // starting where the next one does
  __shared__ int starts[1024], from[1024], to[1024], total;
  starts[tid] = tid < E ? first : 0x7FFFFFFF;
  from[tid] = lo;
  to[tid] = hi;
  if (tid == E - 1) total = first + nt;
  __syncthreads();
  for (int i = tid; i < total; i += 1024) {
    int e = 0;
#pragma unroll
    for (int d = 512; d >= 1; d >>= 1)
      if (e + d < 1024 && starts[e + d] <= i) e += d;
    tiles[i] = make_int4(e, starts[e], from[e], to[e]);
  }
}

hipError_t launch_grouped_tiles(const int32_t* offsets, int E, int R, int BM, const GroupedScratch& s,
                                const RestRows& rest, hipStream_t st) {
  hipLaunchKernelGGL(grouped_tiles_kernel, dim3(rest.C && R > 0 ? 1 + kRestBlocks : 1), dim3(1024), 0, st, offsets, E, R,
                     BM, s.ranges, s.tiles, s.n_mtiles, rest);
  return hipGetLastError();
}

template <int FORM, int OUT>
static void launch_form(const GroupedArgs& a, const GroupedPlan& plan, int64_t grid, hipStream_t st) {
  const dim3 g((unsigned)grid);
  if constexpr (FORM != FORM_TN) {
    if (plan.bm == 32) {
      if (plan.ksplit)
        hipLaunchKernelGGL((grouped_kernel<FORM, 32, 128, 1, 4, 2, EPI_F32, 4, 4>), g, dim3(256), 0, st, a);
      else
        hipLaunchKernelGGL((grouped_kernel<FORM, 32, 128, 1, 4, 2, OUT, 4, 4>), g, dim3(256), 0, st, a);
      return;
    }
  }
  if (plan.bm == 256)
    hipLaunchKernelGGL((grouped_kernel<FORM, 256, 256, 2, 4, 2, OUT, 2, 3>), g, dim3(512), 0, st, a);
  else if (plan.ksplit)
    hipLaunchKernelGGL((grouped_kernel<FORM, 128, 128, 2, 2, 1, EPI_F32, 4, 4>), g, dim3(256), 0, st, a);
  else if (plan.deep)
    hipLaunchKernelGGL((grouped_kernel<FORM, 128, 128, 2, 2, 1, OUT, 4, 4>), g, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((grouped_kernel<FORM, 128, 128, 2, 2, 2, OUT, 2, 2>), g, dim3(256), 0, st, a);
}

// Which tiles, from what the host knows (the rows' number, not their spread; an
// expert's last M tile is taken as half used). us of a call, 256 x 256 tiles /
// 128 x 128 tiles / the latter with four stages:
//   rows product, R 20000, E 2, [640, 640] (237 big tiles)   22 / 26 / 37
//   rows product, R 32768, E 128, [2048, 5120]              819 / 1034 / 1101
//   wgrad, R 8000, E 30, [504, 3000] (720 big tiles)         68 / 70 / 104 (with dx 119 / 155)
//   wgrad, R 20000, E 2, [640, 640] (18 big, 50 small)        - / 100 / 62
//   dgrad, R 2000, E 16, [1200, 400] (124 small tiles)        - / 15.8 / 13.2
//   rows product, R 17097, E 12, [368, 4952] (144 big tiles)  90 / 94 / 104
//   wgrad, R 76894, E 329, [112, 560] (half of a big tile)    50 / 37 / -
// So the big tile where its tiles are more than half the 256 CUs' number and
// compute little beyond the output's edge (kBigPadding times the small tiles'),
// else the small one, with four stages while every workgroup has a CU to itself
// (more of them then ask for more than the L2 gives: 0.25 us of MFMA a k tile, 32 KB).
constexpr int64_t kBigTiles = 136, kDeepGrid = 256;
constexpr double kBigPadding = 1.3;
// Few rows to an expert (fewer than this many on average): the weights' bytes
// bound the product, and what counts is how many of them are on their way. Tiles
// of 32 rows with four stages, two workgroups to a CU, have 96 KB of weights in
// flight a CU, 128-row tiles of two stages 32. us, 128-row / 32-row tiles, E 100,
// [1024, 2048]: 20 rows 104 / 96 (dgrad 97 / 87), 40 rows 91 / 92 (102 / 106), 80
// rows 115 / 126 (115 / 124); codes 43 / 39, 45 / 41, 49 / 49.
constexpr int kFewRows = 24, kFewRowsCodes = 48;
static int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
// Grids of at most this many workgroups find their tiles in the offsets
// (OffsetScan) and need no table; with more than 128 experts, 16 to a lane, of
// at most the second number.
constexpr int64_t kScanGrid = 1024, kScanGridWide = 512;
// A rows product of few tiles and a long reduction (kSplitMinSteps k tiles) is
// summed in pieces side by side, as many as give every CU a workgroup but of 4 k
// tiles at least, and joined in order.
constexpr int kSplitMinSteps = 24;

static void finish_plan(GroupedPlan& p, int E) {
  p.deep = p.bm == 128 && p.grid <= kDeepGrid;
  p.scan = p.grid <= (E <= 2 * kWave ? kScanGrid : kScanGridWide);
}

GroupedPlan grouped_rows_plan(int64_t R, int E, int N, int kd, int kstep, bool few) {
  GroupedPlan p{};
  const int64_t big = (R / 256 + std::min<int64_t>(R, E) / 2) * ((N + 255) / 256);
  const bool fits = up(N, 256) <= kBigPadding * up(N, 128);
  const int64_t few_rows = (int64_t)E * (kstep == 64 ? kFewRows : kFewRowsCodes);
  p.bm = R >= (int64_t)E * 128 && big >= kBigTiles && fits ? 256 : few && R < few_rows ? 32 : 128;
  const int bn = std::max(p.bm, 128);
  p.ntiles = (N + bn - 1) / bn;
  p.grid = grouped_max_tiles(R, E, p.bm) * p.ntiles;
  finish_plan(p, E);
  if (p.bm == 256 && p.grid > kCus) p.grid += kTailBlocks;
  const int steps = (kd + kstep - 1) / kstep;
  const int unit = kstep == 64 ? 1 : kstep;             // (codes: pieces in whole blocks)
  if (p.bm <= 128 && p.grid > 0 && p.grid <= kDeepGrid / 2 && steps * kstep >= kSplitMinSteps * 64) {
    const int pieces = (int)std::min<int64_t>(kDeepGrid / p.grid, std::max(2, steps / 4));
    const int per = (steps + pieces - 1) / pieces;
    p.ksplit = (steps + per - 1) / per;
    p.klen = per * (kstep / unit);
    if (p.ksplit < 2) p.ksplit = p.klen = 0;
    else p.scan = true;
  }
  return p;
}

size_t grouped_row_partial_bytes(const GroupedPlan& p, int64_t R, int N) {
  return p.ksplit ? (size_t)p.ksplit * R * N * sizeof(float) : 0;
}

// A thread takes 8 columns of a row. Rows of no expert have no sums: zeros, or left as they are.
__global__ void __launch_bounds__(256) rows_join_kernel(const float* __restrict__ partial, int pieces, int R, int N,
                                                        const int32_t* __restrict__ offsets, int E, uint16_t* C,
                                                        int64_t ldc, int rest) {
  const int lane = threadIdx.x & 63;
  const int2 c = with_scan(offsets, E, R, lane, [&](const auto& scan) { return scan.covered(); });
  const int cpr = N / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)R * cpr) return;
  const int r = (int)(i / cpr), n = (int)(i - (int64_t)r * cpr) * 8;
  const bool own = r >= c.x && r < c.y;
  if (!own && !rest) return;
  f32x4 u{0.f, 0.f, 0.f, 0.f}, v = u;
  if (own) {
    const float* p = partial + (int64_t)r * N + n;
    const int64_t step = (int64_t)R * N;
#pragma unroll 4
    for (int k = 0; k < pieces; ++k, p += step) {
      u += *reinterpret_cast<const f32x4*>(p);
      v += *reinterpret_cast<const f32x4*>(p + 4);
    }
  }
  *reinterpret_cast<u32x4*>(C + (int64_t)r * ldc + n) =
      u32x4{cvt_pk_bf16(u[0], u[1]), cvt_pk_bf16(u[2], u[3]), cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
}

hipError_t launch_rows_join(const float* partial, const GroupedPlan& plan, int64_t R, int N, const int32_t* offsets,
                            int E, uint16_t* C, int64_t ldc, bool rest, hipStream_t st) {
  const int64_t blocks = (R * (N / 8) + 255) / 256;
  hipLaunchKernelGGL(rows_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, partial, plan.ksplit, (int)R, N,
                     offsets, E, C, ldc, rest);
  return hipGetLastError();
}

// A weight gradient of few tiles and many rows (less than half the CUs, 1024
// rows) sums pieces of each expert's rows side by side, as many as give every
// CU a workgroup, and joins them in row order: [640, 640] x 2 experts over
// 20000 rows 62 us in one piece each. Pieces are multiples of a k tile, 256 rows or more.
GroupedPlan grouped_wgrad_plan(int64_t R, int E, int M, int N, bool big) {
  GroupedPlan p{};
  const bool fits = up(M, 256) * up(N, 256) <= kBigPadding * up(M, 128) * up(N, 128);
  p.bm = big && (int64_t)E * ((M + 255) / 256) * ((N + 255) / 256) >= kBigTiles && fits ? 256 : 128;
  p.mtiles = (M + p.bm - 1) / p.bm;
  p.ntiles = (N + p.bm - 1) / p.bm;
  const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
  p.grid = E * tiles;
  if (p.bm == 128 && p.grid <= kDeepGrid / 2 && R >= 1024) {
    const int64_t pieces = kDeepGrid / tiles;
    p.split = (int)std::max<int64_t>(256, (R + pieces - 1) / pieces + 63) / 64 * 64;
    p.pieces = grouped_max_tiles(R, E, p.split);
    p.grid = p.pieces * tiles;
  }
  finish_plan(p, E);
  if (p.split) p.deep = p.scan = true;
  return p;
}

size_t grouped_partial_bytes(const GroupedPlan& p, int M, int N) {
  return p.split ? (size_t)p.pieces * M * N * sizeof(float) : 0;
}

// dW[e] = the sum of expert e's pieces, in row order (zero pieces: zeros), added
// to what it holds if asked. A thread takes 4 elements.
template <int OUT>
__global__ void __launch_bounds__(256) wgrad_join_kernel(const float* __restrict__ partial, const GroupedArgs P,
                                                         int64_t size, int blocks) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x / blocks;
  const int2 own = with_scan(P.offsets, P.E, P.R, lane, [&](const auto& scan) {
    int incl;
    scan.tiles(P.split, incl);
    return scan.tiles_of(e, P.split, incl);
  });
  const int first = own.x, n = own.y;
  if (n == 0 && P.accumulate) return;
  const int64_t i = ((int64_t)(blockIdx.x - e * blocks) * 256 + threadIdx.x) * 4;
  if (i >= size) return;
  const float* src = partial + first * size + i;
  f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < n; ++k) s += *reinterpret_cast<const f32x4*>(src + k * size);
  if constexpr (OUT == EPI_F32) {
    f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(P.C) + e * size + i);
    if (P.accumulate) s += *dst;
    *dst = s;
  } else {
    u32x2* dst = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(P.C) + e * size + i);
    if (P.accumulate) {
      const u32x2 o = *dst;
      s += f32x4{bf16_bits_to_f32(o.x & 0xFFFFu), bf16_bits_to_f32(o.x >> 16), bf16_bits_to_f32(o.y & 0xFFFFu),
                 bf16_bits_to_f32(o.y >> 16)};
    }
    *dst = u32x2{cvt_pk_bf16(s[0], s[1]), cvt_pk_bf16(s[2], s[3])};
  }
}

static GroupedArgs rows_args(const GroupedProduct& p, const GroupedPlan& plan, const GroupedScratch& s, bool rest) {
  GroupedArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.C = p.C;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.ldc = p.ldc;
  a.b_estride = p.estride;
  a.N = p.N;
  a.Kd = p.Kd;
  a.tiles = plan.scan ? nullptr : s.tiles;
  a.n_mtiles = s.n_mtiles;
  a.offsets = p.offsets;
  a.E = p.E;
  a.R = (int)p.R;
  a.rest_blocks = plan.scan && rest && !plan.ksplit ? kScanRestBlocks : 0;
  a.ntiles = plan.ntiles;
  if (plan.ksplit) {
    a.C = s.row_partial;
    a.ldc = p.N;
    a.c_estride = p.R * p.N;
    a.ksplit = plan.ksplit;
    a.klen = plan.klen;
  }
  return a;
}

// (a split gradient: of the launch that sums the pieces)
static GroupedArgs wgrad_args(const GroupedProduct& p, int M, bool accumulate, const GroupedPlan& plan,
                              const GroupedScratch& s) {
  GroupedArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.C = plan.split ? s.partial : p.C;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.ldc = plan.split ? p.N : p.ldc;
  a.c_estride = plan.split ? (int64_t)M * p.N : p.estride;
  a.M = M;
  a.N = p.N;
  a.ranges = plan.scan ? nullptr : s.ranges;
  a.offsets = p.offsets;
  a.E = p.E;
  a.R = (int)p.R;
  a.mtiles = plan.mtiles;
  a.ntiles = plan.ntiles;
  a.split = plan.split;
  a.accumulate = accumulate && !plan.split;
  return a;
}

static hipError_t launch_join(const GroupedProduct& p, int M, bool f32, bool accumulate, const GroupedPlan& plan,
                              const GroupedScratch& s, hipStream_t st) {
  GroupedArgs a = wgrad_args(p, M, false, plan, s);
  a.C = p.C;
  a.accumulate = accumulate;
  const int64_t size = (int64_t)M * p.N;
  const int blocks = (int)((size + 1023) / 1024);
  const dim3 grid((unsigned)((int64_t)p.E * blocks));
  if (f32) hipLaunchKernelGGL(wgrad_join_kernel<EPI_F32>, grid, dim3(256), 0, st, s.partial, a, size, blocks);
  else hipLaunchKernelGGL(wgrad_join_kernel<EPI_BF16>, grid, dim3(256), 0, st, s.partial, a, size, blocks);
  return hipGetLastError();
}

hipError_t launch_grouped_rows(const GroupedProduct& p, const GroupedPlan& plan, const GroupedScratch& s, bool rest,
                               hipStream_t st) {
  const GroupedArgs a = rows_args(p, plan, s, rest);
  const int64_t grid = plan.grid * std::max(1, plan.ksplit) + a.rest_blocks;
  if (p.transposed_b) launch_form<FORM_NN, EPI_BF16>(a, plan, grid, st);
  else launch_form<FORM_NT, EPI_BF16>(a, plan, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !plan.ksplit) return e;
  return launch_rows_join(s.row_partial, plan, p.R, p.N, p.offsets, p.E, static_cast<uint16_t*>(p.C), p.ldc, rest, st);
}

hipError_t launch_grouped_wgrad(const GroupedProduct& p, int M, bool f32, bool accumulate, const GroupedPlan& plan,
                                const GroupedScratch& s, hipStream_t st) {
  const GroupedArgs a = wgrad_args(p, M, accumulate, plan, s);
  if (f32 || plan.split) launch_form<FORM_TN, EPI_F32>(a, plan, plan.grid, st);
  else launch_form<FORM_TN, EPI_BF16>(a, plan, plan.grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !plan.split) return e;
  return launch_join(p, M, f32, accumulate, plan, s, st);
}

bool grouped_grad_in_one(const GroupedPlan& rows, const GroupedPlan& wgrad) {
  return rows.bm == wgrad.bm && rows.grid + wgrad.grid < kMaxGrid;
}

template <int BM, int BN, int WM, int WN, int OCC, int AST, int BST>
static void launch_grad_form(const GroupedArgs& a, const GroupedArgs& b, int g0, dim3 grid, bool wide, hipStream_t st) {
  constexpr int NT = 64 * WM * WN;
  if constexpr (BM == 128) {
    if (a.ksplit) {
      if (wide)
        hipLaunchKernelGGL((grouped_grad_kernel<BM, BN, WM, WN, OCC, EPI_F32, EPI_F32, AST, BST>), grid, dim3(NT), 0,
                           st, a, b, g0);
      else
        hipLaunchKernelGGL((grouped_grad_kernel<BM, BN, WM, WN, OCC, EPI_F32, EPI_BF16, AST, BST>), grid, dim3(NT), 0,
                           st, a, b, g0);
      return;
    }
  }
  if (wide)
    hipLaunchKernelGGL((grouped_grad_kernel<BM, BN, WM, WN, OCC, EPI_BF16, EPI_F32, AST, BST>), grid, dim3(NT), 0, st,
                       a, b, g0);
  else
    hipLaunchKernelGGL((grouped_grad_kernel<BM, BN, WM, WN, OCC, EPI_BF16, EPI_BF16, AST, BST>), grid, dim3(NT), 0, st,
                       a, b, g0);
}

hipError_t launch_grouped_grad(const GroupedProduct& dx, const GroupedPlan& rows, bool rest, const GroupedProduct& dw,
                               const GroupedPlan& wgrad, int M, bool f32, bool accumulate, const GroupedScratch& s,
                               hipStream_t st) {
  GroupedArgs a = rows_args(dx, rows, s, rest);
  const GroupedArgs b = wgrad_args(dw, M, accumulate, wgrad, s);
  a.before = (int)wgrad.grid;
  const int g0 = (int)wgrad.grid;
  const int64_t gx = rows.grid * std::max(1, rows.ksplit) + a.rest_blocks;
  const dim3 grid((unsigned)(g0 + gx));
  const bool deep = g0 + gx <= kDeepGrid;
  if (rows.bm == 256) launch_grad_form<256, 256, 2, 4, 2, 2, 3>(a, b, g0, grid, f32 || wgrad.split, st);
  else if (deep) launch_grad_form<128, 128, 2, 2, 1, 4, 4>(a, b, g0, grid, f32 || wgrad.split, st);
  else launch_grad_form<128, 128, 2, 2, 2, 2, 2>(a, b, g0, grid, f32 || wgrad.split, st);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && rows.ksplit)
    e = launch_rows_join(s.row_partial, rows, dx.R, dx.N, dx.offsets, dx.E, static_cast<uint16_t*>(dx.C), dx.ldc, rest,
                         st);
  if (e != hipSuccess || !wgrad.split) return e;
  return launch_join(dw, M, f32, accumulate, wgrad, s, st);
}

}  // namespace moe
