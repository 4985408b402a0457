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
                                                             int32_t* __restrict__ n_mtiles,
                                                             int32_t* __restrict__ counters, const RestRows rest) {
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
  if (blockIdx.x == 0 && tid < kGemmCounters) counters[tid] = 0;
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
  if (tid < E) {
    ranges[tid] = make_int2(lo, hi);
    if (tiles != nullptr)
      for (int i = 0; i < nt; ++i) tiles[first + i] = make_int4(tid, first, lo, hi);
  }
  if (tid == E - 1) *n_mtiles = first + nt;
}

hipError_t launch_grouped_tiles(const int32_t* offsets, int E, int R, int BM, const GroupedScratch& s,
                                const RestRows& rest, hipStream_t st) {
  hipLaunchKernelGGL(grouped_tiles_kernel, dim3(rest.C && R > 0 ? 1 + kRestBlocks : 1), dim3(1024), 0, st, offsets, E, R,
                     BM, s.ranges, s.tiles, s.n_mtiles, s.counters, rest);
  return hipGetLastError();
}

#ifndef GT_BIG
#define GT_BIG 2
#endif
#ifndef GT_BST
#define GT_BST 3
#endif
template <int FORM, int OUT>
static void launch_form(const GroupedArgs& a, int BM, int64_t grid, hipStream_t st) {
  if (BM == 256) {
#if GT_BIG == 1
    hipLaunchKernelGGL((grouped_kernel<FORM, 256, 256, 2, 2, 1, OUT, GT_BST>), dim3((unsigned)grid), dim3(256), 0, st, a);
#else
    hipLaunchKernelGGL((grouped_kernel<FORM, 256, 256, 2, 4, 2, OUT, GT_BST>), dim3((unsigned)grid), dim3(512), 0, st, a);
#endif
  } else
    hipLaunchKernelGGL((grouped_kernel<FORM, 128, 128, 2, 2, 2, OUT, 2>), dim3((unsigned)grid), dim3(256), 0, st, a);
}

// Which tiles, from what the host knows (the rows' number, not how they spread).
// 256-row tiles where an expert has 128 rows or more on average; else 128.
int grouped_bm(int64_t R, int E) { return R >= (int64_t)E * 128 ? 256 : 128; }

// Grids of at most this many workgroups find their tiles in the offsets
// (OffsetScan) and need no table.
constexpr int64_t kScanGrid = 1024;
constexpr int kScanExperts = 128;

GroupedPlan grouped_rows_plan(int64_t R, int E, int N) {
  GroupedPlan p;
  p.bm = grouped_bm(R, E);
  p.mtiles = 0;
  p.ntiles = (N + p.bm - 1) / p.bm;
  p.grid = grouped_max_tiles(R, E, p.bm) * p.ntiles;
  p.scan = p.grid <= kScanGrid && E <= kScanExperts;
  return p;
}

GroupedPlan grouped_wgrad_plan(int E, int M, int N) {
  GroupedPlan p;
  p.bm = (int64_t)E * ((M + 255) / 256) * ((N + 255) / 256) >= 256 ? 256 : 128;
  p.mtiles = (M + p.bm - 1) / p.bm;
  p.ntiles = (N + p.bm - 1) / p.bm;
  p.grid = (int64_t)E * p.mtiles * p.ntiles;
  p.scan = p.grid <= kScanGrid && E <= kScanExperts;
  return p;
}

hipError_t launch_grouped_rows(const GroupedProduct& p, const GroupedPlan& plan, const GroupedScratch& s, bool rest,
                               hipStream_t st) {
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
  a.rest_blocks = plan.scan && rest ? kScanRestBlocks : 0;
  a.ntiles = plan.ntiles;
  if (plan.grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int64_t grid = plan.grid + a.rest_blocks;
  if (p.transposed_b) launch_form<FORM_NN, EPI_BF16>(a, plan.bm, grid, st);
  else launch_form<FORM_NT, EPI_BF16>(a, plan.bm, grid, st);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedProduct& p, int M, bool f32, bool accumulate, const GroupedPlan& plan,
                                const GroupedScratch& s, hipStream_t st) {
  GroupedArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.C = p.C;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.ldc = p.ldc;
  a.c_estride = p.estride;
  a.M = M;
  a.N = p.N;
  a.ranges = plan.scan ? nullptr : s.ranges;
  a.offsets = p.offsets;
  a.E = p.E;
  a.R = (int)p.R;
  a.mtiles = plan.mtiles;
  a.ntiles = plan.ntiles;
  a.accumulate = accumulate;
  if (plan.grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (f32) launch_form<FORM_TN, EPI_F32>(a, plan.bm, plan.grid, st);
  else launch_form<FORM_TN, EPI_BF16>(a, plan.bm, plan.grid, st);
  return hipGetLastError();
}

}  // namespace moe
