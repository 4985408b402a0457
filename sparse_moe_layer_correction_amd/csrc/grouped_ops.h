// Private declarations shared by the expert operators' kernels and their C ABI layer.
#pragma once

#include "kernels.h"

namespace moe {

// Device scratch of one grouped call.
struct GroupedScratch {
  int2* ranges;        // [E] rows of each expert
  int4* tiles;         // [grouped_max_tiles] M tile table
  int32_t* n_mtiles;   // [1]
  float* partial;      // sums of the pieces of a split weight gradient
  float* row_partial;  // sums of the pieces of a split rows product
};

// M tiles that R rows in E experts can need
inline int64_t grouped_max_tiles(int64_t R, int E, int BM) { return R / BM + (R < E ? R : E); }

struct GroupedProduct {
  const uint16_t *A, *B;
  void* C;
  int64_t lda, ldb, ldc;
  int64_t estride;     // experts' B (rows products), experts' C (wgrad)
  int64_t R;
  int E, N, Kd;
  bool transposed_b;   // B stored [Kd, N]
  const int32_t* offsets;
};

// a grid's threads are counted in 32 bits; workgroups have up to 512
constexpr int64_t kMaxGrid = (int64_t)1 << 23;

// Tiles and grid of one product.
struct GroupedPlan {
  int bm, mtiles, ntiles;
  int64_t grid;
  int ksplit, klen;    // rows products: pieces of the reduction (0: none) and their length (codes: in blocks)
  int64_t pieces;      // split: the most pieces the rows can make
  int split;           // wgrad: rows of a piece, 0 for whole experts
  bool deep;           // four LDS stages
  bool scan;           // the kernel finds its tiles itself; else it needs launch_grouped_tiles
};
constexpr int kScanRestBlocks = 16;   // workgroups that zero the rows of no expert, without a table
// kd: the reduction's length; kstep: of a k tile (64, or 128 codes); few: the tile for few rows may be taken
GroupedPlan grouped_rows_plan(int64_t R, int E, int N, int kd, int kstep, bool few = true);
// big: 256 x 256 tiles may be taken
GroupedPlan grouped_wgrad_plan(int64_t R, int E, int M, int N, bool big = true);
size_t grouped_partial_bytes(const GroupedPlan& p, int M, int N);
size_t grouped_row_partial_bytes(const GroupedPlan& p, int64_t R, int N);
// C = the sum of a split rows product's pieces, over the rows of experts; rest: zero the others
hipError_t launch_rows_join(const float* partial, const GroupedPlan& plan, int64_t R, int N, const int32_t* offsets,
                            int E, uint16_t* C, int64_t ldc, bool rest, hipStream_t st);

// Output whose rows of no expert are to be zeroed (C null: none).
struct RestRows {
  uint16_t* C;
  int64_t ldc;
  int N;               // multiple of 8
};

hipError_t launch_grouped_tiles(const int32_t* offsets, int E, int R, int BM, const GroupedScratch& s,
                                const RestRows& rest, hipStream_t st);
// rest: without a table, also zero C's rows of no expert
hipError_t launch_grouped_rows(const GroupedProduct& p, const GroupedPlan& plan, const GroupedScratch& s, bool rest,
                               hipStream_t st);
hipError_t launch_grouped_wgrad(const GroupedProduct& p, int M, bool f32, bool accumulate, const GroupedPlan& plan,
                                const GroupedScratch& s, hipStream_t st);

// whether one launch can do dx and dW (one tile size)
bool grouped_grad_in_one(const GroupedPlan& rows, const GroupedPlan& wgrad);
hipError_t launch_grouped_grad(const GroupedProduct& dx, const GroupedPlan& rows, bool rest, const GroupedProduct& dw,
                               const GroupedPlan& wgrad, int M, bool f32, bool accumulate, const GroupedScratch& s,
                               hipStream_t st);

// E4M3 codes, one scale per 128 (fp8.h)
struct Fp8Args {
  const uint8_t* A;            // [R, K] codes of the rows
  const float* sx;             // [kb, R]
  const uint16_t* x;           // 32-row tiles: not null, the bf16 rows (row stride ldx) that A and sx are made of first
  int64_t ldx;
  const uint8_t* B;            // [E, N, K] codes of the weights
  const float* sw;             // [E, nb, kb]
  void* C;                     // bf16, or (a split reduction) the pieces' fp32 sums
  int64_t ldc, R;
  int64_t c_stride;
  int ksplit, klen;            // pieces of the reduction (0: none), their length in blocks of 128
  int N, K, nb, kb;
  const int4* tiles;           // null: found in the offsets
  const int32_t* n_mtiles;
  const int32_t* offsets;
  int E, rest_blocks;
  int ntiles;
};
hipError_t launch_fp8_rows(const uint16_t* x, int64_t R, int K, int64_t ldx, uint8_t* codes, float* scales,
                           hipStream_t st);
hipError_t launch_fp8_blocks(const uint16_t* w, int64_t count, int N, int K, uint8_t* codes, float* scales,
                             hipStream_t st);
// whether the product quantises its rows itself
bool fp8_quantises(const GroupedPlan& plan, int64_t R, int K);
hipError_t launch_grouped_fp8(const Fp8Args& a, const GroupedPlan& plan, hipStream_t st);

// Gradient tensors of one launch; entry i's chunks of 2^chunk_log2 elements are
// first[i] .. first[i + 1] of the launch's (the last entry's end at chunks). The
// table is a kernel argument: few tensors take the short one.
constexpr int kGradTableSize = 120, kGradShortTable = 16;
template <int SIZE>
struct GradTableOf {
  const void* src[SIZE];
  void* dst[SIZE];
  int64_t n[SIZE];
  int first[SIZE];
  uint32_t f32[(SIZE + 31) / 32];   // bit i: entry i is fp32, else bf16
  int count, chunks, chunk_log2;
};
typedef GradTableOf<kGradTableSize> GradTable;
static_assert(sizeof(GradTable) <= 4000, "kernel arguments");
hipError_t launch_grad_sumsq(const GradTable& t, int blocks, double* partial, hipStream_t st);
// the norm and (clip) the scaled gradients of one table by one workgroup
hipError_t launch_grad_one(const GradTable& t, double max_norm, bool clip, float* norm, hipStream_t st);
hipError_t launch_grad_norm(const double* partial, int n, float* norm, hipStream_t st);
// norm: where to write the norm (one launch of a call does), or null
hipError_t launch_grad_scale(const GradTable& t, int blocks, const double* partial, int n, double max_norm, float* norm,
                             hipStream_t st);

}  // namespace moe
