// C ABI of the operators around the layer: the grouped products and their
// gradients, the 8-bit products and quantisers, gradient norm and clipping.
// Argument checks, workspace carving and launch sequences; host code only.
#include "../../include/moe_api.h"

#include <algorithm>
#include <initializer_list>
#include <new>
#include <utility>
#include <vector>

#include "grouped_ops.h"

namespace {

using namespace moe;

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
bool ws_ok(const void* ws, size_t have, size_t need) {
  if (need == 0) return true;
  return ws != nullptr && have >= need && (reinterpret_cast<uintptr_t>(ws) % kAlign) == 0;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

constexpr int64_t kMaxBlocks = ((int64_t)1 << 28) - 16;   // 16 to a workgroup of 256 threads, whose number is 32 bits
constexpr int64_t kMaxStride = (int64_t)1 << 21;   // 256 rows of 2 bytes and their k offsets stay below 2 GiB
constexpr int64_t kMaxRows = (int64_t)1 << 30;     // row counts round up to whole tiles in 32 bits

// dims with the dense strides filled in
int grouped_dims(const moe_grouped_dims* in, moe_grouped_dims* d) {
  if (in == nullptr) return MOE_ERR_INVALID;
  *d = *in;
  if (d->R < 0 || d->E <= 0 || d->N <= 0 || d->K <= 0) return MOE_ERR_INVALID;
  if (d->ldx < 0 || d->ldy < 0 || d->ldw < 0 || d->w_stride < 0 || d->lddx < 0) return MOE_ERR_INVALID;
  if (d->ldx == 0) d->ldx = d->K;
  if (d->ldy == 0) d->ldy = d->N;
  if (d->ldw == 0) d->ldw = d->K;
  if (d->lddx == 0) d->lddx = d->K;
  const int64_t extent = (int64_t)(d->N - 1) * d->ldw + d->K;
  if (d->w_stride == 0) d->w_stride = (int64_t)d->N * d->ldw;
  if (d->ldx < d->K || d->ldy < d->N || d->ldw < d->K || d->lddx < d->K || d->w_stride < extent)
    return MOE_ERR_INVALID;
  if (d->E > kMaxExperts || d->R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if ((d->N | d->K) % 8 || (d->ldx | d->ldy | d->ldw | d->w_stride | d->lddx) % 8) return MOE_ERR_UNSUPPORTED;
  if (std::max(std::max(d->ldx, d->ldy), std::max(d->ldw, d->lddx)) >= kMaxStride) return MOE_ERR_UNSUPPORTED;
  if (grouped_rows_plan(d->R, d->E, d->N, d->K, 64).grid >= kMaxGrid ||
      grouped_rows_plan(d->R, d->E, d->N, d->K, 128).grid >= kMaxGrid ||
      grouped_rows_plan(d->R, d->E, d->K, d->N, 64).grid >= kMaxGrid)
    return MOE_ERR_UNSUPPORTED;
  if (grouped_wgrad_plan(d->R, d->E, d->N, d->K).grid >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Memory of a tensor: `rows` rows of `width` bytes, `pitch` apart.
struct Region {
  const void* p;
  int64_t rows, width, pitch;
};

// Whether two regions share memory (columns side by side in one matrix do not).
bool overlap(const Region& a, const Region& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t al = reinterpret_cast<uintptr_t>(a.p), bl = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ah = al + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t bh = bl + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (ah <= bl || bh <= al) return false;
  if (a.pitch != b.pitch) return true;
  const bool a_first = al <= bl;
  const int64_t at = (int64_t)((a_first ? bl - al : al - bl) % (uintptr_t)a.pitch);
  return at < (a_first ? a.width : b.width) || at + (a_first ? b.width : a.width) > a.pitch;
}
bool overlaps_any(const Region& out, std::initializer_list<Region> others) {
  for (const Region& o : others)
    if (overlap(out, o)) return true;
  return false;
}
Region rows_region(const void* p, int64_t R, int64_t cols, int64_t ld, int bytes) {
  return Region{p, R, cols * bytes, ld * bytes};
}
Region dense_region(const void* p, int64_t bytes) { return Region{p, 1, bytes, bytes}; }
Region weight_region(const void* w, const moe_grouped_dims& d) {
  return dense_region(w, ((d.E - 1) * d.w_stride + (int64_t)(d.N - 1) * d.ldw + d.K) * 2);
}
Region offsets_region(const int32_t* o, const moe_grouped_dims& d) { return dense_region(o, (int64_t)(d.E + 1) * 4); }

// Workspace of a call: the tile table of the products that need one, and what the call adds.
struct GroupedLayout {
  size_t n_mtiles, ranges, tiles, partial, row_partial, codes, scales, total;
};

GroupedLayout grouped_layout(const moe_grouped_dims& d, int table_bm, size_t partial, size_t row_partial,
                             bool quantise) {
  GroupedLayout l{};
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes); return at; };
  if (table_bm > 0) {
    l.n_mtiles = take(4);
    l.ranges = take((size_t)d.E * 8);
    l.tiles = take((size_t)grouped_max_tiles(d.R, d.E, table_bm) * 16);
  }
  if (partial > 0) l.partial = take(partial);
  if (row_partial > 0) l.row_partial = take(row_partial);
  if (quantise) {
    l.codes = take((size_t)d.R * d.K);
    l.scales = take((size_t)((d.K + 127) / 128) * d.R * 4);
  }
  l.total = o;
  return l;
}

GroupedScratch grouped_scratch(const GroupedLayout& l, void* ws) {
  char* p = static_cast<char*>(ws);
  return GroupedScratch{reinterpret_cast<int2*>(p + l.ranges), reinterpret_cast<int4*>(p + l.tiles),
                        reinterpret_cast<int32_t*>(p + l.n_mtiles), reinterpret_cast<float*>(p + l.partial),
                        reinterpret_cast<float*>(p + l.row_partial)};
}

int table_of(const GroupedPlan& p) { return p.scan ? 0 : p.bm; }

GroupedLayout forward_layout(const moe_grouped_dims& d, const GroupedPlan& p, bool quantise = false) {
  return grouped_layout(d, d.R > 0 ? table_of(p) : 0, 0, grouped_row_partial_bytes(p, d.R, d.N), quantise);
}

// Rows per expert up to which dW gives up its big tiles to share a launch with a
// dx of small ones. us, two launches / one: R 2000, E 20, [1000, 704] 34.4 / 28.3,
// 230 x 4, [1824, 2096] 36 / 30, 363 x 3, [1112, 2344] 28.4 / 25.1; 3000 x 3,
// [2048, 2048] 64 / 67.
constexpr int64_t kJointRows = 256;

struct GradPlans {
  GroupedPlan rows, wgrad;
  bool one;                  // dx and dw in one launch
  int table_bm;              // of the one table both use (the rows product's tiles; the gradient takes its ranges)
};

GradPlans grad_plans(const moe_grouped_dims& d, bool dx, bool dw) {
  GradPlans g{grouped_rows_plan(d.R, d.E, d.K, d.N, 64, false), grouped_wgrad_plan(d.R, d.E, d.N, d.K), false, 0};
  // one launch needs one tile size: few rows take the tile that is theirs, in a
  // launch of their own, unless both products are small
  const GroupedPlan alone = grouped_rows_plan(d.R, d.E, d.K, d.N, 64);
  if (dx && dw && g.rows.bm == 128 && g.wgrad.bm == 256 && d.R <= d.E * kJointRows) {
    const GroupedPlan small = grouped_wgrad_plan(d.R, d.E, d.N, d.K, false);
    if (g.rows.scan && small.scan) g.wgrad = small;
  }
  g.one = dx && dw && grouped_grad_in_one(g.rows, g.wgrad) &&
          (alone.bm == g.rows.bm || (g.rows.scan && g.wgrad.scan));
  if (!g.one) g.rows = alone;
  if ((dx && !g.rows.scan) || (dw && !g.wgrad.scan)) g.table_bm = g.rows.bm;
  return g;
}

GroupedLayout grad_layout(const moe_grouped_dims& d, const GradPlans& g, bool dx, bool dw) {
  return grouped_layout(d, g.table_bm, dw ? grouped_partial_bytes(g.wgrad, d.N, d.K) : 0,
                        dx ? grouped_row_partial_bytes(g.rows, d.R, d.K) : 0, false);
}

}  // namespace

extern "C" {

size_t moe_grouped_workspace_bytes(const moe_grouped_dims* dims) {
  moe_grouped_dims d;
  if (grouped_dims(dims, &d) != MOE_OK) return 0;
  size_t grad = kAlign;
  for (int outs = 1; outs <= 3; ++outs)                 // dx, dw, both: their plans differ
    grad = std::max(grad, grad_layout(d, grad_plans(d, outs & 1, outs & 2), outs & 1, outs & 2).total);
  const size_t q = d.K % 16 == 0 ? forward_layout(d, grouped_rows_plan(d.R, d.E, d.N, d.K, 128), true).total : 0;
  return std::max(std::max(forward_layout(d, grouped_rows_plan(d.R, d.E, d.N, d.K, 64)).total, q), grad);
}

int moe_grouped_matmul(const moe_grouped_dims* dims, const uint16_t* x, const uint16_t* w, const int32_t* offsets,
                       uint16_t* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_grouped_dims d;
  const int st = grouped_dims(dims, &d);
  if (st != MOE_OK) return st;
  if (!w || !offsets || (d.R > 0 && (!x || !y))) return MOE_ERR_INVALID;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y)) return MOE_ERR_INVALID;
  const GroupedPlan plan = grouped_rows_plan(d.R, d.E, d.N, d.K, 64);
  const GroupedLayout l = forward_layout(d, plan);
  if (!ws_ok(ws, ws_bytes, l.total)) return MOE_ERR_WORKSPACE;
  if (overlaps_any(rows_region(y, d.R, d.N, d.ldy, 2),
                   {rows_region(x, d.R, d.K, d.ldx, 2), weight_region(w, d), offsets_region(offsets, d)}))
    return MOE_ERR_INVALID;
  if (d.R == 0) return MOE_OK;
  const GroupedScratch s = grouped_scratch(l, ws);
  const RestRows rest{d.zero_rest ? y : nullptr, d.ldy, d.N};
  if (!plan.scan && launch_grouped_tiles(offsets, d.E, (int)d.R, plan.bm, s, rest, stream) != hipSuccess)
    return MOE_ERR_HIP;
  const GroupedProduct p{x, w, y, d.ldx, d.ldw, d.ldy, d.w_stride, d.R, d.E, d.N, d.K, false, offsets};
  return hip_status(launch_grouped_rows(p, plan, s, d.zero_rest != 0, stream));
}

int moe_grouped_matmul_grad(const moe_grouped_dims* dims, const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                            const int32_t* offsets, uint16_t* dx, void* dw, int32_t dw_dtype, int32_t accumulate,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_grouped_dims d;
  const int st = grouped_dims(dims, &d);
  if (st != MOE_OK) return st;
  if (!offsets || (!dx && !dw && d.R > 0)) return MOE_ERR_INVALID;
  if (dw_dtype != MOE_BF16 && dw_dtype != MOE_FP32) return MOE_ERR_INVALID;
  if (d.R > 0 && (!dy || (dx && !w) || (dw && !x))) return MOE_ERR_INVALID;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned16(dw)) return MOE_ERR_INVALID;
  const bool run_dx = dx && d.R > 0;
  const GradPlans plans = grad_plans(d, run_dx, dw != nullptr);
  const GroupedPlan &rows = plans.rows, &wg = plans.wgrad;
  const GroupedLayout l = grad_layout(d, plans, run_dx, dw != nullptr);
  if (!ws_ok(ws, ws_bytes, l.total)) return MOE_ERR_WORKSPACE;
  const Region rdy = rows_region(dy, d.R, d.N, d.ldy, 2), rx = rows_region(dw ? x : nullptr, d.R, d.K, d.ldx, 2);
  const Region rw = weight_region(run_dx ? w : nullptr, d), ro = offsets_region(offsets, d);
  const Region rdx = rows_region(run_dx ? dx : nullptr, d.R, d.K, d.lddx, 2);
  const Region rdw = dense_region(dw, (int64_t)d.E * d.N * d.K * (dw_dtype == MOE_FP32 ? 4 : 2));
  if (overlaps_any(rdx, {rdy, rx, rw, ro, rdw}) || overlaps_any(rdw, {rdy, rx, rw, ro})) return MOE_ERR_INVALID;
  const GroupedScratch s = grouped_scratch(l, ws);
  const RestRows rest{run_dx && !rows.scan && d.zero_rest ? dx : nullptr, d.lddx, d.K};
  if (plans.table_bm > 0)
    if (launch_grouped_tiles(offsets, d.E, (int)d.R, rows.bm, s, rest, stream) != hipSuccess) return MOE_ERR_HIP;
  const GroupedProduct px{dy, w, dx, d.ldy, d.ldw, d.lddx, d.w_stride, d.R, d.E, d.K, d.N, true, offsets};
  const GroupedProduct pw{dy, x, dw, d.ldy, d.ldx, d.K, (int64_t)d.N * d.K, d.R, d.E, d.K, 0, true, offsets};
  const bool f32 = dw_dtype == MOE_FP32, rest_rows = d.zero_rest != 0;
  if (plans.one)
    return hip_status(launch_grouped_grad(px, rows, rest_rows, pw, wg, d.N, f32, accumulate != 0, s, stream));
  if (run_dx && launch_grouped_rows(px, rows, s, rest_rows, stream) != hipSuccess) return MOE_ERR_HIP;
  if (dw && launch_grouped_wgrad(pw, d.N, f32, accumulate != 0, wg, s, stream) != hipSuccess) return MOE_ERR_HIP;
  return MOE_OK;
}

int moe_quantize_fp8_rows(const uint16_t* x, int64_t R, int32_t K, int64_t ldx, uint8_t* codes, float* scales,
                          hipStream_t stream) {
  if (R < 0 || K <= 0 || ldx < 0) return MOE_ERR_INVALID;
  if (ldx == 0) ldx = K;
  if (ldx < K || (R > 0 && (!x || !codes || !scales)) || !aligned16(x) || !aligned16(codes)) return MOE_ERR_INVALID;
  if (K % 8 || ldx % 8 || R > kMaxBlocks / ((K + 127) / 128)) return MOE_ERR_UNSUPPORTED;
  const Region rq = dense_region(codes, R * K), rs = dense_region(scales, R * ((K + 127) / 128) * 4);
  const Region rx = rows_region(x, R, K, ldx, 2);
  if (R > 0 && (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs))) return MOE_ERR_INVALID;
  return hip_status(launch_fp8_rows(x, R, K, ldx, codes, scales, stream));
}

int moe_quantize_fp8_blocks(const uint16_t* w, int64_t count, int32_t N, int32_t K, uint8_t* codes, float* scales,
                            hipStream_t stream) {
  if (count < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID;
  if ((count > 0 && (!w || !codes || !scales)) || !aligned16(w) || !aligned16(codes)) return MOE_ERR_INVALID;
  if (K % 8 || (int64_t)N * K > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  if (count >= (kMaxGrid * 2) / ((int64_t)((N + 127) / 128) * ((K + 127) / 128))) return MOE_ERR_UNSUPPORTED;
  const int64_t n = count * N * K;
  const Region rq = dense_region(codes, n), rw = dense_region(w, n * 2);
  const Region rs = dense_region(scales, count * ((N + 127) / 128) * ((K + 127) / 128) * 4);
  if (count > 0 && (overlap(rw, rq) || overlap(rw, rs) || overlap(rq, rs))) return MOE_ERR_INVALID;
  return hip_status(launch_fp8_blocks(w, count, N, K, codes, scales, stream));
}

}  // extern "C"

namespace {

// The 8-bit product of checked dims; codes and scales of the rows given, or x (bf16) to quantise into the workspace.
int fp8_impl(const moe_grouped_dims* dims, bool quantise, const uint16_t* x, const uint8_t* xq, const float* xs, const uint8_t* wq,
             const float* w_scale, const int32_t* offsets, uint16_t* y, void* ws, size_t ws_bytes,
             hipStream_t stream) {
  if (dims == nullptr) return MOE_ERR_INVALID;
  moe_grouped_dims d = *dims;
  d.ldw = d.w_stride = d.lddx = 0;                      // codes are dense
  if (!quantise) d.ldx = 0;
  const int st = grouped_dims(&d, &d);
  if (st != MOE_OK) return st;
  if (d.K % 16) return MOE_ERR_UNSUPPORTED;
  if (quantise && d.R > kMaxBlocks / ((d.K + 127) / 128)) return MOE_ERR_UNSUPPORTED;
  if (!wq || !w_scale || !offsets || (d.R > 0 && (!y || (quantise ? !x : !xq || !xs)))) return MOE_ERR_INVALID;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(wq) || !aligned16(y)) return MOE_ERR_INVALID;
  const GroupedPlan plan = grouped_rows_plan(d.R, d.E, d.N, d.K, 128);
  const GroupedLayout l = forward_layout(d, plan, quantise);
  if (!ws_ok(ws, ws_bytes, l.total)) return MOE_ERR_WORKSPACE;
  const int64_t kb = (d.K + 127) / 128, nb = (d.N + 127) / 128;
  if (overlaps_any(rows_region(y, d.R, d.N, d.ldy, 2),
                   {rows_region(x, d.R, d.K, d.ldx, 2), dense_region(xq, d.R * d.K), dense_region(xs, kb * d.R * 4),
                    dense_region(wq, (int64_t)d.E * d.N * d.K), dense_region(w_scale, d.E * nb * kb * 4),
                    offsets_region(offsets, d)}))
    return MOE_ERR_INVALID;
  if (d.R == 0) return MOE_OK;
  const GroupedScratch s = grouped_scratch(l, ws);
  const bool own = quantise && fp8_quantises(plan, d.R, d.K);
  if (quantise) {
    uint8_t* codes = static_cast<uint8_t*>(ws) + l.codes;
    float* scales = reinterpret_cast<float*>(static_cast<char*>(ws) + l.scales);
    if (!own && launch_fp8_rows(x, d.R, d.K, d.ldx, codes, scales, stream) != hipSuccess) return MOE_ERR_HIP;
    xq = codes;
    xs = scales;
  }
  const RestRows rest{!plan.scan && d.zero_rest ? y : nullptr, d.ldy, d.N};
  if (!plan.scan && launch_grouped_tiles(offsets, d.E, (int)d.R, plan.bm, s, rest, stream) != hipSuccess)
    return MOE_ERR_HIP;
  Fp8Args a{};
  a.A = xq;
  a.sx = xs;
  a.x = own ? x : nullptr;
  a.ldx = d.ldx;
  a.B = wq;
  a.sw = w_scale;
  a.C = y;
  a.ldc = d.ldy;
  a.R = d.R;
  a.N = d.N;
  a.K = d.K;
  a.nb = (int)nb;
  a.kb = (int)kb;
  a.tiles = plan.scan ? nullptr : s.tiles;
  a.n_mtiles = s.n_mtiles;
  a.offsets = offsets;
  a.E = d.E;
  a.rest_blocks = plan.scan && d.zero_rest && !plan.ksplit ? kScanRestBlocks : 0;
  a.ntiles = plan.ntiles;
  if (plan.ksplit) {
    a.C = s.row_partial;
    a.ldc = d.N;
    a.c_stride = d.R * d.N;
    a.ksplit = plan.ksplit;
    a.klen = plan.klen;
  }
  if (launch_grouped_fp8(a, plan, stream) != hipSuccess) return MOE_ERR_HIP;
  if (!plan.ksplit) return MOE_OK;
  return hip_status(launch_rows_join(s.row_partial, plan, d.R, d.N, offsets, d.E, y, d.ldy, d.zero_rest != 0, stream));
}

}  // namespace

extern "C" {

int moe_grouped_matmul_fp8(const moe_grouped_dims* dims, const uint8_t* xq, const float* xs, const uint8_t* wq,
                           const float* w_scale, const int32_t* offsets, uint16_t* y, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  return fp8_impl(dims, false, nullptr, xq, xs, wq, w_scale, offsets, y, ws, ws_bytes, stream);
}

int moe_grouped_matmul_fp8_rows(const moe_grouped_dims* dims, const uint16_t* x, const uint8_t* wq,
                                const float* w_scale, const int32_t* offsets, uint16_t* y, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  return fp8_impl(dims, true, x, nullptr, nullptr, wq, w_scale, offsets, y, ws, ws_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// gradient norm and clipping
// ---------------------------------------------------------------------------

namespace {

// workgroups of one launch: enough to fill the card eight deep, never more than chunks
constexpr int kGradBlocks = 2048;

size_t dtype_size(int32_t dt) { return dt == MOE_FP32 ? 4 : 2; }
int64_t chunks_of(int64_t n, int log2) { return (n + ((int64_t)1 << log2) - 1) >> log2; }

// Chunks of 2^11 elements (8 of a thread's 256 each) for few, so that they spread
// over the CUs, up to 2^20 for many: 4 to 8 to a workgroup and launch, which
// evens out the workgroups' shares (320 tensors in three launches, 1.6 GB: 1.09
// ms with 1.4 to a workgroup).
int chunk_log2(const moe_grad_tensor* t, int32_t count) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) total += t[i].n;
  const int64_t launches = (count + kGradTableSize - 1) / kGradTableSize;
  int log2 = 11;
  while (log2 < 20 && (total >> log2) > 8 * kGradBlocks * launches) ++log2;
  return log2;
}

int check_tensors(const moe_grad_tensor* t, int32_t count) {
  if (count < 0 || (count > 0 && t == nullptr)) return MOE_ERR_INVALID;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || (t[i].dtype != MOE_BF16 && t[i].dtype != MOE_FP32)) return MOE_ERR_INVALID;
    if (t[i].n == 0) continue;
    const size_t sz = dtype_size(t[i].dtype);
    if (t[i].grad == nullptr || reinterpret_cast<uintptr_t>(t[i].grad) % sz) return MOE_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(t[i].out) % sz) return MOE_ERR_INVALID;
    if (t[i].n > ((int64_t)1 << 40) - total) return MOE_ERR_UNSUPPORTED;
    total += t[i].n;
  }
  return MOE_OK;
}

// Calls f(table) for every launch's table of non-empty tensors, in order or from the last tensor to the first.
template <typename F>
int for_tables(const moe_grad_tensor* t, int32_t count, bool reverse, F&& f) {
  GradTable tab;
  tab.chunk_log2 = chunk_log2(t, count);
  auto clear = [&]() {
    tab.count = tab.chunks = 0;
    for (uint32_t& w : tab.f32) w = 0;
  };
  clear();
  auto flush = [&]() -> int {
    if (tab.count == 0) return MOE_OK;
    const int rc = f(tab);
    clear();
    return rc;
  };
  for (int32_t j = 0; j < count; ++j) {
    const moe_grad_tensor& g = t[reverse ? count - 1 - j : j];
    if (g.n == 0) continue;
    const int64_t c = chunks_of(g.n, tab.chunk_log2);   // at most 2^20 + 1
    if (tab.count == kGradTableSize || tab.chunks + c > 0x7FFFFFFF) {
      const int rc = flush();
      if (rc != MOE_OK) return rc;
    }
    const int k = tab.count++;
    tab.src[k] = g.grad;
    tab.dst[k] = g.out ? g.out : const_cast<void*>(g.grad);
    tab.n[k] = g.n;
    tab.first[k] = tab.chunks;
    if (g.dtype == MOE_FP32) tab.f32[k / 32] |= 1u << (k % 32);
    tab.chunks += (int)c;
  }
  return flush();
}

int table_blocks(const GradTable& t) { return std::min(t.chunks, kGradBlocks); }

// the partial sums' number: the workgroups of all launches
size_t partials_of(const moe_grad_tensor* t, int32_t count) {
  size_t n = 0;
  const int log2 = chunk_log2(t, count);
  int in_table = 0;
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const int64_t c = chunks_of(t[i].n, log2);
    if (in_table == kGradTableSize || chunks + c > 0x7FFFFFFF) {
      n += (size_t)std::min<int64_t>(chunks, kGradBlocks);
      in_table = 0;
      chunks = 0;
    }
    ++in_table;
    chunks += c;
  }
  return n + (size_t)std::min<int64_t>(chunks, kGradBlocks);
}

// Elements up to which one workgroup does all: the second launch costs the host
// more than the spread over the CUs saves. us of a clip, two launches / one: 1
// tensor of 8192 or 65536 elements 14.9 / 11.9, of 131072 14.9 / 15.8 (fp32 18.2);
// 16 tensors of 65536 together 22.4 / 19.5.
constexpr int64_t kGradOneMax = 65536;
bool grad_is_small(const moe_grad_tensor* t, int32_t count) {
  int64_t total = 0;
  int32_t some = 0;
  for (int32_t i = 0; i < count; ++i) {
    total += t[i].n;
    some += t[i].n > 0;
  }
  return some > 0 && some <= kGradTableSize && total <= kGradOneMax;
}

size_t grad_ws_bytes(size_t partials) { return align_up((partials + 1) * sizeof(double)); }

int norm_impl(const moe_grad_tensor* t, int32_t count, double max_norm, float* norm, bool clip, void* ws,
              size_t ws_bytes, hipStream_t stream) {
  if (norm == nullptr) return MOE_ERR_INVALID;
  const size_t n = partials_of(t, count);
  if (!ws_ok(ws, ws_bytes, grad_ws_bytes(n))) return MOE_ERR_WORKSPACE;
  if (grad_is_small(t, count))
    return for_tables(t, count, false, [&](const GradTable& tab) -> int {
      return hip_status(launch_grad_one(tab, max_norm, clip, norm, stream));
    });
  double* partial = static_cast<double*>(ws);
  size_t at = 0;
  const int rc = for_tables(t, count, false, [&](const GradTable& tab) -> int {
    const int blocks = table_blocks(tab);
    const hipError_t e = launch_grad_sumsq(tab, blocks, partial + at, stream);
    at += blocks;
    return hip_status(e);
  });
  if (rc != MOE_OK) return rc;
  if (!clip || n == 0) return hip_status(launch_grad_norm(partial, (int)n, norm, stream));
  float* out = norm;
  return for_tables(t, count, true, [&](const GradTable& tab) -> int {
    const hipError_t e = launch_grad_scale(tab, table_blocks(tab), partial, (int)n, max_norm, out, stream);
    out = nullptr;
    return hip_status(e);
  });
}

// Outputs (the norm is one) that overlap each other, or a gradient that is not the output's own.
bool outputs_overlap(const moe_grad_tensor* t, int32_t count, const float* norm) {
  struct Span { uintptr_t lo, hi; bool out; };
  std::vector<Span> v;
  v.reserve(2 * (size_t)count + 1);
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  if (norm) v.push_back({at, at + sizeof(float), true});
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), o = t[i].out ? reinterpret_cast<uintptr_t>(t[i].out) : g;
    const uintptr_t b = (uintptr_t)t[i].n * dtype_size(t[i].dtype);
    v.push_back({o, o + b, true});
    if (o != g) v.push_back({g, g + b, false});
  }
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  // sweep: the furthest end so far of outputs and of gradients
  uintptr_t out_hi = 0, in_hi = 0;
  for (const Span& s : v) {
    if (s.lo < out_hi || (s.out && s.lo < in_hi)) return true;
    if (s.out) out_hi = std::max(out_hi, s.hi);
    else in_hi = std::max(in_hi, s.hi);
  }
  return false;
}

}  // namespace

extern "C" {

size_t moe_grad_norm_workspace_bytes(const moe_grad_tensor* tensors, int32_t count) {
  if (check_tensors(tensors, count) != MOE_OK) return 0;
  return grad_ws_bytes(partials_of(tensors, count));
}

int moe_grad_norm(const moe_grad_tensor* tensors, int32_t count, float* norm, void* ws, size_t ws_bytes,
                  hipStream_t stream) {
  const int st = check_tensors(tensors, count);
  if (st != MOE_OK) return st;
  return norm_impl(tensors, count, 0.0, norm, false, ws, ws_bytes, stream);
}

int moe_clip_grad_norm(const moe_grad_tensor* tensors, int32_t count, float max_norm, float* norm, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  const int st = check_tensors(tensors, count);
  if (st != MOE_OK) return st;
  if (!(max_norm >= 0.f)) return MOE_ERR_INVALID;
  try {
    if (outputs_overlap(tensors, count, norm)) return MOE_ERR_INVALID;
  } catch (const std::bad_alloc&) {
    return MOE_ERR_WORKSPACE;
  }
  return norm_impl(tensors, count, (double)max_norm, norm, true, ws, ws_bytes, stream);
}

}  // extern "C"
