// The global norm of many gradient tensors, and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2);  out = g * (max_norm / norm) where norm > max_norm
//
// Bound by HBM: the gradients are read once for the norm and, where it passes
// the bound, once more to be scaled (the norm is needed before the first of
// them can be). Squares are summed in float64: no finite gradient overflows,
// and the sum of 10^10 terms keeps every bit of the fp32 result. The order of
// the sums is fixed by the sizes alone (a thread's own elements, the wave, the
// workgroup, then the workgroups' partials in order), so a call repeats bit
// for bit.
//
// Small lists are one launch of one workgroup, whose waves take the chunks.
//
// The tensors' addresses travel in the kernel arguments (kGradTableSize a
// launch): nothing is copied to the device, and nothing of them is kept.
#include "grouped_ops.h"

namespace moe {

constexpr int kGradThreads = 256;

__device__ __forceinline__ double block_sum_f64(double v, double* part) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  double s = part[0];
  for (int w = 1; w < (int)blockDim.x / kWave; ++w) s += part[w];
  __syncthreads();
  return s;
}

__device__ __forceinline__ double sq2(uint32_t w) {
  const double a = (double)bf16_bits_to_f32(w & 0xFFFFu), b = (double)bf16_bits_to_f32(w >> 16);
  return a * a + b * b;
}

// the table entry that holds chunk c: the last one that starts at or before it
template <int SIZE>
__device__ __forceinline__ int grad_entry(const GradTableOf<SIZE>& t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// elements of a chunk that come before its first 16-byte boundary
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int mis = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return min(mis, n);
}

// a thread's part of the sum of squares, thread tid of the NT of group `block` of `blocks`
template <int NT, int SIZE>
__device__ __forceinline__ double sum_squares(const GradTableOf<SIZE>& t, int tid, int block, int blocks) {
  double s = 0.0;
  for (int c = block; c < t.chunks; c += blocks) {
    const int i = grad_entry(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) << t.chunk_log2;
    const int n = (int)min((int64_t)1 << t.chunk_log2, t.n[i] - at);
    if ((t.f32[i >> 5] >> (i & 31)) & 1) {
      const float* p = static_cast<const float*>(t.src[i]) + at;
      const int h = head_of(p, n), nv = (n - h) / 4, tail = h + nv * 4;
      const f32x4* v = reinterpret_cast<const f32x4*>(p + h);
      for (int j = tid; j < nv; j += NT) {
        const f32x4 q = v[j];
        s += (double)q[0] * q[0] + (double)q[1] * q[1] + (double)q[2] * q[2] + (double)q[3] * q[3];
      }
      if (tid < h) s += (double)p[tid] * p[tid];
      if (tail + tid < n) s += (double)p[tail + tid] * p[tail + tid];
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.src[i]) + at;
      const int h = head_of(p, n), nv = (n - h) / 8, tail = h + nv * 8;
      const u32x4* v = reinterpret_cast<const u32x4*>(p + h);
      for (int j = tid; j < nv; j += NT) {
        const u32x4 q = v[j];
        s += sq2(q[0]) + sq2(q[1]) + sq2(q[2]) + sq2(q[3]);
      }
      if (tid < h) s += sq2(p[tid]);
      if (tail + tid < n) s += sq2(p[tail + tid]);
    }
  }
  return s;
}

template <int SIZE>
__global__ void __launch_bounds__(kGradThreads) grad_sumsq_kernel(const GradTableOf<SIZE> t,
                                                                  double* __restrict__ partial) {
  __shared__ double part[kGradThreads / kWave];
  const double s = block_sum_f64(sum_squares<kGradThreads>(t, threadIdx.x, blockIdx.x, gridDim.x), part);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// the sum of a call's partials, the same in every workgroup that takes it
template <int THREADS>
__device__ __forceinline__ double sum_partials(const double* partial, int n, double* part) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) s += partial[i];
  return block_sum_f64(s, part);
}

__global__ void __launch_bounds__(1024) grad_norm_kernel(const double* __restrict__ partial, int n,
                                                         float* __restrict__ norm) {
  __shared__ double part[16];
  const double s = sum_partials<1024>(partial, n, part);
  if (threadIdx.x == 0) *norm = (float)__builtin_sqrt(s);
}

// out = g * (max_norm / norm) where norm passes max_norm, else g. The chunks are
// walked from the last to the first, as the end of what the first pass read is
// what the caches still hold.
template <int NT, int SIZE>
__device__ __forceinline__ void scale_gradients(const GradTableOf<SIZE>& t, double norm, double max_norm, int tid,
                                                int block, int blocks) {
  // a norm that is not finite leaves the gradients as they are
  const double f = norm > max_norm && norm < __builtin_inf() ? max_norm / norm : 1.0;
  for (int c = t.chunks - 1 - block; c >= 0; c -= blocks) {
    const int i = grad_entry(t, c);
    if (f == 1.0 && t.src[i] == t.dst[i]) continue;      // in place and nothing to scale
    const int64_t at = (int64_t)(c - t.first[i]) << t.chunk_log2;
    const int n = (int)min((int64_t)1 << t.chunk_log2, t.n[i] - at);
    if ((t.f32[i >> 5] >> (i & 31)) & 1) {
      const float* p = static_cast<const float*>(t.src[i]) + at;
      float* o = static_cast<float*>(t.dst[i]) + at;
      const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
      const int h = same ? head_of(p, n) : n, nv = (n - h) / 4, tail = h + nv * 4;
      for (int j = tid; j < nv; j += NT) {
        f32x4 q = reinterpret_cast<const f32x4*>(p + h)[j];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = (float)((double)q[k] * f);
        reinterpret_cast<f32x4*>(o + h)[j] = q;
      }
      for (int j = tid; j < h; j += NT) o[j] = (float)((double)p[j] * f);
      for (int j = tail + tid; j < n; j += NT) o[j] = (float)((double)p[j] * f);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.src[i]) + at;
      uint16_t* o = static_cast<uint16_t*>(t.dst[i]) + at;
      const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
      const int h = same ? head_of(p, n) : n, nv = (n - h) / 8, tail = h + nv * 8;
      auto one = [&](uint32_t b) { return (float)((double)bf16_bits_to_f32(b) * f); };
      for (int j = tid; j < nv; j += NT) {
        u32x4 q = reinterpret_cast<const u32x4*>(p + h)[j];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = cvt_pk_bf16(one(q[k] & 0xFFFFu), one(q[k] >> 16));
        reinterpret_cast<u32x4*>(o + h)[j] = q;
      }
      for (int j = tid; j < h; j += NT) o[j] = (uint16_t)cvt_pk_bf16(one(p[j]), 0.f);
      for (int j = tail + tid; j < n; j += NT) o[j] = (uint16_t)cvt_pk_bf16(one(p[j]), 0.f);
    }
  }
}

// Every workgroup sums the partials itself (16 KB, from the L2): no launch
// between the two passes.
template <int SIZE>
__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const GradTableOf<SIZE> t,
                                                                  const double* __restrict__ partial, int np,
                                                                  double max_norm, float* __restrict__ norm_out) {
  __shared__ double part[kGradThreads / kWave];
  const double norm = __builtin_sqrt(sum_partials<kGradThreads>(partial, np, part));
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  scale_gradients<kGradThreads>(t, norm, max_norm, threadIdx.x, blockIdx.x, gridDim.x);
}

// Few elements (kGradOneMax, ops_api.hip): one workgroup does both passes, a chunk a wave.
template <int SIZE>
__global__ void __launch_bounds__(1024) grad_one_kernel(const GradTableOf<SIZE> t, double max_norm, int clip,
                                                        float* __restrict__ norm_out) {
  __shared__ double part[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const double norm = __builtin_sqrt(block_sum_f64(sum_squares<kWave>(t, lane, wave, 16), part));
  if (threadIdx.x == 0) *norm_out = (float)norm;
  if (clip) scale_gradients<kWave>(t, norm, max_norm, lane, wave, 16);
}

static GradTableOf<kGradShortTable> short_table(const GradTable& t) {
  GradTableOf<kGradShortTable> s{};
  for (int i = 0; i < t.count; ++i) {
    s.src[i] = t.src[i];
    s.dst[i] = t.dst[i];
    s.n[i] = t.n[i];
    s.first[i] = t.first[i];
  }
  s.f32[0] = t.f32[0];
  s.count = t.count;
  s.chunks = t.chunks;
  s.chunk_log2 = t.chunk_log2;
  return s;
}

hipError_t launch_grad_sumsq(const GradTable& t, int blocks, double* partial, hipStream_t st) {
  if (t.count <= kGradShortTable)
    hipLaunchKernelGGL(grad_sumsq_kernel<kGradShortTable>, dim3(blocks), dim3(kGradThreads), 0, st, short_table(t),
                       partial);
  else
    hipLaunchKernelGGL(grad_sumsq_kernel<kGradTableSize>, dim3(blocks), dim3(kGradThreads), 0, st, t, partial);
  return hipGetLastError();
}
hipError_t launch_grad_one(const GradTable& t, double max_norm, bool clip, float* norm, hipStream_t st) {
  if (t.count <= kGradShortTable)
    hipLaunchKernelGGL(grad_one_kernel<kGradShortTable>, dim3(1), dim3(1024), 0, st, short_table(t), max_norm, clip,
                       norm);
  else
    hipLaunchKernelGGL(grad_one_kernel<kGradTableSize>, dim3(1), dim3(1024), 0, st, t, max_norm, clip, norm);
  return hipGetLastError();
}
hipError_t launch_grad_norm(const double* partial, int n, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(1024), 0, st, partial, n, norm);
  return hipGetLastError();
}
hipError_t launch_grad_scale(const GradTable& t, int blocks, const double* partial, int n, double max_norm, float* norm,
                             hipStream_t st) {
  if (t.count <= kGradShortTable)
    hipLaunchKernelGGL(grad_scale_kernel<kGradShortTable>, dim3(blocks), dim3(kGradThreads), 0, st, short_table(t),
                       partial, n, max_norm, norm);
  else
    hipLaunchKernelGGL(grad_scale_kernel<kGradTableSize>, dim3(blocks), dim3(kGradThreads), 0, st, t, partial, n,
                       max_norm, norm);
  return hipGetLastError();
}

}  // namespace moe
