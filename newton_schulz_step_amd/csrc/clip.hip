// The global norm of many gradient tensors, and their clipping (gfx950).
//
//   sumsq = sum g^2 over all tensors, in 64 bits;  norm = sqrt(sumsq)
//   factor = min(1, max_norm / (norm + 1e-6));     out = g factor, rounded to out's type
// 64 bits keep squares of 1e20 and of 1e-30 and the sum of 2^36 of them; two operations per
// element at 64 bits stay behind the memory. Bound by memory: the gradients twice (the factor
// is known after the last one only), the results once. A launch takes up to 120 tensors by value;
// each workgroup finds its tensor from the first workgroups of all. 810 million fp32 gradients into
// bf16: 1450 us, 5.6 TB/s over both passes (a large copy reaches 5.1); loads past the caches 1477.
#include "fp8.hpp"
#include "layer.hpp"
#include "quant8.hpp"
#include "rows.hpp"

namespace muon {

// The tensor of workgroup b: the last one that does not begin behind it (empty ones are not in the list).
__device__ __forceinline__ int tensor_of(const ClipArgs& a, int b) {
  const int lane = threadIdx.x & 63;
  const unsigned long long lower = __ballot(lane < a.n && a.t[min(lane, a.n - 1)].first <= b);
  const unsigned long long upper = __ballot(lane + 64 < a.n && a.t[min(lane + 64, a.n - 1)].first <= b);
  return __builtin_amdgcn_readfirstlane(__popcll(lower) + __popcll(upper) - 1);
}

constexpr int kClipThreads = 256, kClipStep = kClipThreads * 8;

template <int DT>
__device__ __forceinline__ double chunk_sumsq(const void* p, int64_t lo, int64_t hi) {
  double s0 = 0.0, s1 = 0.0;
  for (int64_t i0 = lo + threadIdx.x * 8; i0 < hi; i0 += 4 * kClipStep) {
    Raw8<DT> x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kClipStep;
      const int n = static_cast<int>(max<int64_t>(0, min<int64_t>(8, hi - i)));
      x[u].load(p, n > 0 ? i : 0, n);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const double v = x[u].get(e), w = x[u].get(e + 1);
        s0 = fma(v, v, s0);
        s1 = fma(w, w, s1);
      }
  }
  return s0 + s1;
}

__global__ __launch_bounds__(kClipThreads) void grad_sumsq_kernel(ClipArgs a) {
  __shared__ double part[kClipThreads / 64];
  const int b = static_cast<int>(blockIdx.x);
  const ClipTensor& t = a.t[tensor_of(a, b)];
  const int64_t lo = static_cast<int64_t>(b - t.first) * a.chunk, hi = min(t.n, lo + a.chunk);
  double s;
  if (t.in_dtype == MUON_DTYPE_F32) s = chunk_sumsq<MUON_DTYPE_F32>(t.in, lo, hi);
  else if (t.in_dtype == MUON_DTYPE_BF16) s = chunk_sumsq<MUON_DTYPE_BF16>(t.in, lo, hi);
  else s = chunk_sumsq<MUON_DTYPE_F16>(t.in, lo, hi);
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[b] = part[0] + part[1] + part[2] + part[3];
}

__global__ __launch_bounds__(1024) void sum_partials_kernel(const double* partial, int64_t n, int accumulate, double* out) {
  __shared__ double part[16];
  double s = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += partial[i];
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < 16; ++w) s += part[w];
    *out = accumulate ? *out + s : s;
  }
}

// The factor as two floats: one below fp32's normal numbers would lose bits, so that 2^-100 of it is
// apart there (1 otherwise). A value that the first product takes out of the normal numbers ends as 0.
struct Factor {
  float first, second;
  __device__ __forceinline__ float of(float x) const { return x * first * second; }
};

template <int IT, int OT>
__device__ __forceinline__ void chunk_scale(const void* p, void* o, int64_t lo, int64_t hi, Factor factor) {
  for (int64_t i0 = lo + threadIdx.x * 8; i0 < hi; i0 += 4 * kClipStep) {
    Raw8<IT> x[4];
    int n[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kClipStep;
      n[u] = static_cast<int>(max<int64_t>(0, min<int64_t>(8, hi - i)));
      x[u].load(p, n[u] > 0 ? i : 0, n[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = factor.of(x[u].get(e));
      write8<OT>(o, i0 + u * kClipStep, n[u], v);
    }
  }
}

template <int IT>
__device__ __forceinline__ void scale_to(int dtype, const void* p, void* o, int64_t lo, int64_t hi, Factor factor) {
  if (dtype == MUON_DTYPE_F32) chunk_scale<IT, MUON_DTYPE_F32>(p, o, lo, hi, factor);
  else if (dtype == MUON_DTYPE_BF16) chunk_scale<IT, MUON_DTYPE_BF16>(p, o, lo, hi, factor);
  else chunk_scale<IT, MUON_DTYPE_F16>(p, o, lo, hi, factor);
}

__global__ __launch_bounds__(kClipThreads) void grad_clip_kernel(ClipArgs a) {
  const double norm = sqrt(*a.sumsq);
  const double ratio = static_cast<double>(a.max_norm) / (norm + 1e-6);
  const bool never = a.max_norm == __builtin_huge_valf();
  const double limited = ratio > 1.0 || never ? 1.0 : ratio;   // NaN stays
  const bool small = limited < 0x1p-126;
  const Factor factor{small ? 0x1p-100f : 1.0f, static_cast<float>(small ? limited * 0x1p100 : limited)};
  if (a.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(norm);
  // last chunks first: those that the norm read last may still lie in the last-level cache
  const int b = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  if (b >= a.blocks) return;
  const ClipTensor& t = a.t[tensor_of(a, b)];
  if (t.in == t.out && factor.second == 1.0f) return;
  const int64_t lo = static_cast<int64_t>(b - t.first) * a.chunk, hi = min(t.n, lo + a.chunk);
  if (t.in_dtype == MUON_DTYPE_F32) scale_to<MUON_DTYPE_F32>(t.out_dtype, t.in, t.out, lo, hi, factor);
  else if (t.in_dtype == MUON_DTYPE_BF16) scale_to<MUON_DTYPE_BF16>(t.out_dtype, t.in, t.out, lo, hi, factor);
  else scale_to<MUON_DTYPE_F16>(t.out_dtype, t.in, t.out, lo, hi, factor);
}

hipError_t launch_grad_sumsq(const ClipArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(grad_sumsq_kernel, dim3(a.blocks), dim3(kClipThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_sum_partials(const double* partial, int64_t n, bool accumulate, double* out, hipStream_t s) {
  hipLaunchKernelGGL(sum_partials_kernel, dim3(1), dim3(1024), 0, s, partial, n, accumulate ? 1 : 0, out);
  return hipGetLastError();
}
hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(grad_clip_kernel, dim3(std::max(1, a.blocks)), dim3(kClipThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
