// RMS norm of rows with the residual's addition and an output in 8 bits, and its gradient
// (gfx950).
//
//   s = x + r, rounded to the rows' type;   rstd = (mean(s^2) + eps)^(-1/2);   y = s rstd w
// With n = s rstd and g = dy w the gradient is
//   dx = rstd (g - n mean(g n)) + ds,   dw = sum over rows of dy n.
// Sums are in fp32 or more, in a fixed order. Bound by memory: every row is read once into registers,
// a team of 1, 4 or 8 waves per row, eight columns per lane and load. 8192 x 4096 bf16 rows
// with residual, sum and 8-bit output: 41 us (5.7 TB/s; a large copy reaches 5.1); gradient of
// 16383 x 2048 with the residual stream's: 52 us (5.2 TB/s), of which 5 join the weight's.
#include "fp8.hpp"
#include "layer.hpp"
#include "quant8.hpp"
#include "rows.hpp"

namespace muon {

__device__ __forceinline__ void read8_as(int dtype, const void* p, int64_t i, int n, float (&v)[8]) {
  if (dtype == MUON_DTYPE_F32) read8<MUON_DTYPE_F32>(p, i, n, v);
  else if (dtype == MUON_DTYPE_BF16) read8<MUON_DTYPE_BF16>(p, i, n, v);
  else read8<MUON_DTYPE_F16>(p, i, n, v);
}

// v rounded to the type DT and back.
template <int DT>
__device__ __forceinline__ void round8(float (&v)[8]) {
  if constexpr (DT != MUON_DTYPE_F32) {
    using T = std::conditional_t<DT == MUON_DTYPE_BF16, __bf16, _Float16>;
    T o[8];
    rne<T, 8>(v, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(o[e]);
  }
}

// The sum over a team's lanes, in all of them. `scratch`: a float per wave of the workgroup.
template <int WAVES, typename T = float>
__device__ __forceinline__ T team_sum(float v, float* scratch) {
  v = wave_sum(v);
  T sum = v;
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += scratch[w];
    __syncthreads();
  }
  return sum;
}

// x^(-1/2), rounded once: the instruction's, off by a last bit, and a step of Newton's in 64 bits. The last bits of
// rstd decide the ties of the 8-bit values (rstd of 8192 x 4096 rows off by 2.8e-8 in the mean; by a root and a division
// in fp32 3.5e-8; the same time).
__device__ __forceinline__ float inverse_root(double x) {
  const float r = rsqrtf(static_cast<float>(x));
  const double d = r, next = d * (1.5 - 0.5 * x * d * d);
  return r > 0.0f && r <= 3.402823466e38f ? static_cast<float>(next) : r;   // 0, infinity and NaN stay
}

// How rows end: filling the team's registers (every lane's columns are its own: 41 and 52 us in the cases
// above, 41.6 and 54 with the tests that other rows take), anywhere behind the eighth column, or before it.
enum Ends { kWhole, kTail, kNarrow };
template <Ends ENDS>
__device__ __forceinline__ Eight lane_columns(int64_t c, int64_t cols) {
  Eight r(c, cols);
  if constexpr (ENDS == kWhole) {
    r.at = static_cast<int>(c);
    r.skip = 0;
  }
  if constexpr (ENDS != kNarrow) r.n = 8;
  return r;
}

template <int WAVES> constexpr int kNormRows = WAVES < 4 ? 4 / WAVES : 1;   // rows of a workgroup
template <int WAVES> constexpr int kNormThreads = kNormRows<WAVES> * WAVES * 64;

template <int XT, int WAVES, int V, Ends ENDS>
__global__ __launch_bounds__(kNormThreads<WAVES>) void rms_norm_kernel(NormArgs a) {
  constexpr int TEAM = WAVES * 64;
  __shared__ float scratch[WAVES];
  const int64_t row = static_cast<int64_t>(flat_block()) * kNormRows<WAVES> + threadIdx.x / TEAM;
  if (row >= a.rows) return;   // whole teams; with several waves per row, whole workgroups
  const int lane = threadIdx.x % TEAM;

  Raw8<XT> x[V], r[V];
  float w[V][8], v[V][8];
  Eight c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = lane_columns<ENDS>((static_cast<int64_t>(i) * TEAM + lane) * 8, a.cols);
    x[i].load_once(a.x, row * a.ld_x + c[i].at, c[i].n);
    if (a.residual != nullptr) r[i].load_once(a.residual, row * a.ld_residual + c[i].at, c[i].n);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.weight != nullptr) {
      read8_as(a.weight_dtype, a.weight, c[i].at, c[i].n, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.0f;
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = x[i].get(e);
    if (a.residual != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += r[i].get(e);
      round8<XT>(v[i]);
    }
    if (a.sum != nullptr) write_own<XT>(a.sum, row * a.ld_sum, c[i], v[i]);
    if (c[i].skip > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = e < c[i].skip ? 0.0f : v[i][e];
    }
    float part = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) part += v[i][e] * v[i][e];
    sum += part;
  }
  const float rstd = inverse_root(team_sum<WAVES, double>(sum, scratch) * a.inv_cols + a.eps);
  if (a.rstd != nullptr && lane == 0) a.rstd[row] = rstd;

#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t chunk = static_cast<int64_t>(i) * TEAM + lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rstd * w[i][e];
    round8<XT>(v[i]);
    if (a.y != nullptr) write_own<XT>(a.y, row * a.ld_y, c[i], v[i]);
    if (a.q != nullptr) {
      // 16 neighbouring lanes hold a block of 128; what is behind the last column is zeros
      if (c[i].skip > 0) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = (c[i].skip & o) == 0 ? v[i][e] : e + o < 8 ? v[i][e + o] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = chunk * 8 + e < a.cols ? v[i][e] : 0.0f;
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_abs(v[i][e]));
      m = row_max(m);
      const bool e4m3 = a.format == MUON_FP8_E4M3;
      const int byte = e4m3 ? scale_byte<MUON_FP8_E4M3>(m) : scale_byte<MUON_FP8_E5M2>(m);
      if (chunk * 8 < a.qp) {
        const float inv = inverse_scale(byte);
        *reinterpret_cast<u32x2*>(a.q + row * a.qp + chunk * 8) =
            e4m3 ? pack8<MUON_FP8_E4M3>(v[i], inv) : pack8<MUON_FP8_E5M2>(v[i], inv);
        const int64_t block = chunk >> 4, of = chunk & 15;
        if (of == 0) a.s[row * a.qs + block] = static_cast<uint8_t>(byte);
        if ((block + 1) * MUON_FP8_BLOCK == a.qp && of > 0 && block + of < a.qs) a.s[row * a.qs + block + of] = 127;
      }
    }
  }
}

// Workgroups walk over rows, so that a lane's columns of the weight gradient are summed in
// registers; what is left is a row of partial sums per workgroup, joined by norm_weight_kernel.
template <int XT, int WAVES, int V, Ends ENDS>
__global__ __launch_bounds__(kNormThreads<WAVES>) void rms_norm_backward_kernel(NormArgs a) {
  constexpr int TEAM = WAVES * 64, ROWS = kNormRows<WAVES>;
  __shared__ float scratch[WAVES];
  __shared__ float joined[ROWS > 1 ? TEAM * V * 8 : 1];
  const int team = threadIdx.x / TEAM, lane = threadIdx.x % TEAM;
  Eight c[V];
  float w[V][8], acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = lane_columns<ENDS>((static_cast<int64_t>(i) * TEAM + lane) * 8, a.cols);
    if (a.weight != nullptr) {
      read8_as(a.weight_dtype, a.weight, c[i].at, c[i].n, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = e < c[i].skip ? 0.0f : w[i][e];   // for the sum over the row
      acc[i][e] = 0.0f;
    }
  }
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + team; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * ROWS) {
    Raw8<XT> dy[V], s[V], ds[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dy[i].load_once(a.dy, row * a.ld_dy + c[i].at, c[i].n);
      s[i].load_once(a.x, row * a.ld_x + c[i].at, c[i].n);
      if (a.dsum != nullptr) ds[i].load_once(a.dsum, row * a.ld_dsum + c[i].at, c[i].n);
    }
    const float rstd = a.rstd_in[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gn = dy[i].get(e) * (s[i].get(e) * rstd);
        acc[i][e] += gn;
        dot += gn * w[i][e];
      }
    const float mean = team_sum<WAVES>(dot, scratch) * inv;
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = rstd * (dy[i].get(e) * w[i][e] - s[i].get(e) * rstd * mean);
        if (a.dsum != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] += ds[i].get(e);
        }
        write_own<XT>(a.dx, row * a.ld_dx, c[i], d);
      }
    }
  }
  if (a.partial == nullptr) return;
  if constexpr (ROWS > 1) {   // the teams' sums, one after the other
    for (int r = 0; r < ROWS; ++r) {
      if (team == r) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* at = joined + (i * 8 + e) * TEAM + lane;
            if (r > 0) acc[i][e] += *at;
            *at = acc[i][e];
          }
      }
      __syncthreads();
    }
    if (team != ROWS - 1) return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    write_own<MUON_DTYPE_F32>(a.partial, blockIdx.x * a.cols, c[i], acc[i]);
}

template <int DT>
__device__ __forceinline__ void finish_weight(const NormArgs& a, int64_t c, double v) {
  if (a.accumulate) v += load1<DT>(a.dweight, c);
  store1<DT>(a.dweight, c, static_cast<float>(v));
}

// 64 columns per workgroup, its 16 waves share the partial rows, whose sums are in 64 bits (0.3 us of 42, for an
// error of 7e-8 instead of 1.6e-7 over 16383 rows).
__global__ __launch_bounds__(1024) void norm_weight_kernel(NormArgs a, int32_t blocks) {
  __shared__ double part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  double v = 0.0;
  if (c < a.cols) {
#pragma unroll 8
    for (int b = wave; b < blocks; b += 16) v += a.partial[b * a.cols + c];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= a.cols) return;
  v = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += part[i][lane];
  if (a.dweight_dtype == MUON_DTYPE_F32) finish_weight<MUON_DTYPE_F32>(a, c, v);
  else if (a.dweight_dtype == MUON_DTYPE_BF16) finish_weight<MUON_DTYPE_BF16>(a, c, v);
  else finish_weight<MUON_DTYPE_F16>(a, c, v);
}

// The smallest team whose registers hold a row (of whole blocks of 128). With three loads per lane beside two
// and four: gradient of 8192 x 5120 52 us instead of 75, norm of 4096 x 11008 61 instead of 70.
template <int W, int V> struct Team {
  static constexpr int waves = W, loads = V;
};
template <typename F>
static hipError_t with_team(int64_t cols, F&& f) {
  if (cols <= 512) return f(Team<1, 1>());
  if (cols <= 1024) return f(Team<1, 2>());
  if (cols <= 1536) return f(Team<1, 3>());
  if (cols <= 2048) return f(Team<1, 4>());
  if (cols <= 4096) return f(Team<4, 2>());
  if (cols <= 6144) return f(Team<4, 3>());
  if (cols <= 8192) return f(Team<4, 4>());
  if (cols <= 12288) return f(Team<8, 3>());
  return f(Team<8, 4>());
}

template <int XT>
static hipError_t launch_forward(const NormArgs& a, hipStream_t s) {
  return with_team(a.cols, [&](auto team) {
    constexpr int W = decltype(team)::waves, V = decltype(team)::loads;
    const dim3 grid = flat_grid((a.rows + kNormRows<W> - 1) / kNormRows<W>), block(kNormThreads<W>);
    if (a.cols == W * V * 512) hipLaunchKernelGGL((rms_norm_kernel<XT, W, V, kWhole>), grid, block, 0, s, a);
    else if (a.cols >= 8) hipLaunchKernelGGL((rms_norm_kernel<XT, W, V, kTail>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_norm_kernel<XT, 1, 1, kNarrow>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}
hipError_t launch_rms_norm(int dtype, const NormArgs& a, hipStream_t s) {
  if (dtype == MUON_DTYPE_F32) return launch_forward<MUON_DTYPE_F32>(a, s);
  if (dtype == MUON_DTYPE_BF16) return launch_forward<MUON_DTYPE_BF16>(a, s);
  return launch_forward<MUON_DTYPE_F16>(a, s);
}

int32_t norm_blocks(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 2048 ? 4 : 1;
  return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, 768)));
}

template <int XT>
static hipError_t launch_backward(const NormArgs& a, hipStream_t s) {
  return with_team(a.cols, [&](auto team) {
    constexpr int W = decltype(team)::waves, V = decltype(team)::loads;
    const dim3 grid = dim3(norm_blocks(a.rows, a.cols)), block(kNormThreads<W>);
    if (a.cols == W * V * 512) hipLaunchKernelGGL((rms_norm_backward_kernel<XT, W, V, kWhole>), grid, block, 0, s, a);
    else if (a.cols >= 8) hipLaunchKernelGGL((rms_norm_backward_kernel<XT, W, V, kTail>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_norm_backward_kernel<XT, 1, 1, kNarrow>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}
hipError_t launch_rms_norm_backward(int dtype, const NormArgs& a, hipStream_t s) {
  if (dtype == MUON_DTYPE_F32) return launch_backward<MUON_DTYPE_F32>(a, s);
  if (dtype == MUON_DTYPE_BF16) return launch_backward<MUON_DTYPE_BF16>(a, s);
  return launch_backward<MUON_DTYPE_F16>(a, s);
}
hipError_t launch_norm_weight(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_weight_kernel, dim3(static_cast<unsigned>((a.cols + 63) / 64)), dim3(1024), 0, s, a,
                     norm_blocks(a.rows, a.cols));
  return hipGetLastError();
}

}  // namespace muon
