// Quantisation to 8 bits with a power-of-two scale for each block of 128 (gfx950).
//
// Per block: amax = max |x| over the finite values, e = the least integer >= -126
// with amax <= 1.75 * 2^(t + e) (t = 8 for e4m3, whose largest value is 448, and 15
// for e5m2, 57344), q = round(x * 2^-e) to nearest even, scale byte e + 127. The
// exponent of amax and one comparison of its mantissa give e without a logarithm or a
// division, and x * 2^-e is exact (but for fp32 subnormals), so q carries one rounding.
//
// One workgroup takes a 128 x 128 tile: it reads the tile once and writes it in both
// orientations, since a training step needs the rows for one product and the columns
// for another. What bounds it is HBM: the source once, one byte per element and
// orientation, 1/128 byte of scales. Both orientations of 8192 x 4096 bf16: 32.5
// us (4.1 TB/s; 43 us with the inputs held as floats); of 64 x 1408 x 2048 fp32 weights:
// 202 us (5.5 TB/s, a large copy reaches 5.1).
#include "common.hpp"
#include "fp8.hpp"

namespace muon {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 8 elements of dtype XT as they are stored, taken out one by one as floats: 16-bit inputs
// wait for their scales in half the registers. `fresh` makes the compiler convert again
// instead of keeping the floats of an earlier pass.
template <int XT> struct Raw8 {
  typedef u16x8 u16x8_any __attribute__((aligned(2)));
  u16x8 u;
  __device__ __forceinline__ void load(const void* x, int64_t i, int n) {
    const unsigned short* p = static_cast<const unsigned short*>(x) + i;
    if (n >= 8) {
      u = *reinterpret_cast<const u16x8_any*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = e < n ? p[e] : static_cast<unsigned short>(0);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    return XT == MUON_DTYPE_BF16 ? bf16_bits_to_f32(u[e]) : f16_bits_to_f32(u[e]);
  }
  __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(u)); }
};
template <> struct Raw8<MUON_DTYPE_F32> {
  typedef f32x4 f32x4_any __attribute__((aligned(4)));
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* x, int64_t i, int n) {
    const float* p = static_cast<const float*>(x) + i;
    if (n >= 8) {
      a = reinterpret_cast<const f32x4_any*>(p)[0];
      b = reinterpret_cast<const f32x4_any*>(p)[1];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = e < n ? p[e] : 0.0f;
        b[e] = 4 + e < n ? p[4 + e] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e] : b[e - 4]; }
  __device__ __forceinline__ void fresh() {}
};

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;   // false for NaN too
}

// The largest of 16 neighbouring lanes, in all of them: rotations within the 16.
template <int CTRL>
__device__ __forceinline__ float rotated(float v) {
  return __uint_as_float(static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, rotated<0x128>(v));
  v = fmaxf(v, rotated<0x124>(v));
  v = fmaxf(v, rotated<0x122>(v));
  return fmaxf(v, rotated<0x121>(v));
}

// The scale byte of a block and 2^-e.
template <int FMT>
__device__ __forceinline__ int scale_byte(float amax) {
  constexpr int T = FMT == MUON_FP8_E4M3 ? 8 : 15;
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - T + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax > 0.0f ? max(e, -126) + 127 : 127;
}
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }

// 8 floats times `inv`, rounded to 8 bits.
template <int FMT>
__device__ __forceinline__ u32x2 pack8(const float (&v)[8], float inv) {
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    if constexpr (FMT == MUON_FP8_E4M3) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
    }
    r[h] = static_cast<uint32_t>(w);
  }
  return r;
}

// Thread t of 256 holds rows 8 (t / 16) .. + 7 and columns 8 (t % 16) .. + 7 of the
// tile, 64 values in registers. A row's 128 columns lie in 16 neighbouring lanes (four
// rotations within them give its amax); a column's 128 rows lie in 16 threads 16 apart (two
// butterfly steps, then LDS across the four waves). The transposed tile goes through
// LDS in 8-byte pieces (8 rows of a column), piece g of column c at place
// g ^ ((c / 8) % 16), so that the 16 columns a wave writes at once fall in 16 places.
template <int XT, int FMT, bool BLOCKS, bool WEIGHTED>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(QuantArgs a) {
  __shared__ float cmax[4][128];
  __shared__ __align__(16) unsigned char tile[128 * 128];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const uint32_t b = flat_block();
  if (b >= static_cast<uint32_t>(a.total_tiles)) return;
  const uint32_t per = static_cast<uint32_t>(a.row_tiles * a.col_tiles);
  const int64_t batch = b / per;
  const int rest = static_cast<int>(b % per);
  const int rt = rest / a.col_tiles, ct = rest - rt * a.col_tiles;
  const int64_t r0 = static_cast<int64_t>(rt) * 128 + rg * 8;
  const int64_t c0 = static_cast<int64_t>(ct) * 128 + cg * 8;
  const int ncol = static_cast<int>(min<int64_t>(8, max<int64_t>(0, a.cols - c0)));

  Raw8<XT> raw[8];
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i;
    int64_t sr = r < a.rows ? r : -1;
    w[i] = 1.0f;
    if (a.row_index != nullptr && sr >= 0) {
      const int32_t id = a.row_index[r];
      sr = id >= 0 ? id / a.row_div : -1;
      if (sr >= a.src_rows) sr = -1;
      if (WEIGHTED && sr >= 0) {
        if (id < a.n_weights) w[i] = a.row_weight[id];
        else sr = -1;
      }
    }
    if (WEIGHTED && sr < 0) w[i] = 0.0f;
    raw[i].load(a.x, sr >= 0 ? batch * a.x_batch + sr * a.ldx + c0 : 0, sr >= 0 ? ncol : 0);
  }
  auto value = [&](int i, int e) { return WEIGHTED ? raw[i].get(e) * w[i] : raw[i].get(e); };

  float rmax[8], xmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rmax[i] = xmax[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = finite_abs(value(i, e));
      rmax[i] = fmaxf(rmax[i], m);
      xmax[e] = fmaxf(xmax[e], m);
    }
  if constexpr (BLOCKS) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, rmax[i]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((t & 63) == 0) cmax[wave][0] = m;
    __syncthreads();
    m = fmaxf(fmaxf(cmax[0][0], cmax[1][0]), fmaxf(cmax[2][0], cmax[3][0]));
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = xmax[i] = m;
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i].fresh();
  if (a.q != nullptr) {
    uint8_t* q = a.q + batch * a.rows * a.qp;
    uint8_t* s = a.s + batch * a.rows * a.qs;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = rmax[i];
      if constexpr (!BLOCKS) {
        m = row_max(m);
      }
      const int byte = scale_byte<FMT>(m);
      const int64_t r = r0 + i;
      if (r < a.rows) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = value(i, e);
        if (WEIGHTED && ncol < 8) {   // columns behind the last one stay zeros, also for a weight that is not finite
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = e < ncol ? v[e] : 0.0f;
        }
        *reinterpret_cast<u32x2*>(q + r * a.qp + c0) = pack8<FMT>(v, inverse_scale(byte));
        if (cg == 0) s[r * a.qs + ct] = static_cast<uint8_t>(byte);
        if (ct == a.col_tiles - 1 && cg > 0 && ct + cg < a.qs) s[r * a.qs + ct + cg] = 127;   // padding
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i].fresh();
  if (a.qt != nullptr) {
    if constexpr (!BLOCKS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xmax[e] = fmaxf(xmax[e], __shfl_xor(xmax[e], 16, 64));
        xmax[e] = fmaxf(xmax[e], __shfl_xor(xmax[e], 32, 64));
      }
      if ((t & 48) == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) cmax[wave][cg * 8 + e] = xmax[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = cg * 8 + e;
        xmax[e] = fmaxf(fmaxf(cmax[0][c], cmax[1][c]), fmaxf(cmax[2][c], cmax[3][c]));
      }
    }
    uint8_t* qt = a.qt + batch * a.cols * a.tp;
    uint8_t* st = a.st + batch * a.cols * a.ts;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int byte = scale_byte<FMT>(xmax[e]);
      float col[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) col[i] = value(i, e);
      *reinterpret_cast<u32x2*>(tile + (cg * 8 + e) * 128 + ((rg ^ cg) << 3)) = pack8<FMT>(col, inverse_scale(byte));
      if (rg == 0 && e < ncol) st[(c0 + e) * a.ts + rt] = static_cast<uint8_t>(byte);
      if (rt == a.row_tiles - 1 && rg > 0 && rt + rg < a.ts && e < ncol) st[(c0 + e) * a.ts + rt + rg] = 127;
    }
    __syncthreads();
    // 8 threads write one column's 128 rows; the two 8-byte pieces of a 16-byte read
    // are swapped where the place's lowest bit is flipped
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = i * 32 + (t >> 3), k = t & 7, sw = (c >> 3) & 15;
      const u32x4 p = *reinterpret_cast<const u32x4*>(tile + c * 128 + ((((2 * k) ^ sw) & ~1) << 3));
      const u32x4 o = (sw & 1) ? u32x4{p[2], p[3], p[0], p[1]} : p;
      const int64_t cc = static_cast<int64_t>(ct) * 128 + c;
      if (cc < a.cols) *reinterpret_cast<u32x4*>(qt + cc * a.tp + static_cast<int64_t>(rt) * 128 + k * 16) = o;
    }
  }
}

hipError_t launch_fp8_quantize(int x_dtype, int format, bool blocks, const QuantArgs& a, hipStream_t s) {
  if (a.total_tiles <= 0) return hipSuccess;
  const dim3 grid = flat_grid(a.total_tiles);
  const bool weighted = a.row_weight != nullptr;
#define MUON_QB(XT, FMT, B)                                                                                    \
  do {                                                                                                         \
    if (weighted) hipLaunchKernelGGL((fp8_quantize_kernel<XT, FMT, B, true>), grid, dim3(256), 0, s, a);       \
    else hipLaunchKernelGGL((fp8_quantize_kernel<XT, FMT, B, false>), grid, dim3(256), 0, s, a);               \
  } while (0)
#define MUON_Q(XT, FMT)                 \
  do {                                  \
    if (blocks) MUON_QB(XT, FMT, true); \
    else MUON_QB(XT, FMT, false);       \
  } while (0)
#define MUON_QX(XT)                                       \
  do {                                                    \
    if (format == MUON_FP8_E4M3) MUON_Q(XT, MUON_FP8_E4M3); \
    else MUON_Q(XT, MUON_FP8_E5M2);                       \
  } while (0)
  switch (x_dtype) {
    case MUON_DTYPE_BF16: MUON_QX(MUON_DTYPE_BF16); break;
    case MUON_DTYPE_F16: MUON_QX(MUON_DTYPE_F16); break;
    default: MUON_QX(MUON_DTYPE_F32);
  }
#undef MUON_QX
#undef MUON_Q
#undef MUON_QB
  return hipGetLastError();
}

}  // namespace muon
