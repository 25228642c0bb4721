// Pieces of the quantisation to 8 bits that several kernels share: eight elements as they are
// stored, a block's scale, and its rounding.
#pragma once

#include "common.hpp"

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
  // the same for what is read once: past the caches (norm of 8192 x 4096 bf16 rows: 46 -> 41 us; fp32 the same
  // either way)
  __device__ __forceinline__ void load_once(const void* x, int64_t i, int n) {
    if (n >= 8) u = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(static_cast<const unsigned short*>(x) + i));
    else load(x, i, n);
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
  __device__ __forceinline__ void load_once(const void* x, int64_t i, int n) { load(x, i, n); }
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

}  // namespace muon
