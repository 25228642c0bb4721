// Products of 8-bit operands with a power-of-two scale for each block of 128 along the
// contraction (gfx950): C[i][j] (+)= sum_k A[i][k] B[j][k], both operands contiguous
// along k.
//
// The scaled matrix instructions take one scale byte per row and 32 elements of each
// operand and multiply by 2^(byte - 127) exactly, so the scales cost one register per
// row and 512 elements (four bytes, selected by the instruction) and no arithmetic on
// the accumulators, which stay in fp32 over the whole contraction.
//
// All 32-element pieces of a 128-block share its scale and a product does not depend on
// the order of its terms' places in the instruction, as long as both operands use the
// same places. So a lane may fetch any 32 of the block's bytes: it takes two 16-byte
// pieces that make the lanes of one row read 64 contiguous bytes per load.
//
// Precision. The 8-bit matrix instructions form the sum of eight neighbouring products
// before they add it to the fp32 accumulator, and cut each product to 13 bits below the
// exponent of the largest of the eight (measured; all shapes of the instruction, scaled
// or not, do the same). On normal data that is 1.3e-5 of the result's norm at any K,
// which a 16-bit result (2e-4 for fp16, 2e-3 for bf16) does not show. For a 32-bit
// result the operands are converted to bf16 in registers, scale included (exact: 8-bit
// values have at most 4 significant bits), and multiplied by the bf16 instructions,
// whose sums keep 24 bits: 2e-7 of the norm, at half the rate.
#include "common.hpp"
#include "fp8.hpp"

namespace muon {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Group of a row tile. Every wave of the workgroup finds it by itself: 64 groups at a
// time, a prefix sum of their tile counts. Returns false for a tile beyond the last
// group's.
__device__ __forceinline__ bool find_group(const int32_t* offsets, int n_groups, int64_t limit, int tile_rows, int tile,
                                           int& group, int64_t& first, int64_t& end) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int g0 = 0; g0 < n_groups; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < n_groups) {
      lo = static_cast<int>(min<int64_t>(max(offsets[g], 0), limit));
      hi = static_cast<int>(min<int64_t>(max(offsets[g + 1], lo), limit));
    }
    const int n = (hi - lo + tile_rows - 1) / tile_rows;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    const int total = __shfl(incl, 63, 64);
    if (tile < base + total) {
      const unsigned long long past = __ballot(base + incl > tile);
      const int l = __builtin_ctzll(past);
      group = g0 + l;
      const int before = base + __shfl(incl - n, l, 64);
      const int glo = __shfl(lo, l, 64), ghi = __shfl(hi, l, 64);
      first = glo + static_cast<int64_t>(tile - before) * tile_rows;
      end = ghi;
      return true;
    }
    base += total;
  }
  return false;
}

// What a workgroup computes: rows [m0, mend) of A (a tile of them), matrix `mat` of B
// and C, blocks [kb0, kb1) of the contraction.
struct Work {
  int64_t m0, mend;
  int mat, amat, bmat;
  int kb0, kb1;
};

template <int TM>
__device__ __forceinline__ bool find_work(const Fp8Gemm& g, int mtile, int z, Work& w) {
  w.kb0 = 0;
  w.kb1 = g.kb;
  w.m0 = static_cast<int64_t>(mtile) * TM;
  w.mend = g.M;
  w.mat = w.amat = w.bmat = z;
  if (g.mode == FP8_GROUP_ROWS) {
    w.amat = 0;
    if (!find_group(g.offsets, g.batch, g.M, TM, mtile, w.mat, w.m0, w.mend)) return false;
    w.mat = __builtin_amdgcn_readfirstlane(w.mat);
    w.bmat = w.mat;
  } else if (g.mode == FP8_GROUP_K) {
    w.amat = w.bmat = 0;
    const int64_t limit = static_cast<int64_t>(g.kb) * 128;
    const int lo = static_cast<int>(min<int64_t>(max(g.offsets[z], 0), limit));
    const int hi = static_cast<int>(min<int64_t>(max(g.offsets[z + 1], lo), limit));
    w.kb0 = lo / 128;
    w.kb1 = hi > lo ? (hi + 127) / 128 : w.kb0;
  }
  return true;
}

__device__ __forceinline__ float load_c(const void* c, int dtype, int64_t i) {
  if (dtype == MUON_DTYPE_F32) return static_cast<const float*>(c)[i];
  const unsigned short u = static_cast<const unsigned short*>(c)[i];
  return dtype == MUON_DTYPE_BF16 ? bf16_bits_to_f32(u) : f16_bits_to_f32(u);
}

__device__ __forceinline__ void store_c(void* c, int dtype, int64_t i, float v) {
  if (dtype == MUON_DTYPE_F32) static_cast<float*>(c)[i] = v;
  else if (dtype == MUON_DTYPE_BF16) static_cast<__bf16*>(c)[i] = static_cast<__bf16>(v);
  else static_cast<_Float16*>(c)[i] = static_cast<_Float16>(v);
}

// ---------------------------------------------------------------------------
// Conversion of 8-bit pairs to bf16, times 2^e.

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float scale_value(int word, int byte) {
  const uint32_t b = (static_cast<uint32_t>(word) >> (8 * byte)) & 255u;
  return __uint_as_float(b != 0 ? b << 23 : 0x400000u);   // byte 0 is 2^-127
}

template <int F, bool HI>
__device__ __forceinline__ bf16x2 to_bf16(int w, float s) {
  if constexpr (F == MUON_FP8_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI);
  else return __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, HI);
}

template <int F>
__device__ __forceinline__ bf16x8 to_bf16x8(int lo, int hi, float s) {
  const bf16x2 a = to_bf16<F, false>(lo, s), b = to_bf16<F, true>(lo, s), c = to_bf16<F, false>(hi, s),
               d = to_bf16<F, true>(hi, s);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// Few rows: 16 x 16 outputs per workgroup, the contraction split over its eight waves
// four blocks (one register of scales) at a time, joined in LDS in a fixed order. The
// weights are read once from memory straight into the instruction's registers; with
// four blocks in flight per wave that keeps the memory system busy, which is all that
// bounds a product of a few tokens. Rows beyond the matrix repeat its last row (their
// results are not stored).
constexpr int kFewWaves = 8;

template <int FA, int FB, bool WIDE, int U>
__device__ __forceinline__ void few_step(const i32x4 (&a0)[4], const i32x4 (&a1)[4], const i32x4 (&b0)[4],
                                         const i32x4 (&b1)[4], int sa, int sb, f32x4& acc) {
  // B's rows are the instruction's rows: register e of lane l is column 4 (l / 16) + e
  // of the tile, row l % 16
  if constexpr (WIDE) {
    const float fsa = scale_value(sa, U), fsb = scale_value(sb, U);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16x8<FB>(b0[U][2 * h], b0[U][2 * h + 1], fsb),
                                                    to_bf16x8<FA>(a0[U][2 * h], a0[U][2 * h + 1], fsa), acc, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16x8<FB>(b1[U][2 * h], b1[U][2 * h + 1], fsb),
                                                    to_bf16x8<FA>(a1[U][2 * h], a1[U][2 * h + 1], fsa), acc, 0, 0, 0);
    }
  } else {
    const i32x8 fa = __builtin_shufflevector(a0[U], a1[U], 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 fb = __builtin_shufflevector(b0[U], b1[U], 0, 1, 2, 3, 4, 5, 6, 7);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, FB, FA, U, sb, U, sa);
  }
}

template <int FA, int FB, bool WIDE>
__global__ __launch_bounds__(64 * kFewWaves) void fp8_few_rows_kernel(Fp8Gemm g, int mtiles, int ntiles) {
  __shared__ float part[kFewWaves][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = mtiles * ntiles;
  const int z = blockIdx.x / per;
  const int rest = blockIdx.x - z * per;
  const int nt = rest / mtiles, mt = rest - nt * mtiles;
  Work w;
  if (!find_work<16>(g, mt, z, w)) return;
  const int r = lane & 15, p = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(nt) * 16;
  const int64_t ra = min(w.m0 + r, w.mend - 1), rb = min(n0 + r, g.N - 1);
  const uint8_t* pa = g.a + w.amat * g.a_batch + ra * g.pitch + p * 16;
  const uint8_t* pb = g.b + w.bmat * g.b_batch + rb * g.pitch + p * 16;
  const uint8_t* psa = g.sa + w.amat * g.sa_batch + ra * g.s_pitch;
  const uint8_t* psb = g.sb + w.bmat * g.sb_batch + rb * g.s_pitch;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int q = w.kb0 / 4 + wave; q * 4 < w.kb1; q += kFewWaves) {
    const int sa = *reinterpret_cast<const int*>(psa + q * 4);
    const int sb = *reinterpret_cast<const int*>(psb + q * 4);
    i32x4 a0[4], a1[4], b0[4], b1[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // blocks outside [kb0, kb1) load the first one of the range and are not used
      const int kb = q * 4 + u >= w.kb0 && q * 4 + u < w.kb1 ? q * 4 + u : w.kb0;
      b0[u] = *reinterpret_cast<const i32x4*>(pb + static_cast<int64_t>(kb) * 128);
      b1[u] = *reinterpret_cast<const i32x4*>(pb + static_cast<int64_t>(kb) * 128 + 64);
      a0[u] = *reinterpret_cast<const i32x4*>(pa + static_cast<int64_t>(kb) * 128);
      a1[u] = *reinterpret_cast<const i32x4*>(pa + static_cast<int64_t>(kb) * 128 + 64);
    }
    if (q * 4 >= w.kb0 && q * 4 < w.kb1) few_step<FA, FB, WIDE, 0>(a0, a1, b0, b1, sa, sb, acc);
    if (q * 4 + 1 >= w.kb0 && q * 4 + 1 < w.kb1) few_step<FA, FB, WIDE, 1>(a0, a1, b0, b1, sa, sb, acc);
    if (q * 4 + 2 >= w.kb0 && q * 4 + 2 < w.kb1) few_step<FA, FB, WIDE, 2>(a0, a1, b0, b1, sa, sb, acc);
    if (q * 4 + 3 >= w.kb0 && q * 4 + 3 < w.kb1) few_step<FA, FB, WIDE, 3>(a0, a1, b0, b1, sa, sb, acc);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[wave][r][p * 4 + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int i = threadIdx.x >> 4, j = threadIdx.x & 15;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) v += part[k][i][j];
    const int64_t m = w.m0 + i, n = n0 + j;
    if (m < w.mend && n < g.N) {
      const int64_t at = (g.mode == FP8_GROUP_ROWS ? 0 : w.mat * g.c_batch) + m * g.ldc + n;
      if (g.accumulate) v += load_c(g.c, g.c_dtype, at);
      store_c(g.c, g.c_dtype, at, v);
    }
  }
}

Fp8Plan plan_fp8_gemm(int64_t, int64_t, int64_t, int32_t, int64_t, bool) { return {0, 1}; }

template <int FA, int FB>
static hipError_t launch(const Fp8Plan&, const Fp8Gemm& g, hipStream_t s) {
  const int64_t nt = (g.N + 15) / 16;
  int64_t mt = (g.M + 15) / 16, z = g.batch;
  if (g.mode == FP8_GROUP_ROWS) {
    mt = std::min<int64_t>(g.M, g.M / 16 + g.batch);
    z = 1;
  }
  const int64_t total = mt * nt * z;
  if (total <= 0) return hipSuccess;
  if (total > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(total)), block(64 * kFewWaves);
  if (g.c_dtype == MUON_DTYPE_F32)
    hipLaunchKernelGGL((fp8_few_rows_kernel<FA, FB, true>), grid, block, 0, s, g, static_cast<int>(mt),
                       static_cast<int>(nt));
  else
    hipLaunchKernelGGL((fp8_few_rows_kernel<FA, FB, false>), grid, block, 0, s, g, static_cast<int>(mt),
                       static_cast<int>(nt));
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(int fmt_a, int fmt_b, const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  if (fmt_a == MUON_FP8_E4M3) return fmt_b == MUON_FP8_E4M3 ? launch<0, 0>(p, g, s) : launch<0, 1>(p, g, s);
  return fmt_b == MUON_FP8_E4M3 ? launch<1, 0>(p, g, s) : launch<1, 1>(p, g, s);
}

hipError_t launch_fp8_reduce(const Fp8Gemm&, hipStream_t) { return hipSuccess; }

}  // namespace muon
