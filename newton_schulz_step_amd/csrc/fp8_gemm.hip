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
// whose sums keep 24 bits: 2e-7 of the norm, at half the rate. bf16 has fp32's range, which
// values times scales can leave. So scales are raised by 2^17, which takes in the smallest
// ones, and where a result is not finite then (large ones beyond about 2^95, or NaN and
// infinities in the data) its sums are made once more: scales cut to what bf16 takes, each
// block's sum multiplied by what was cut off. Ordinary data never comes there.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "fp8.hpp"

namespace muon {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Groups of rows. Every wave finds a tile's group by itself: 64 groups at a time, a prefix
// sum of their tile counts. The first 64 groups stay in registers. Where an offset falls, the
// largest one before it takes its place, so that no two groups own a row: a prefix maximum,
// made only then (ascending offsets are found by one vote).

__device__ __forceinline__ int wave_inclusive_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(v, o, 64);
    if (lane >= o) v += up;
  }
  return v;
}

struct Groups {
  int lo, hi, incl;   // of group `lane` of the 64: rows, tiles of it and the ones before it
  int first;          // the first of the 64

  // `before`: where the groups before g0 end
  __device__ __forceinline__ void fetch(const int32_t* offsets, int n_groups, int limit, int tile_rows, int g0,
                                        int before) {
    const int lane = threadIdx.x & 63, g = g0 + lane;
    lo = hi = before;
    if (g < n_groups) {
      lo = min(max(offsets[g], 0), limit);
      hi = min(max(offsets[g + 1], 0), limit);
    }
    if (__ballot(lo < before || hi < lo) != 0) {
      lo = max(lo, before);
      hi = max(lo, hi);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(hi, o, 64);
        if (lane >= o) hi = max(hi, up);
      }
      const int up = __shfl_up(hi, 1, 64);
      if (lane > 0) lo = up;
    }
    incl = wave_inclusive_sum((hi - lo + tile_rows - 1) / tile_rows);
    first = g0;
  }
  __device__ __forceinline__ int end() const { return __builtin_amdgcn_readlane(hi, 63); }   // of all 64
  __device__ __forceinline__ int tiles() const { return __builtin_amdgcn_readlane(incl, 63); }
};

// Row tiles of all groups.
__device__ __forceinline__ int count_group_tiles(const int32_t* offsets, int n_groups, int limit, int tile_rows,
                                                 Groups& cache) {
  cache.fetch(offsets, n_groups, limit, tile_rows, 0, 0);
  int n = cache.tiles(), before = cache.end();
  for (int g0 = 64; g0 < n_groups; g0 += 64) {
    Groups more;
    more.fetch(offsets, n_groups, limit, tile_rows, g0, before);
    n += more.tiles();
    before = more.end();
  }
  return n;
}

// The group and rows of row tile `tile`; false for one beyond the last group's.
__device__ __forceinline__ bool find_group(const int32_t* offsets, int n_groups, int limit, int tile_rows,
                                           const Groups& cache, int tile, int& group, int& first, int& end) {
  Groups g = cache;
  while (tile >= g.tiles()) {
    tile -= g.tiles();
    if (g.first + 64 >= n_groups) return false;
    g.fetch(offsets, n_groups, limit, tile_rows, g.first + 64, g.end());
  }
  const int l = __builtin_ctzll(__ballot(g.incl > tile));
  const int lo = __builtin_amdgcn_readlane(g.lo, l), hi = __builtin_amdgcn_readlane(g.hi, l);
  const int before = __builtin_amdgcn_readlane(g.incl, l) - (hi - lo + tile_rows - 1) / tile_rows;
  group = g.first + l;
  first = lo + (tile - before) * tile_rows;
  end = hi;
  return true;
}

// Whether no offset of a grouped contraction falls.
__device__ __forceinline__ bool offsets_ascend(const Fp8Gemm& g) {
  bool falls = false;
  for (int z = threadIdx.x & 63; z < g.batch; z += 64) falls = falls || g.offsets[z + 1] < g.offsets[z];
  return __ballot(falls) == 0;
}

// Blocks [kb0, kb1) of group z of a grouped contraction (scalar loads: z is uniform), [0, 0)
// of one without columns: its first block may lie behind the operand's last.
__device__ __forceinline__ void group_blocks(const Fp8Gemm& g, int z, bool ascend, int& kb0, int& kb1) {
  const auto* off = (const __attribute__((address_space(4))) int32_t*)(g.offsets);
  const int limit = g.kb * 128;
  int most = off[z];   // of the offsets up to it
  if (!ascend)
    for (int i = 0; i < z; ++i) most = max(most, off[i]);
  const int lo = min(max(most, 0), limit);
  const int hi = min(max(off[z + 1], lo), limit);
  kb0 = hi > lo ? lo / 128 : 0;
  kb1 = hi > lo ? (hi + 127) / 128 : 0;
}

// 64 groups of a contraction from the one with most blocks to the one with least: lane r
// holds the r-th. A lane counts the longer groups (those as long, before it) and sends its
// number to that lane; lanes without a group are the shortest ones. (An order only: where
// offsets fall, the lengths here are not the groups' own.)
__device__ __forceinline__ int longest_first(const Fp8Gemm& g, int first) {
  const int lane = threadIdx.x & 63, limit = g.kb * 128, z = first + lane;
  int blocks = -1;
  if (z < g.batch) {
    const int lo = min(max(g.offsets[z], 0), limit), hi = min(max(g.offsets[z + 1], lo), limit);
    blocks = (hi - lo + 127) / 128;
  }
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < 64; ++i) {
    const int other = __builtin_amdgcn_readlane(blocks, i);
    rank += other > blocks || (other == blocks && i < lane) ? 1 : 0;
  }
  return __builtin_amdgcn_ds_permute(rank * 4, z);
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

// The scale bytes whose 8-bit values are normal bf16 numbers, from the smallest (2^-9 for
// e4m3, 2^-16 for e5m2) to the largest (448, 57344).
template <int F> struct ScaleRange {
  static constexpr int LOW = F == MUON_FP8_E4M3 ? 10 : 17, HIGH = F == MUON_FP8_E4M3 ? 246 : 239;
};
template <int F>
__device__ __forceinline__ int near_scale(int byte) { return min(max(byte, ScaleRange<F>::LOW), ScaleRange<F>::HIGH); }
// What near_scale cut off, as a factor; byte 255 stands for a NaN.
template <int F>
__device__ __forceinline__ float rest_scale(int byte) {
  return byte == 255 ? __builtin_nanf("") : __uint_as_float(static_cast<uint32_t>(byte - near_scale<F>(byte) + 127) << 23);
}

__device__ __forceinline__ float scale_value(int byte) { return __uint_as_float(static_cast<uint32_t>(byte) << 23); }

// 2^17 times the scale: every value of the smallest scales is a normal number then. Scales
// too large for that become a NaN, their values or the sum infinite, so that a finite sum
// of such products, 2^34 times the wanted one, is right.
constexpr int kRaise = ScaleRange<MUON_FP8_E5M2>::LOW;
constexpr float kLower = 1.0f / (1ull << (2 * kRaise));
__device__ __forceinline__ float raised_scale(int byte) { return scale_value(min(byte + kRaise, 255)); }

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
// Few rows: 16 MT rows x 16 columns of outputs per workgroup, the contraction split over
// its eight waves four blocks (one word of scales) at a time, joined in LDS in a fixed
// order. The weights are read once from memory straight into the instruction's registers;
// with four blocks in flight per wave that keeps the memory system busy, which is all that
// bounds a product of a few tokens. Rows beyond the matrix repeat its last row (their
// results are not stored). One token, 11008 x 4096: 12.4 us where the weights are still in
// the last-level cache, 12.5 to 12.8 from memory (3.6 TB/s).
constexpr int kFewWaves = 8;

template <int FA, int FB, bool WIDE, bool FAR, int U>
__device__ __forceinline__ void few_step(const i32x4& a0, const i32x4& a1, const i32x4& b0, const i32x4& b1, int sa,
                                         int sb, f32x4& acc) {
  // B's rows are the instruction's rows: register e of lane l is column 4 (l / 16) + e
  // of the tile, row l % 16
  if constexpr (WIDE) {
    const int ba = (static_cast<uint32_t>(sa) >> (8 * U)) & 255, bb = (static_cast<uint32_t>(sb) >> (8 * U)) & 255;
    const float fsa = FAR ? scale_value(near_scale<FA>(ba)) : raised_scale(ba);
    const float fsb = FAR ? scale_value(near_scale<FB>(bb)) : raised_scale(bb);
    const f32x4 sum = acc;
    if constexpr (FAR) acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16x8<FB>(b0[2 * h], b0[2 * h + 1], fsb),
                                                    to_bf16x8<FA>(a0[2 * h], a0[2 * h + 1], fsa), acc, 0, 0, 0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16x8<FB>(b1[2 * h], b1[2 * h + 1], fsb),
                                                    to_bf16x8<FA>(a1[2 * h], a1[2 * h + 1], fsa), acc, 0, 0, 0);
    if constexpr (FAR) {
      const float ra = rest_scale<FA>(ba);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[e] = sum[e] + acc[e] * (ra * rest_scale<FB>(__shfl(bb, ((threadIdx.x >> 4) & 3) * 4 + e, 64)));
    }
  } else {
    const i32x8 fa = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 fb = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, FB, FA, U, sb, U, sa);
  }
}

template <int FA, int FB, bool WIDE, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void fp8_few_rows_kernel(Fp8Gemm g, int mtiles, int ntiles) {
  constexpr int TM = 16 * MT;
  __shared__ float part[kFewWaves][TM][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t per = static_cast<uint32_t>(mtiles * ntiles), block = flat_block();
  const int z = static_cast<int>(block / per);
  if (z >= (g.mode == FP8_GROUP_ROWS ? 1 : g.batch)) return;
  const int rest = static_cast<int>(block - z * per);
  const int nt = rest / mtiles, mt = rest - nt * mtiles;
  // rows [m0, mend) of A (a tile of them), matrix `mat` of B and C, blocks [kb0, kb1)
  struct { int m0, mend, mat, amat, bmat, kb0, kb1; } w = {mt * TM, static_cast<int>(g.M), z, z, z, 0, g.kb};
  if (g.mode == FP8_GROUP_ROWS) {
    Groups groups;
    groups.fetch(g.offsets, g.batch, static_cast<int>(g.M), TM, 0, 0);
    if (!find_group(g.offsets, g.batch, static_cast<int>(g.M), TM, groups, mt, w.mat, w.m0, w.mend)) return;
    w.amat = 0;
    w.bmat = w.mat;
  } else if (g.mode == FP8_GROUP_K) {
    w.amat = w.bmat = 0;
    group_blocks(g, z, offsets_ascend(g), w.kb0, w.kb1);
  }
  const int r = lane & 15, p = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(nt) * 16;
  const int64_t rb = min(n0 + r, g.N - 1);
  const uint8_t* pb = g.b + w.bmat * g.b_batch + rb * g.pitch + p * 16;
  const uint8_t* psb = g.sb + w.bmat * g.sb_batch + rb * g.s_pitch;
  const uint8_t* pa[MT];
  const uint8_t* psa[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ra = min(w.m0 + i * 16 + r, w.mend - 1);
    pa[i] = g.a + w.amat * g.a_batch + ra * g.pitch + p * 16;
    psa[i] = g.sa + w.amat * g.sa_batch + ra * g.s_pitch;
    acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  auto contract = [&](auto far) {
    constexpr bool FAR = decltype(far)::value;
    for (int q = w.kb0 / 4 + wave; q * 4 < w.kb1; q += kFewWaves) {
      const int sb = *reinterpret_cast<const int*>(psb + q * 4);
      // blocks outside [kb0, kb1) load the first one of the range and are not used
      int64_t at[4];
      bool in[4];
      i32x4 b0[4], b1[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        in[u] = q * 4 + u >= w.kb0 && q * 4 + u < w.kb1;
        at[u] = static_cast<int64_t>(in[u] ? q * 4 + u : w.kb0) * 128;
        b0[u] = *reinterpret_cast<const i32x4*>(pb + at[u]);
        b1[u] = *reinterpret_cast<const i32x4*>(pb + at[u] + 64);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int sa = *reinterpret_cast<const int*>(psa[i] + q * 4);
        i32x4 a0[4], a1[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          a0[u] = *reinterpret_cast<const i32x4*>(pa[i] + at[u]);
          a1[u] = *reinterpret_cast<const i32x4*>(pa[i] + at[u] + 64);
        }
        if (in[0]) few_step<FA, FB, WIDE, FAR, 0>(a0[0], a1[0], b0[0], b1[0], sa, sb, acc[i]);
        if (in[1]) few_step<FA, FB, WIDE, FAR, 1>(a0[1], a1[1], b0[1], b1[1], sa, sb, acc[i]);
        if (in[2]) few_step<FA, FB, WIDE, FAR, 2>(a0[2], a1[2], b0[2], b1[2], sa, sb, acc[i]);
        if (in[3]) few_step<FA, FB, WIDE, FAR, 3>(a0[3], a1[3], b0[3], b1[3], sa, sb, acc[i]);
      }
    }
  };
  contract(std::false_type{});
  if constexpr (WIDE) {
    float test = 0.0f;   // a NaN if a sum is not finite
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        test += acc[i][e] * 0.0f;
        acc[i][e] *= kLower;
      }
    if (__ballot(test != 0.0f) != 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      contract(std::true_type{});
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][i * 16 + r][p * 4 + e] = acc[i][e];
  __syncthreads();
  for (int k = threadIdx.x; k < TM * 16; k += 64 * kFewWaves) {
    const int i = k >> 4, j = k & 15;
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < kFewWaves; ++x) v += part[x][i][j];
    const int64_t m = w.m0 + i, n = n0 + j;
    if (m < w.mend && n < g.N) {
      const int64_t c = (g.mode == FP8_GROUP_ROWS ? 0 : w.mat * g.c_batch) + m * g.ldc + n;
      if (g.accumulate) v += load_c(g.c, g.c_dtype, c);
      store_c(g.c, g.c_dtype, c, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: TILE x TILE outputs (256 or 128) by four waves in a 2 x 2 grid, each owning
// (TILE / 2)^2 outputs as 32 x 32 blocks in registers. A workgroup walks over tiles
// (one workgroup per CU with 256-tiles, two with 128-tiles).
//
// Slices of both operands, one block (128 bytes) of every row, go straight from memory to
// LDS (no registers) into two buffers. A slice is multiplied in two periods of 64 bytes,
// one 32 x 32 x 64 instruction per block pair each. During a period a wave multiplies
// from one set of registers and reads the next period's operands from LDS into the other
// set, so a slice's buffer has been read by the end of its first period; one barrier
// then frees it and publishes the next slice, and the loads of the slice after next are
// issued into it, spread over the second period. They have one to two periods (256-tiles:
// 1000 to 2000 matrix cycles) to arrive. Rows are fetched 128 bytes at a time: against four
// buffers of 64 bytes per row that halves the requests to the last-level cache (51 to 25
// million on 8192 x 8192 x 8192) and takes the conflicts out of LDS, at the same time per
// slice.
//
// The slices of a workgroup's tiles form one stream: the last slices of a tile are
// followed by the first ones of the next, which arrive while the results of the tile are
// stored. Results therefore pass through a part of LDS of their own (4 KB per wave).
//
// LDS rows of a slice are 128 bytes, eight 16-byte chunks; chunk c of row r is stored at
// place c ^ swz(r), so lanes that read one chunk of neighbouring rows spread over the
// banks (no conflicts counted). A direct load writes consecutive lanes to consecutive
// places, so the lanes fetch permuted chunks instead. Rows and slices beyond the operand
// or the group are fetched as zeros: the buffer resource's bounds.
//
// The loop body is two slices: their buffers are then known at compile time, and the
// compiler waits for exactly the loads of the buffer that is read. An odd last slice is
// paired with one of zeros, whose scales are set to 2^-127.
//
// Scales: 16 bytes (16 blocks) of every row at a time, also by direct loads, in two parts
// of LDS: while one is used the other is fetched, once in 16 slices. (One word at a time
// fetches 64 cache lines for 256 bytes; with that in every fourth slice the loop was 12%
// slower.)

__device__ __forceinline__ int row_swizzle(int r) { return (r ^ ((r >> 3) & 3)) & 7; }   // of r modulo 32

template <int V> using Int = std::integral_constant<int, V>;

template <int N, typename F>
__device__ __forceinline__ void each_step(F&& f) {
  if constexpr (N > 0) {
    each_step<N - 1>(f);
    f(Int<N - 1>{});
  }
}

// 16 bytes of results at any element-aligned place
typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// What a tile does with its results: rounds them to bf16 or fp16, adds them to 16-bit ones,
// or (WIDE products) stores or adds fp32.
enum { OUT_BF16 = 0, OUT_F16 = 1, OUT_ADD_16 = 2, OUT_F32 = 3 };

template <typename T>
__device__ __forceinline__ u16x4 round4(float a, float b, float c, float d) {
  const float v[4] = {a, b, c, d};
  T o[4];
  rne<T, 4>(v, o);
  u16x4 u;
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = __builtin_bit_cast(unsigned short, o[e]);
  return u;
}

// A tile: rows [m0, mend) of A and C (its own TILE of them), columns from n0, matrix `mat`
// of C, blocks [kb0, kb1) of the contraction; its operands' first rows and the bytes of
// their rows (what lies behind reads as zeros).
struct Tile {
  int m0, mend, n0, mat;
  int kb0, kb1;
  const uint8_t *a, *b;
  int na, nb;
};

template <int FA, int FB, int OUT, int TILE>
__device__ __forceinline__ void tile_product(const Fp8Gemm& g, int mtiles, int ntiles) {
  constexpr bool WIDE = OUT == OUT_F32;
  constexpr int HALF = TILE / 2, WB = HALF / 32;
  constexpr int SLICE = TILE * 128;             // bytes of one operand's slice
  constexpr int LOADS = TILE / 32;              // 1-KB loads per wave, operand and slice
  constexpr int STAGE = TILE * 16;              // bytes of a wave's results in LDS
  __shared__ __align__(1024) char buf0[2 * SLICE], buf1[2 * SLICE];
  __shared__ __align__(16) unsigned char scales[2][2 * TILE * 16];
  __shared__ __align__(16) char stages[4 * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int pitch = static_cast<int>(g.pitch), sp = static_cast<int>(g.s_pitch);

  Groups groups{};
  if (g.mode == FP8_GROUP_ROWS)
    mtiles = count_group_tiles(g.offsets, g.batch, static_cast<int>(g.M), TILE, groups);
  const int total = mtiles * ntiles * (g.mode == FP8_GROUP_ROWS ? 1 : g.batch);

  // Workgroups are dealt round-robin over the eight XCDs. In every round of the chip each
  // XCD takes consecutive tiles (its own last-level cache then sees neighbours), and all
  // XCDs stay close together. Within a matrix, bands of four tile columns are walked row
  // by row.
  // Contractions of groups differ in length, so a workgroup's tiles would add up to as much
  // as 1.2 to 1.4 times the average. With several rounds the groups (64 at a time) come
  // longest first, and every second round runs backwards: 1.05 to 1.13 times.
  constexpr int ROUND = TILE == 256 ? 256 : 512;
  const bool by_length = g.mode == FP8_GROUP_K && total > ROUND;
  const bool ascend = g.mode == FP8_GROUP_K && offsets_ascend(g);
  int sorted = 0, sorted_first = -1;   // the 64 groups from sorted_first on
  auto tile_at = [&](int index) {
    const int chunk = index / ROUND, inside = index % ROUND;
    const int size = min(ROUND, total - chunk * ROUND);
    int place = (inside & 7) * (size / 8) + min(inside & 7, size % 8) + (inside >> 3);
    if (by_length && (chunk & 1)) place = size - 1 - place;
    const int b = chunk * ROUND + place;
    const int per = mtiles * ntiles;
    int z = b / per;
    const int rest = b - z * per;
    if (by_length) {
      if (sorted_first != (z & ~63)) {
        sorted_first = z & ~63;
        sorted = longest_first(g, sorted_first);
      }
      z = __builtin_amdgcn_readlane(sorted, z & 63);
    }
    const int band = rest / (4 * mtiles);
    const int width = min(4, ntiles - band * 4);
    const int in = rest - band * 4 * mtiles;
    const int mt = in / width;
    Tile t;
    t.n0 = (band * 4 + in - mt * width) * TILE;
    t.m0 = mt * TILE;
    t.mend = static_cast<int>(g.M);
    t.mat = z;
    t.kb0 = 0;
    t.kb1 = g.kb;
    if (g.mode == FP8_GROUP_ROWS)
      find_group(g.offsets, g.batch, static_cast<int>(g.M), TILE, groups, mt, t.mat, t.m0, t.mend);
    else if (g.mode == FP8_GROUP_K)
      group_blocks(g, z, ascend, t.kb0, t.kb1);
    t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    t.mend = __builtin_amdgcn_readfirstlane(t.mend);
    t.mat = __builtin_amdgcn_readfirstlane(t.mat);
    t.a = g.a + (g.mode == FP8_DENSE ? t.mat * g.a_batch : 0) + t.m0 * g.pitch;
    t.b = g.b + (g.mode == FP8_GROUP_K ? 0 : t.mat * g.b_batch) + t.n0 * g.pitch;
    t.na = min(TILE, t.mend - t.m0) * pitch;
    t.nb = static_cast<int>(min<int64_t>(TILE, g.N - t.n0)) * pitch;
    return t;
  };
  // slices of a tile, counted in pairs
  auto slices_of = [](const Tile& t) { return max(2, (t.kb1 - t.kb0 + 1) & ~1); };

  // per-lane offsets of operand rows (both operands have the same). Scale rows come 64 per
  // load: of a 256-tile each wave fetches 64 rows of both operands, of a 128-tile waves 0 and
  // 1 rows of A, 2 and 3 of B.
  int vo[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = (wave * LOADS + i) * 8 + (lane >> 3);
    vo[i] = r * pitch + ((lane & 7) ^ row_swizzle(r)) * 16;
  }
  const bool sfirst = TILE == 256 || wave < 2;
  const int srow = (TILE == 256 ? wave : wave & 1) * 64;
  const int vs = (srow + lane) * sp;

  // per-lane read offsets within a slice, period 0: two neighbouring chunks of row lane %
  // 32 (the second one at ^ 16, those of period 1 at ^ 64; the swizzle only depends on the
  // row modulo 32)
  const int r = lane & 31, h = lane >> 5;
  const int chunk0 = ((2 * h) ^ row_swizzle(r)) * 16;
  const int ao = (wm * HALF + r) * 128 + chunk0, bo = SLICE + (wn * HALF + r) * 128 + chunk0;

#define MUON_RSRC(p, n) __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, n, 0x00027000)
#define MUON_GLDS(rsrc, lds, size, voff, soff)                                                              \
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MUON_LDS void*)(lds), size, voff, soff, 0, 0)
  // slice `s` of a tile (zeros behind its last one: no bytes and no offset, since the
  // bounds are what the offset leaves of the bytes)
  auto load_slice = [&](char* to, const uint8_t* a, const uint8_t* b, int na, int nb, int kb0, int kb1, int s) {
    const bool there = kb0 + s < kb1;
    const auto ra = MUON_RSRC(a, there ? na : 0), rb = MUON_RSRC(b, there ? nb : 0);
    const int so = there ? (kb0 + s) * 128 : 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) MUON_GLDS(ra, to + (wave * LOADS + i) * 1024, 16, vo[i], so);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) MUON_GLDS(rb, to + SLICE + (wave * LOADS + i) * 1024, 16, vo[i], so);
  };
  // 16 blocks of scales of a tile's rows, by (first row, rows) of both operands
  auto load_scales = [&](int slot, int mat, int m0, int rows_a, int n0, int rows_b, int part) {
    unsigned char* to = scales[slot];
    const uint8_t* sa = g.sa + (g.mode == FP8_DENSE ? mat * g.sa_batch : 0) + m0 * g.s_pitch;
    const uint8_t* sb = g.sb + (g.mode == FP8_GROUP_K ? 0 : mat * g.sb_batch) + n0 * g.s_pitch;
    const auto ra = MUON_RSRC(sa, rows_a * sp), rb = MUON_RSRC(sb, rows_b * sp);
    if (sfirst) MUON_GLDS(ra, to + srow * 16, 16, vs, part * 16);
    else MUON_GLDS(rb, to + (TILE + srow) * 16, 16, vs, part * 16);
    if constexpr (TILE == 256) MUON_GLDS(rb, to + (TILE + srow) * 16, 16, vs, part * 16);
  };
  auto scales_of = [&](int slot, const Tile& t, int part, bool any) {
    load_scales(slot, t.mat, t.m0, any ? min(TILE, t.mend - t.m0) : 0, t.n0,
                any ? static_cast<int>(min<int64_t>(TILE, g.N - t.n0)) : 0, part);
  };

  f32x16 acc[WB][WB];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
      for (int j = 0; j < WB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  };
  i32x4 fa[2][WB][2], fb[2][WB][2];
  auto read = [&](int set, const char* from) {   // set = period of the slice
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      fa[set][i][0] = *reinterpret_cast<const i32x4*>(from + (ao ^ (set * 64)) + i * 4096);
      fa[set][i][1] = *reinterpret_cast<const i32x4*>(from + (ao ^ (set * 64 + 16)) + i * 4096);
    }
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      fb[set][i][0] = *reinterpret_cast<const i32x4*>(from + (bo ^ (set * 64)) + i * 4096);
      fb[set][i][1] = *reinterpret_cast<const i32x4*>(from + (bo ^ (set * 64 + 16)) + i * 4096);
    }
  };
  // scale bytes of the lane's rows of A, then of B, for the two slices of a body. They are
  // read in the period before their slice's first one and masked in that one (0, 2^-127,
  // for a slice behind the last: its zeros must not meet another group's NaN scale).
  int sc[2][2 * WB];
  auto read_scales = [&](int set, int slot, int kb) {
    const unsigned char* from = scales[slot] + (kb & 15);
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      sc[set][i] = from[(wm * HALF + i * 32 + r) * 16];
      sc[set][WB + i] = from[(TILE + wn * HALF + i * 32 + r) * 16];
    }
  };
  auto mask_scales = [&](int set, bool there) {
    const int mask = there ? 255 : 0;
#pragma unroll
    for (int i = 0; i < 2 * WB; ++i) sc[set][i] &= mask;
  };
  auto publish = [&]() {   // own reads and loads are done, then everybody's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto multiply = [&](auto set, auto slice) {
    constexpr int SET = decltype(set)::value, U = decltype(slice)::value;
    if constexpr (WIDE) {
      float fs[2 * WB];
#pragma unroll
      for (int i = 0; i < 2 * WB; ++i) fs[i] = raised_scale(sc[U][i]);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 xa[WB], xb[WB];
#pragma unroll
        for (int i = 0; i < WB; ++i) {
          xa[i] = to_bf16x8<FA>(fa[SET][i][s >> 1][2 * (s & 1)], fa[SET][i][s >> 1][2 * (s & 1) + 1], fs[i]);
          xb[i] = to_bf16x8<FB>(fb[SET][i][s >> 1][2 * (s & 1)], fb[SET][i][s >> 1][2 * (s & 1) + 1], fs[WB + i]);
        }
#pragma unroll
        for (int i = 0; i < WB; ++i)
#pragma unroll
          for (int j = 0; j < WB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xb[j], xa[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < WB; ++i)
#pragma unroll
        for (int j = 0; j < WB; ++j) {
          const i32x8 x = __builtin_shufflevector(fa[SET][i][0], fa[SET][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
          const i32x8 y = __builtin_shufflevector(fb[SET][j][0], fb[SET][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(y, x, acc[i][j], FB, FA, 0, sc[U][WB + j], 0, sc[U][i]);
        }
    }
  };
  // reads and loads spread over the period's matrix instructions
  auto schedule = [&](auto loads) {
    if constexpr (!WIDE) {
      constexpr int NM = WB * WB;
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        if constexpr (decltype(loads)::value) {
          // 4 WB operand and 2 WB scale reads, 2 LOADS loads
          __builtin_amdgcn_sched_group_barrier(0x100, NM == 16 ? 2 : 3, 0);        // LDS reads
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
          __builtin_amdgcn_sched_group_barrier(0x020, 2 * LOADS / NM, 0);          // loads to LDS
        } else {
          __builtin_amdgcn_sched_group_barrier(0x100, 4 * WB / NM, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // Results of a tile, a few blocks at a time through the wave's part of LDS, in 16-byte
  // chunks swizzled by the row, so that they leave as 64 or 128 neighbouring bytes of a
  // row. Register 4 q + e of block (i, j) in lane l is row l % 32, column 8 q + 4 (l / 32)
  // + e of the block. 16-bit results are rounded before (TILE / 128 blocks together), fp32
  // ones and sums with what is there pass in fp32, 32 rows of a block (128-tiles: 16) at a
  // time. LDS keeps a wave's order, so the next blocks are written behind the reads of
  // these without a wait. Whole tiles take no masks: with a branch per store, each waiting
  // for its own read, a tile took 7 us to leave.
  constexpr bool ROUNDED = OUT == OUT_BF16 || OUT == OUT_F16;
  constexpr int NB = ROUNDED ? TILE / 128 : 1;          // blocks at a time
  constexpr int RS = ROUNDED ? 32 : STAGE / 128;        // rows at a time
  constexpr int CH = ROUNDED ? 4 * NB : 8;              // chunks of a staged row
  constexpr int LPR = ROUNDED ? CH : 4, RPP = 64 / LPR; // lanes per row (8 columns each), rows per pass
  constexpr int NP = RS / RPP;                          // passes
  constexpr int ESZ = WIDE ? 4 : 2;
  constexpr int NS = 32 / RS, NJ = WB / NB;             // steps: rows of a row of blocks, groups of blocks
  char* stage = stages + wave * STAGE;
  auto stage_write = [&](auto step) {
    constexpr int I = decltype(step)::value / (NS * NJ), S = decltype(step)::value / NJ % NS,
                  J = decltype(step)::value % NJ * NB;
    // the blocks stay in accumulation registers until here
    if constexpr (TILE == 256) {
#pragma unroll
      for (int b = 0; b < NB; ++b) asm volatile("" : "+a"(acc[I][J + b]));
    }
    if (RS == 32 || (r >> 4) == S) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& x = acc[I][J + b];
          if constexpr (ROUNDED) {
            using T = std::conditional_t<OUT == OUT_BF16, __bf16, _Float16>;
            *reinterpret_cast<u16x4*>(stage + r * (CH * 16) + (((b * 4 + q) ^ (r & (CH - 1))) * 16) + h * 8) =
                round4<T>(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          } else {
            constexpr float f = WIDE ? kLower : 1.0f;
            *reinterpret_cast<f32x4*>(stage + (r % RS) * 128 + (((2 * q + h) ^ (r & 7)) * 16)) =
                f32x4{x[4 * q] * f, x[4 * q + 1] * f, x[4 * q + 2] * f, x[4 * q + 3] * f};
          }
        }
    }
    __builtin_amdgcn_wave_barrier();
  };
  // what a lane takes out of LDS per pass: 8 rounded results, or 8 in fp32
  struct Taken {
    u16x8 u;
    f32x4 lo, hi;
  };
  auto stage_read = [&](Taken (&to)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int row = p * RPP + lane / LPR;
      if constexpr (ROUNDED) {
        to[p].u = *reinterpret_cast<const u16x8*>(stage + row * (CH * 16) + (((lane % LPR) ^ (row & (CH - 1))) * 16));
      } else {
        to[p].lo = *reinterpret_cast<const f32x4*>(stage + row * 128 + (((2 * (lane % LPR)) ^ (row & 7)) * 16));
        to[p].hi = *reinterpret_cast<const f32x4*>(stage + row * 128 + (((2 * (lane % LPR) + 1) ^ (row & 7)) * 16));
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  // 16-bit values of C added to 8 fp32 results
  auto add_16 = [&](Taken& x, const u16x8& u) {
    const bool bf = g.c_dtype == MUON_DTYPE_BF16;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x.lo[e] += bf ? bf16_bits_to_f32(u[e]) : f16_bits_to_f32(u[e]);
      x.hi[e] += bf ? bf16_bits_to_f32(u[4 + e]) : f16_bits_to_f32(u[4 + e]);
    }
    const u16x4 y = bf ? round4<__bf16>(x.lo[0], x.lo[1], x.lo[2], x.lo[3]) : round4<_Float16>(x.lo[0], x.lo[1], x.lo[2], x.lo[3]);
    const u16x4 z = bf ? round4<__bf16>(x.hi[0], x.hi[1], x.hi[2], x.hi[3]) : round4<_Float16>(x.hi[0], x.hi[1], x.hi[2], x.hi[3]);
    x.u = __builtin_shufflevector(y, z, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto store = [&](const Tile& t) {
    const int col = (lane % LPR) * 8;
    const int rows = t.mend - (t.m0 + wm * HALF) - lane / LPR;          // beyond the lane's first row
    const int cols = static_cast<int>(g.N - (t.n0 + wn * HALF)) - col;  // beyond the lane's first column
    char* c = static_cast<char*>(g.c) +
              ((g.mode == FP8_GROUP_ROWS ? 0 : t.mat * g.c_batch) + (t.m0 + wm * HALF + lane / LPR) * g.ldc + t.n0 +
               wn * HALF + col) * ESZ;
    const int64_t step = RPP * g.ldc * ESZ;   // bytes from pass to pass
    const int wrows = t.mend - (t.m0 + wm * HALF), wcols = static_cast<int>(min<int64_t>(HALF, g.N - (t.n0 + wn * HALF)));
    if (wrows <= 0 || wcols <= 0) return;
    const bool whole = wrows >= HALF && wcols >= HALF;   // of this wave's part
    const bool add = OUT == OUT_ADD_16 || (WIDE && g.accumulate);
    stage_write(Int<0>{});
    each_step<WB * NS * NJ>([&](auto number) {
      constexpr int K = decltype(number)::value, J = K % NJ * NB, ROW = K / (NS * NJ) * 32 + K / NJ % NS * RS;
      Taken v[NP];
      // what is added comes while LDS is read
      [[maybe_unused]] f32x4 plo[NP], phi[NP];
      [[maybe_unused]] u16x8 pu[NP];
      if constexpr (!ROUNDED) {
        if (whole && add) {
          const char* from = c + J * 32 * ESZ;
#pragma unroll
          for (int p = 0; p < NP; ++p, from += step) {
            if constexpr (WIDE) {
              plo[p] = reinterpret_cast<const f32x4_any*>(from)[0];
              phi[p] = reinterpret_cast<const f32x4_any*>(from)[1];
            } else {
              pu[p] = *reinterpret_cast<const u16x8_any*>(from);
            }
          }
        }
      }
      stage_read(v);
      if (!whole) {
        char* to = c + J * 32 * ESZ;
#pragma unroll
        for (int p = 0; p < NP; ++p, to += step) {
          if (ROW + p * RPP >= rows || J * 32 >= cols) continue;
          if (J * 32 + 8 <= cols) {
            if constexpr (WIDE) {
              f32x4_any* d = reinterpret_cast<f32x4_any*>(to);
              if (add) {
                v[p].lo += d[0];
                v[p].hi += d[1];
              }
              d[0] = v[p].lo;
              d[1] = v[p].hi;
            } else {
              if constexpr (!ROUNDED) add_16(v[p], *reinterpret_cast<const u16x8_any*>(to));
              *reinterpret_cast<u16x8_any*>(to) = v[p].u;
            }
          } else {   // the matrix's last columns, one by one out of LDS
            const int row = p * RPP + lane / LPR;
#pragma unroll 1
            for (int e = 0; e < cols - J * 32; ++e) {
              if constexpr (ROUNDED) {
                reinterpret_cast<unsigned short*>(to)[e] = reinterpret_cast<const unsigned short*>(
                    stage + row * (CH * 16) + (((lane % LPR) ^ (row & (CH - 1))) * 16))[e];
              } else {
                float x = reinterpret_cast<const float*>(
                    stage + row * 128 + (((2 * (lane % LPR) + e / 4) ^ (row & 7)) * 16))[e & 3];
                if (add) x += load_c(to, g.c_dtype, e);
                store_c(to, g.c_dtype, e, x);
              }
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
      if constexpr (K + 1 < WB * NS * NJ) stage_write(Int<K + 1>{});
      if (whole) {
        // Rounded results are not read here again: past the cache they leave room for operands.
        // 256-tiles store whole lines (weight gradients of 64 x 1408 x 2048 over 768 columns
        // each 226 -> 189 us, 8192 x 8192 x 512 67 -> 54), 128-tiles half lines, still the
        // faster way (2048 x 4096 x 4096 36.7 -> 35.5 us, x 512 12.1 -> 11.8). Sums with 16-bit
        // results go through the cache, which has their lines already (past it the weight
        // gradients took 361 instead of 357 us), and so do the half lines of fp32 results, which
        // it has to join (past it 8192 x 8192 x 512 took 176 instead of 97 us).
        char* to = c + J * 32 * ESZ;
#pragma unroll
        for (int p = 0; p < NP; ++p, to += step) {
          if constexpr (WIDE) {
            if (add) {
              v[p].lo += plo[p];
              v[p].hi += phi[p];
            }
            reinterpret_cast<f32x4_any*>(to)[0] = v[p].lo;
            reinterpret_cast<f32x4_any*>(to)[1] = v[p].hi;
          } else {
            if constexpr (ROUNDED) {
              __builtin_nontemporal_store(v[p].u, reinterpret_cast<u16x8_any*>(to));
            } else {
              add_16(v[p], pu[p]);
              *reinterpret_cast<u16x8_any*>(to) = v[p].u;
            }
          }
        }
      }
      if constexpr (K % NJ == NJ - 1) {
        c += step * NP;
        asm volatile("" : "+v"(c));   // one row's address at a time: computed ahead they fill the registers
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // WIDE: whether a result of the wave's part of a tile, or one beyond its edges, is not finite
  auto is_far = [&]() {
    float test = 0.0f;
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
      for (int j = 0; j < WB; ++j) {
        if constexpr (TILE == 256) asm volatile("" : "+a"(acc[i][j]));   // they stay in accumulation registers
#pragma unroll
        for (int e = 0; e < 16; ++e) test += acc[i][j][e] * 0.0f;
        if constexpr (TILE == 256) asm volatile("" : "+a"(acc[i][j]), "+v"(test));
        __builtin_amdgcn_sched_barrier(0);
      }
    return __ballot(test != 0.0f) != 0;
  };
  // Such a part is made once more, one block at a time straight from memory: each slice's sum
  // with the scales that fit, times what they were cut by, is added in fp32 (5632 x 2048 x
  // 16383 of NaN: 2.4 ms instead of 0.32).
  auto store_far = [&](const Tile& t) {
    const uint8_t* da = g.a + (g.mode == FP8_DENSE ? t.mat * g.a_batch : 0) + h * 32;
    const uint8_t* db = g.b + (g.mode == FP8_GROUP_K ? 0 : t.mat * g.b_batch) + h * 32;
    const uint8_t* sa = g.sa + (g.mode == FP8_DENSE ? t.mat * g.sa_batch : 0);
    const uint8_t* sb = g.sb + (g.mode == FP8_GROUP_K ? 0 : t.mat * g.sb_batch);
#pragma unroll 1
    for (int block = 0; block < WB * WB; ++block) {
      const int m = t.m0 + wm * HALF + block / WB * 32, n = t.n0 + wn * HALF + block % WB * 32;
      if (m >= t.mend || n >= g.N) continue;
      const int64_t ra = min(m + r, t.mend - 1), rb = min<int64_t>(n + r, g.N - 1);
      f32x16 total;
#pragma unroll
      for (int e = 0; e < 16; ++e) total[e] = 0.0f;
#pragma unroll 1
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        const int ba = sa[ra * g.s_pitch + kb], bb = sb[rb * g.s_pitch + kb];
        const float fsa = scale_value(near_scale<FA>(ba)), fsb = scale_value(near_scale<FB>(bb));
        f32x16 sum;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = 0.0f;
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {   // 16 of the lane's 64 bytes
          const int at = kb * 128 + (p >> 1) * 64 + (p & 1) * 16;
          const i32x4 xa = *reinterpret_cast<const i32x4*>(da + ra * g.pitch + at);
          const i32x4 xb = *reinterpret_cast<const i32x4*>(db + rb * g.pitch + at);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(to_bf16x8<FB>(xb[2 * s], xb[2 * s + 1], fsb),
                                                          to_bf16x8<FA>(xa[2 * s], xa[2 * s + 1], fsa), sum, 0, 0, 0);
        }
        const float rest = rest_scale<FA>(ba);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          total[e] += sum[e] * (rest * rest_scale<FB>(__shfl(bb, (e >> 2) * 8 + h * 4 + (e & 3), 64)));
          if ((e & 3) == 3) __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t col = n + (e >> 2) * 8 + h * 4 + (e & 3);
        if (m + r >= t.mend || col >= g.N) continue;
        const int64_t at = (g.mode == FP8_GROUP_ROWS ? 0 : t.mat * g.c_batch) + (m + r) * g.ldc + col;
        store_c(g.c, g.c_dtype, at, total[e] + (g.accumulate ? load_c(g.c, g.c_dtype, at) : 0.0f));
      }
    }
  };

  int index = blockIdx.x;
  if (index >= total) return;
  Tile cur = tile_at(index);
  int slot = 0;   // the part of `scales` in use
  scales_of(slot, cur, cur.kb0 >> 4, true);
  load_slice(buf0, cur.a, cur.b, cur.na, cur.nb, cur.kb0, cur.kb1, 0);
  load_slice(buf1, cur.a, cur.b, cur.na, cur.nb, cur.kb0, cur.kb1, 1);
  publish();
  read_scales(0, slot, cur.kb0);
  read(0, buf0);
  clear();
  for (;;) {
    index += gridDim.x;
    const bool more = index < total;
    Tile nxt = cur;
    if (more) nxt = tile_at(index);
    else nxt.na = nxt.nb = nxt.kb0 = nxt.kb1 = 0;   // fetched as zeros, never used
    const int n = slices_of(cur);
    int t = 0, kb = cur.kb0;
    bool fetched = false;   // the next tile's first scales
    while (t < n) {
      // the scales behind this part's; their place was last read before the last barrier
      const int part = kb >> 4;
      fetched = ((cur.kb0 + n - 1) >> 4) == part;
      if (fetched) scales_of(slot ^ 1, nxt, nxt.kb0 >> 4, more);
      else scales_of(slot ^ 1, cur, part + 1, true);
      for (; t < n && (kb >> 4) == part; t += 2, kb += 2) {
        // the slices after next: the next tile's behind the last ones
        const bool last = t + 2 >= n;
        const uint8_t* la = last ? nxt.a : cur.a;
        const uint8_t* lb = last ? nxt.b : cur.b;
        const int lna = last ? nxt.na : cur.na, lnb = last ? nxt.nb : cur.nb;
        const int lk0 = last ? nxt.kb0 : cur.kb0, lk1 = last ? nxt.kb1 : cur.kb1, ls = last ? 0 : t + 2;
        // slice t, first period
        read(1, buf0);
        mask_scales(0, kb < cur.kb1);
        multiply(Int<0>{}, Int<0>{});
        schedule(Int<0>{});
        publish();
        // second period: slice t + 1 is there, buf0 is free
        read_scales(1, ((kb + 1) >> 4) == part ? slot : slot ^ 1, kb + 1);
        read(0, buf1);
        load_slice(buf0, la, lb, lna, lnb, lk0, lk1, ls);
        multiply(Int<1>{}, Int<0>{});
        schedule(Int<1>{});
        // slice t + 1
        read(1, buf1);
        mask_scales(1, kb + 1 < cur.kb1);
        multiply(Int<0>{}, Int<1>{});
        schedule(Int<0>{});
        publish();
        read_scales(0, !last && ((kb + 2) >> 4) == part ? slot : slot ^ 1, last ? nxt.kb0 : kb + 2);
        read(0, buf0);
        load_slice(buf1, la, lb, lna, lnb, lk0, lk1, ls + 1);
        multiply(Int<1>{}, Int<1>{});
        schedule(Int<1>{});
      }
      slot ^= 1;
    }
    if (!fetched) {   // the last slice alone reached into a new part (which is in `slot`)
      scales_of(slot ^ 1, nxt, nxt.kb0 >> 4, more);
      publish();
      slot ^= 1;
      read_scales(0, slot, nxt.kb0);
    }
    // no load may be on its way into LDS when the workgroup ends
    if (!more) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if (WIDE && __builtin_expect(is_far(), 0)) store_far(cur);
    else store(cur);
    if (!more) return;
    cur = nxt;
    clear();
  }
}

template <int FA, int FB, int OUT, int TILE>
__global__ __launch_bounds__(256, TILE == 256 ? 1 : 2) void fp8_tile_kernel(Fp8Gemm g, int mtiles, int ntiles) {
  tile_product<FA, FB, OUT, TILE>(g, mtiles, ntiles);
}

// Which kernel a product takes.
enum { FP8_FEW_16 = 0, FP8_FEW_32 = 1, FP8_FEW_64 = 2, FP8_TILE_128 = 3, FP8_TILE_256 = 4 };

static int tile_rows(int kind) {
  const int rows[] = {16, 32, 64, 128, 256};
  return rows[kind];
}

// The kernel with the least estimated time: rounds of 256 workgroups times what a round
// costs, some us and some per block of the contraction (measured, 8-bit and fp32 results;
// 128-tiles run two workgroups per CU, counted as two rounds). It weighs reading B again
// for every 16 to 64 rows against a wide tile's empty rows and idle CUs. For instance
// (us, few rows 16 / 32 / 64, tiles 128 / 256; bf16, K = 4096):
//   1 x 11008: 12 / 15 / 18 / 23 / 39       64 x 4096: 20 / 15 / 13.5 / 16 / 39
//   128 x 11008: 89 / 68 / 62 / 25 / 39     2048 x 4096: - / - / - / 36 / 45
//   256 x 4096: 66 / 50 / 43 / 17 / 39      8192 x 11008: - / - / - / 342 / 281
// fp32 results: 64 x 4096: 20 / 18 / 14 / 33 / 93    8192 x 11008: - / - / - / 648 / 615
// Of groups only the total of their rows is known here; half a tile is added for each.
Fp8Plan plan_fp8_gemm(int64_t M, int64_t N, int64_t kb, int32_t mode, int64_t batch, bool wide) {
  struct Cost { double start, round, block; };
  static const Cost cost[2][5] = {
      {{2.5, 0.3, 0.13}, {2.7, 0.3, 0.20}, {3.2, 0.3, 0.32}, {3.5, 2.0, 0.48}, {4.0, 5.0, 1.40}},
      {{2.6, 0.4, 0.13}, {3.0, 0.4, 0.22}, {3.8, 0.4, 0.36}, {3.5, 4.0, 1.05}, {4.0, 9.0, 3.20}}};
  const double blocks = mode == FP8_GROUP_K ? static_cast<double>(kb) / static_cast<double>(batch) : static_cast<double>(kb);
  int best = 0;
  double least = 0.0;
  for (int kind = FP8_FEW_16; kind <= FP8_TILE_256; ++kind) {
    const int64_t tm = tile_rows(kind), tn = kind < FP8_TILE_128 ? 16 : tm;
    const int64_t rows = mode == FP8_GROUP_ROWS ? (2 * M / tm + batch + 1) / 2 : (M + tm - 1) / tm * batch;
    const Cost& c = cost[wide][kind];
    const double rounds = std::ceil(static_cast<double>(rows * ((N + tn - 1) / tn)) / 256.0);
    const double us = c.start + rounds * (c.round + c.block * blocks);
    if (kind == FP8_FEW_16 || us < least) {
      best = kind;
      least = us;
    }
  }
  return {best};
}

template <int FA, int FB, int OUT>
static void launch_tiles(const Fp8Plan& p, const Fp8Gemm& g, int64_t total, int m, int n, hipStream_t s) {
  if (p.kind == FP8_TILE_128)   // two workgroups per CU, walking over the tiles
    hipLaunchKernelGGL((fp8_tile_kernel<FA, FB, OUT, 128>), dim3(std::min<int64_t>(total, 512)), dim3(256), 0, s, g, m, n);
  else                          // one per CU
    hipLaunchKernelGGL((fp8_tile_kernel<FA, FB, OUT, 256>), dim3(std::min<int64_t>(total, 256)), dim3(256), 0, s, g, m, n);
}

template <int FA, int FB>
static hipError_t launch(const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  const int tm = tile_rows(p.kind), tn = p.kind < FP8_TILE_128 ? 16 : tm;
  const int64_t nt = (g.N + tn - 1) / tn;
  int64_t mt = (g.M + tm - 1) / tm, z = g.batch;
  if (g.mode == FP8_GROUP_ROWS) {   // every group may end in a part of a tile
    mt = std::min<int64_t>(g.M, g.M / tm + g.batch);
    z = 1;
  }
  const int64_t total = mt * nt * z;
  if (total <= 0) return hipSuccess;
  if (total > 0x7fffffff) return hipErrorInvalidValue;
  const int m = static_cast<int>(mt), n = static_cast<int>(nt);
  const bool wide = g.c_dtype == MUON_DTYPE_F32;
  if (p.kind < FP8_TILE_128) {
    const dim3 grid = flat_grid(total), block(64 * kFewWaves);
#define MUON_FEW(W, MT) hipLaunchKernelGGL((fp8_few_rows_kernel<FA, FB, W, MT>), grid, block, 0, s, g, m, n)
    if (p.kind == FP8_FEW_16) {
      if (wide) MUON_FEW(true, 1);
      else MUON_FEW(false, 1);
    } else if (p.kind == FP8_FEW_32) {
      if (wide) MUON_FEW(true, 2);
      else MUON_FEW(false, 2);
    } else {
      if (wide) MUON_FEW(true, 4);
      else MUON_FEW(false, 4);
    }
#undef MUON_FEW
  } else if (wide) {
    launch_tiles<FA, FB, OUT_F32>(p, g, total, m, n, s);
  } else if (g.accumulate) {
    launch_tiles<FA, FB, OUT_ADD_16>(p, g, total, m, n, s);
  } else if (g.c_dtype == MUON_DTYPE_BF16) {
    launch_tiles<FA, FB, OUT_BF16>(p, g, total, m, n, s);
  } else {
    launch_tiles<FA, FB, OUT_F16>(p, g, total, m, n, s);
  }
  return hipGetLastError();
}

const char* fp8_gemm_kind(const Fp8Plan& p) {
  return p.kind < FP8_TILE_128 ? "fp8_gemm_few_rows" : p.kind == FP8_TILE_128 ? "fp8_gemm_128" : "fp8_gemm_256";
}

hipError_t launch_fp8_gemm(int fmt_a, int fmt_b, const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  if (fmt_a == MUON_FP8_E4M3) return fmt_b == MUON_FP8_E4M3 ? launch<0, 0>(p, g, s) : launch<0, 1>(p, g, s);
  return fmt_b == MUON_FP8_E4M3 ? launch<1, 0>(p, g, s) : launch<1, 1>(p, g, s);
}

}  // namespace muon
