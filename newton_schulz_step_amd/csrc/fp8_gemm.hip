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
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "fp8.hpp"

namespace muon {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Group of a row tile. Every wave of the workgroup finds it by itself: 64 groups at a
// time, a prefix sum of their tile counts. Returns false for a tile beyond the last
// group's.
__device__ __forceinline__ bool find_group(const int32_t* offsets, int n_groups, int limit, int tile_rows, int tile,
                                           int& group, int& first, int& end) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int g0 = 0; g0 < n_groups; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < n_groups) {
      lo = min(max(offsets[g], 0), limit);
      hi = min(max(offsets[g + 1], lo), limit);
    }
    const int n = (hi - lo + tile_rows - 1) / tile_rows;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (tile < base + total) {
      const int l = __builtin_ctzll(__ballot(base + incl > tile));
      group = g0 + l;
      first = __builtin_amdgcn_readlane(lo, l) + (tile - base - __builtin_amdgcn_readlane(incl - n, l)) * tile_rows;
      end = __builtin_amdgcn_readlane(hi, l);
      return true;
    }
    base += total;
  }
  return false;
}

// What a workgroup computes (the same in all its lanes): rows [m0, mend) of A (a tile of
// them), matrix `mat` of B and C, blocks [kb0, kb1) of the contraction.
struct Work {
  int m0, mend;
  int mat, amat, bmat;
  int kb0, kb1;
};

template <int TM>
__device__ __forceinline__ bool find_work(const Fp8Gemm& g, int mtile, int z, Work& w) {
  w.kb0 = 0;
  w.kb1 = g.kb;
  w.m0 = mtile * TM;
  w.mend = static_cast<int>(g.M);
  w.mat = w.amat = w.bmat = z;
  if (g.mode == FP8_GROUP_ROWS) {
    w.amat = 0;
    if (!find_group(g.offsets, g.batch, static_cast<int>(g.M), TM, mtile, w.mat, w.m0, w.mend)) return false;
    w.bmat = w.mat;
  } else if (g.mode == FP8_GROUP_K) {
    w.amat = w.bmat = 0;
    const int limit = g.kb * 128;
    const int lo = min(max(g.offsets[z], 0), limit);
    const int hi = min(max(g.offsets[z + 1], lo), limit);
    w.kb0 = __builtin_amdgcn_readfirstlane(lo / 128);
    w.kb1 = __builtin_amdgcn_readfirstlane(hi > lo ? (hi + 127) / 128 : lo / 128);
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

// ---------------------------------------------------------------------------
// Tiles: TILE x TILE outputs per workgroup (256 or 128), four waves in a 2 x 2 grid, each
// owning (TILE / 2)^2 outputs as 32 x 32 blocks in registers.
//
// Slices of both operands, one block (128 bytes) of every row, go straight from memory to
// LDS (no registers) into two buffers. A slice is multiplied in two periods of 64 bytes,
// one 32 x 32 x 64 instruction per block pair each. During a period a wave multiplies
// from one set of registers and reads the next period's operands from LDS into the other
// set, so a slice's buffer has been read by the end of its first period; one barrier
// then frees it and publishes the next slice, and the loads of the slice after next are
// issued into it, spread over the second period. They have one to two periods (256-tiles:
// 1000 to 2000 matrix cycles) to arrive. Rows are fetched 128 bytes at a time because
// requests, not bytes, bound the way from the last-level cache: with four buffers of 64
// bytes per row the same loop was 10% slower, resident data or not.
//
// LDS rows of a slice are 128 bytes, eight 16-byte chunks; chunk c of row r is stored at
// place c ^ swz(r), so lanes that read one chunk of neighbouring rows spread over the
// banks. A direct load writes consecutive lanes to consecutive places, so the lanes fetch
// permuted chunks instead. Beyond the last slice the loads repeat it (in bounds, never
// used).
//
// The loop body is two slices: their buffers are then known at compile time (and the
// compiler waits for exactly the loads of the buffer that is read). An odd last slice is
// paired with a repeated one whose scales are set to 2^-127, 2^-254 together, which adds
// nothing (8-bit products are below 2^33).
//
// Scales: 16 bytes (16 blocks) of every row at a time, also by direct loads, in two parts
// of LDS: while one is used the other is fetched, once in 16 slices. (One word at a time
// fetches 64 cache lines for 256 bytes; with that in every fourth slice the loop was 12%
// slower.) Reads behind the operand's last scale give zeros: the resource's bounds.
//
// Four waves of 128 x 128 read 32 KB of a 256-tile's LDS per 1024 matrix cycles each: 75%
// of the LDS rate with the writes. Smaller wave tiles would be bound by LDS.

__device__ __forceinline__ int row_swizzle(int r) { return (r ^ ((r >> 3) & 3)) & 7; }   // of r modulo 32

template <int V> using Int = std::integral_constant<int, V>;

#define MUON_GLDS(rsrc, lds, size, voff, soff)                                                              \
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MUON_LDS void*)(lds), size, voff, soff, 0, 0)

// 8 neighbouring results in one row, 16-byte aligned (WIDE: fp32 results).
template <bool WIDE>
__device__ __forceinline__ void store_row8(const Fp8Gemm& g, int64_t at, float (&v)[8]) {
  if constexpr (WIDE) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + at);
    f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if (g.accumulate) {
      a += p[0];
      b += p[1];
    }
    p[0] = a;
    p[1] = b;
  } else {
    u16x8* p = reinterpret_cast<u16x8*>(static_cast<unsigned short*>(g.c) + at);
    if (g.accumulate) {
      const u16x8 u = *p;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += g.c_dtype == MUON_DTYPE_BF16 ? bf16_bits_to_f32(u[e]) : f16_bits_to_f32(u[e]);
    }
    u16x8 u;
    if (g.c_dtype == MUON_DTYPE_BF16) {
      __bf16 o[8];
      rne<__bf16, 8>(v, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __builtin_bit_cast(unsigned short, o[e]);
    } else {
      _Float16 o[8];
      rne<_Float16, 8>(v, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __builtin_bit_cast(unsigned short, o[e]);
    }
    *p = u;
  }
}

template <int FA, int FB, bool WIDE, int TILE>
__device__ __forceinline__ void tile_product(const Fp8Gemm& g, int mtiles, int ntiles, int total) {
  constexpr int HALF = TILE / 2, WB = HALF / 32;
  constexpr int SLICE = TILE * 128;             // bytes of one operand's slice
  constexpr int LOADS = TILE / 32;              // 1-KB loads per wave, operand and slice
  __shared__ __align__(1024) char buf0[2 * SLICE], buf1[2 * SLICE];
  __shared__ __align__(16) unsigned char scales[2][2 * TILE * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // Workgroups are dealt round-robin over the eight XCDs. In every round of the chip each
  // XCD takes consecutive tiles (its own last-level cache then sees neighbours), and all
  // XCDs stay close together. Within a matrix, bands of four tile columns are walked row
  // by row.
  constexpr int ROUND = TILE == 256 ? 256 : 512;
  const int chunk = blockIdx.x / ROUND, inside = blockIdx.x % ROUND;
  const int size = min(ROUND, total - chunk * ROUND);
  const int b = chunk * ROUND + (inside & 7) * (size / 8) + min(inside & 7, size % 8) + (inside >> 3);
  const int per = mtiles * ntiles;
  const int z = b / per;
  const int rest = b - z * per;
  const int band = rest / (4 * mtiles);
  const int first = band * 4, width = min(4, ntiles - first);
  const int in = rest - band * 4 * mtiles;
  const int mt = in / width, nt = first + in % width;
  Work w;
  if (!find_work<TILE>(g, mt, z, w)) return;
  const int64_t m0 = w.m0, n0 = static_cast<int64_t>(nt) * TILE;
  const int mrows = static_cast<int>(min<int64_t>(TILE, w.mend - m0)), nrows = static_cast<int>(min<int64_t>(TILE, g.N - n0));

  // resources of the tile's rows and per-lane offsets (rows beyond the tile repeat its last)
  const int pitch = static_cast<int>(g.pitch), sp = static_cast<int>(g.s_pitch);
  const uint8_t* pa = g.a + w.amat * g.a_batch + m0 * g.pitch;
  const uint8_t* pb = g.b + w.bmat * g.b_batch + n0 * g.pitch;
  const uint8_t* psa = g.sa + w.amat * g.sa_batch + m0 * g.s_pitch;
  const uint8_t* psb = g.sb + w.bmat * g.sb_batch + n0 * g.s_pitch;
  const auto ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pa), 0, mrows * pitch, 0x00027000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pb), 0, nrows * pitch, 0x00027000);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(psa), 0, mrows * sp, 0x00027000);
  const auto rsb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(psb), 0, nrows * sp, 0x00027000);
  int va[LOADS], vb[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = (wave * LOADS + i) * 8 + (lane >> 3);
    const int c = ((lane & 7) ^ row_swizzle(r)) * 16;
    va[i] = min(r, mrows - 1) * pitch + c;
    vb[i] = min(r, nrows - 1) * pitch + c;
  }
  const int nk = w.kb1 - w.kb0;                         // slices
  const int k0 = w.kb0 * 128;
  // scales, 64 rows per load: of a 256-tile each wave fetches 64 rows of both operands, of
  // a 128-tile waves 0 and 1 rows of A, 2 and 3 of B
  const bool sfirst = TILE == 256 || wave < 2;
  const int srow = (TILE == 256 ? wave : wave & 1) * 64;
  const int vs0 = min(srow + lane, (sfirst ? mrows : nrows) - 1) * sp;
  const int vs1 = min(srow + lane, nrows - 1) * sp;

  // per-lane read offsets within a slice, period 0: two neighbouring chunks of row lane %
  // 32 (the second one at ^ 16, those of period 1 at ^ 64; the swizzle only depends on the
  // row modulo 32)
  const int r = lane & 31, h = lane >> 5;
  const int chunk0 = ((2 * h) ^ row_swizzle(r)) * 16;
  const int ao = (wm * HALF + r) * 128 + chunk0, bo = SLICE + (wn * HALF + r) * 128 + chunk0;

  f32x16 acc[WB][WB];
#pragma unroll
  for (int i = 0; i < WB; ++i)
#pragma unroll
    for (int j = 0; j < WB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto load_slice = [&](char* to, int t) {
    const int so = k0 + min(t, nk - 1) * 128;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) MUON_GLDS(ra, to + (wave * LOADS + i) * 1024, 16, va[i], so);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) MUON_GLDS(rb, to + SLICE + (wave * LOADS + i) * 1024, 16, vb[i], so);
  };
  auto load_scales = [&](int c) {   // blocks 16 c .. 16 c + 15
    unsigned char* to = scales[c & 1];
    if (sfirst) MUON_GLDS(rsa, to + srow * 16, 16, vs0, c * 16);
    else MUON_GLDS(rsb, to + (TILE + srow) * 16, 16, vs0, c * 16);
    if constexpr (TILE == 256) MUON_GLDS(rsb, to + (TILE + srow) * 16, 16, vs1, c * 16);
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
  // scale bytes of the lane's rows of A, then of B, for the two slices of a body
  int sc[2][2 * WB];
  auto read_scales = [&](int set, int kb) {
    const unsigned char* from = scales[(kb >> 4) & 1] + (kb & 15);
    const int mask = kb < w.kb1 ? 255 : 0;
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      sc[set][i] = from[(wm * HALF + i * 32 + r) * 16] & mask;
      sc[set][WB + i] = from[(TILE + wn * HALF + i * 32 + r) * 16] & mask;
    }
  };
  auto publish = [&]() {   // own reads and loads are done, then everybody's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  if (nk > 0) {
    load_scales(w.kb0 >> 4);
    load_slice(buf0, 0);
    load_slice(buf1, 1);
    publish();
    read_scales(0, w.kb0);
    read(0, buf0);

    auto multiply = [&](auto set, auto slice) {
      constexpr int SET = decltype(set)::value, U = decltype(slice)::value;
      if constexpr (WIDE) {
        float fs[2 * WB];
#pragma unroll
        for (int i = 0; i < 2 * WB; ++i) fs[i] = scale_value(sc[U][i], 0);
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
        constexpr int NM = WB * WB, NR = 4 * WB, NL = decltype(loads)::value ? 2 * LOADS : 0;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x100, NR / NM > 1 ? NR / NM : 1, 0);   // LDS reads
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                           // MFMA
          if constexpr (NL > 0) __builtin_amdgcn_sched_group_barrier(0x020, NL / NM, 0);  // loads to LDS
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    int t = 0, kb = w.kb0;
    while (t < nk) {
      // the scales behind this part's; their place was last read before the last barrier
      const int part = kb >> 4;
      load_scales(part + 1);
      for (; t < nk && (kb >> 4) == part; t += 2, kb += 2) {
        // slice t, first period
        read(1, buf0);
        multiply(Int<0>{}, Int<0>{});
        schedule(Int<0>{});
        publish();
        // second period: slice t + 1 is there, buf0 is free
        read_scales(1, kb + 1);
        read(0, buf1);
        load_slice(buf0, t + 2);
        multiply(Int<1>{}, Int<0>{});
        schedule(Int<1>{});
        // slice t + 1
        read(1, buf1);
        multiply(Int<0>{}, Int<1>{});
        schedule(Int<0>{});
        publish();
        read_scales(0, kb + 2);
        read(0, buf0);
        load_slice(buf1, t + 3);
        multiply(Int<1>{}, Int<1>{});
        schedule(Int<1>{});
      }
    }
    // the last loads land before the buffers are used again
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Results: 32 rows of a wave at a time through its own part of LDS, then whole rows,
  // 16 bytes per lane where the rows are aligned for it.
  constexpr int SP = HALF + 4;
  float* stage = reinterpret_cast<float*>((wave < 2 ? buf0 : buf1) + (wave & 1) * SLICE);
  static_assert(32 * SP * 4 <= SLICE, "staging fits");
  const int64_t cbase = g.mode == FP8_GROUP_ROWS ? 0 : w.mat * g.c_batch;
  const int64_t nw = n0 + wn * HALF;
  const int ncols = static_cast<int>(max<int64_t>(0, min<int64_t>(HALF, g.N - nw)));
#pragma unroll
  for (int i = 0; i < WB; ++i) {
    const int64_t mw = m0 + wm * HALF + i * 32;
    const int rows = static_cast<int>(max<int64_t>(0, min<int64_t>(32, w.mend - mw)));
#pragma unroll
    for (int j = 0; j < WB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(stage + r * SP + j * 32 + 8 * e + 4 * h) =
            f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (g.c_vec && ncols == HALF) {
      constexpr int LPR = HALF / 8, RPP = 64 / LPR;
      const int col = (lane % LPR) * 8;
#pragma unroll
      for (int p = 0; p < 32 / RPP; ++p) {
        const int row = p * RPP + lane / LPR;
        if (row < rows) {
          float v[8];
          const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + row * SP + col);
          const f32x4 hi = *reinterpret_cast<const f32x4*>(stage + row * SP + col + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
          store_row8<WIDE>(g, cbase + (mw + row) * g.ldc + nw + col, v);
        }
      }
    } else {
      for (int row = 0; row < rows; ++row) {
        const int64_t at = cbase + (mw + row) * g.ldc + nw;
        for (int col = lane; col < ncols; col += 64) {
          float v = stage[row * SP + col];
          if (g.accumulate) v += load_c(g.c, g.c_dtype, at + col);
          store_c(g.c, g.c_dtype, at + col, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FA, int FB, bool WIDE, int TILE>
__global__ __launch_bounds__(256, TILE == 256 ? 1 : 2) void fp8_tile_kernel(Fp8Gemm g, int mtiles, int ntiles,
                                                                           int total) {
  tile_product<FA, FB, WIDE, TILE>(g, mtiles, ntiles, total);
}

// Which kernel a product takes.
enum { FP8_FEW_ROWS = 0, FP8_TILE_128 = 1, FP8_TILE_256 = 2 };

Fp8Plan plan_fp8_gemm(int64_t M, int64_t N, int64_t, int32_t mode, int64_t batch, bool) {
  const int64_t mats = mode == FP8_GROUP_ROWS ? 1 : batch;
  auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t) * mats; };
  if (M <= 32 || N <= 16) return {FP8_FEW_ROWS, 1};
  if (tiles(256) >= 128) return {FP8_TILE_256, 1};
  return {FP8_TILE_128, 1};
}

template <int FA, int FB, bool WIDE>
static hipError_t launch(const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  const int tm = p.kind == FP8_FEW_ROWS ? 16 : p.kind == FP8_TILE_128 ? 128 : 256;
  const int64_t nt = (g.N + tm - 1) / tm;
  int64_t mt = (g.M + tm - 1) / tm, z = g.batch;
  if (g.mode == FP8_GROUP_ROWS) {   // every group may end in a part of a tile
    mt = std::min<int64_t>(g.M, g.M / tm + g.batch);
    z = 1;
  }
  const int64_t total = mt * nt * z;
  if (total <= 0) return hipSuccess;
  if (total > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(total));
  const int m = static_cast<int>(mt), n = static_cast<int>(nt);
  if (p.kind == FP8_FEW_ROWS)
    hipLaunchKernelGGL((fp8_few_rows_kernel<FA, FB, WIDE>), grid, dim3(64 * kFewWaves), 0, s, g, m, n);
  else if (p.kind == FP8_TILE_128)
    hipLaunchKernelGGL((fp8_tile_kernel<FA, FB, WIDE, 128>), grid, dim3(256), 0, s, g, m, n, static_cast<int>(total));
  else
    hipLaunchKernelGGL((fp8_tile_kernel<FA, FB, WIDE, 256>), grid, dim3(256), 0, s, g, m, n, static_cast<int>(total));
  return hipGetLastError();
}

template <int FA, int FB>
static hipError_t launch_dtype(const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  return g.c_dtype == MUON_DTYPE_F32 ? launch<FA, FB, true>(p, g, s) : launch<FA, FB, false>(p, g, s);
}

hipError_t launch_fp8_gemm(int fmt_a, int fmt_b, const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s) {
  if (fmt_a == MUON_FP8_E4M3) return fmt_b == MUON_FP8_E4M3 ? launch_dtype<0, 0>(p, g, s) : launch_dtype<0, 1>(p, g, s);
  return fmt_b == MUON_FP8_E4M3 ? launch_dtype<1, 0>(p, g, s) : launch_dtype<1, 1>(p, g, s);
}

hipError_t launch_fp8_reduce(const Fp8Gemm&, hipStream_t) { return hipSuccess; }

}  // namespace muon
