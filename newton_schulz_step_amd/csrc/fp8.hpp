// Launch interfaces of the 8-bit and mixture-of-experts kernels (internal to
// libmuonstep). Every argument is checked by the C entry points.
#pragma once

#include "common.hpp"

namespace muon {

// Grids of up to 2^31 workgroups. A grid dimension takes less than 2^32 threads, so beyond
// 2^20 workgroups the number is split over two dimensions; the last ones may lie behind the
// count, and kernels leave those alone.
constexpr int kGridBits = 20;
inline dim3 flat_grid(int64_t blocks) {
  const int64_t x = blocks < (int64_t(1) << kGridBits) ? blocks : int64_t(1) << kGridBits;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
}
__device__ __forceinline__ uint32_t flat_block() { return (blockIdx.y << kGridBits) + blockIdx.x; }

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Row pitches of a quantised operand with `cols` columns (bytes).
inline int64_t fp8_data_pitch(int64_t cols) { return round_up(cols, MUON_FP8_BLOCK); }
inline int64_t fp8_scale_pitch(int64_t cols) { return round_up((cols + MUON_FP8_BLOCK - 1) / MUON_FP8_BLOCK, 4); }

struct QuantArgs {
  const void* x;
  int64_t x_batch, ldx;         // elements
  int64_t src_rows;             // rows of the source
  const int32_t* row_index;     // optional, see muon_fp8_source_t
  int32_t row_div;
  const float* row_weight;      // optional
  int64_t n_weights;
  int64_t rows, cols;           // of the quantised matrix
  int32_t row_tiles, col_tiles, total_tiles;
  uint8_t* q;                   // rows x qp, scales rows x qs (NULL: not wanted)
  uint8_t* s;
  uint8_t* qt;                  // cols x tp, scales cols x ts (NULL: not wanted)
  uint8_t* st;
  int64_t qp, qs, tp, ts;
};
hipError_t launch_fp8_quantize(int x_dtype, int format, bool blocks, const QuantArgs& a, hipStream_t s);

// C (+)= A B^T of quantised operands. Batches and groups: see the C ABI.
enum { FP8_DENSE = 0, FP8_GROUP_ROWS = 1, FP8_GROUP_K = 2 };
struct Fp8Gemm {
  const uint8_t *a, *b;          // data
  const uint8_t *sa, *sb;        // scales
  int64_t a_batch, b_batch;      // bytes between matrices
  int64_t sa_batch, sb_batch;
  int64_t pitch, s_pitch;        // bytes of a row of a and of b (the same K)
  int64_t M, N;
  int32_t kb;                    // blocks of 128 along K
  int32_t mode, batch;           // batch: matrices, or groups
  const int32_t* offsets;        // groups
  void* c;
  int64_t c_batch, ldc;          // elements
  int32_t c_dtype, accumulate;
};
struct Fp8Plan {
  int32_t kind;   // which kernel, see plan_fp8_gemm
};
Fp8Plan plan_fp8_gemm(int64_t M, int64_t N, int64_t kb, int32_t mode, int64_t batch, bool wide);
hipError_t launch_fp8_gemm(int fmt_a, int fmt_b, const Fp8Plan& p, const Fp8Gemm& g, hipStream_t s);
const char* fp8_gemm_kind(const Fp8Plan& p);   // its name in the launch statistics

struct RouteArgs {
  const void* logits;
  int64_t ld, tokens;
  const float* bias;
  int32_t experts, top_k, n_groups, top_groups, group_top;
  int32_t score, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};
hipError_t launch_route(int dtype, const RouteArgs& a, hipStream_t s);

struct RouteBackArgs {
  const float* dweights;
  const void* logits;
  int64_t ld, tokens, ld_d;
  const int32_t* ids;
  int32_t experts, top_k, score, renormalize;
  float scale;
  void* dlogits;
};
hipError_t launch_route_backward(int dtype, const RouteBackArgs& a, hipStream_t s);

struct OrderArgs {
  const int32_t* ids;
  int64_t n;
  int32_t experts, align;
  int32_t *offsets, *counts, *rows, *pos;
  int64_t capacity;
  int32_t* hist;      // blocks x experts, where blocks > 1
  int32_t blocks;
  int64_t per_block;  // slots of a block
};
int32_t order_blocks(int64_t n);   // 1: a single launch without workspace
hipError_t launch_order_hist(const OrderArgs& a, hipStream_t s);
hipError_t launch_order_place(const OrderArgs& a, hipStream_t s);

struct CombineArgs {
  const void* o;
  int64_t o_rows, cols, ld_o;
  const int32_t* pos;
  const float* weights;
  int64_t tokens;
  int32_t top_k;
  void* y;              // forward
  int64_t ld_y;
  const void* dy;       // backward
  int64_t ld_dy;
  float* dweights;
  void* d_o;
  int64_t ld_do;
};
hipError_t launch_combine(int dtype, const CombineArgs& a, hipStream_t s);
hipError_t launch_combine_backward(int dtype, const CombineArgs& a, hipStream_t s);

}  // namespace muon
