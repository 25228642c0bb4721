// Launch interfaces of the norm, embedding, clipping and attention kernels (internal to
// libmuonstep). Every argument is checked by the C entry points.
#pragma once

#include "common.hpp"

namespace muon {

struct NormArgs {
  const void* x;             // rows x cols
  const void* residual;      // optional
  const void* weight;        // cols elements of weight_dtype; NULL: ones
  int64_t ld_x, ld_residual;
  int64_t rows, cols;
  int32_t weight_dtype;
  float eps;
  double inv_cols;           // forward
  void* sum;                 // forward: optional outputs
  void* y;
  int64_t ld_sum, ld_y;
  uint8_t* q;                // rows x qp, scales rows x qs
  uint8_t* s;
  int64_t qp, qs;
  int32_t format;
  float* rstd;
  const float* rstd_in;      // backward
  const void* dy;
  const void* dsum;          // optional
  void* dx;                  // optional
  int64_t ld_dy, ld_dsum, ld_dx;
  float* partial;            // weight gradients of norm_blocks() x cols (NULL: not wanted)
  void* dweight;
  int32_t dweight_dtype, accumulate;
};
hipError_t launch_rms_norm(int dtype, const NormArgs& a, hipStream_t s);
int32_t norm_blocks(int64_t rows, int64_t cols);   // workgroups of the gradient
hipError_t launch_rms_norm_backward(int dtype, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_weight(const NormArgs& a, hipStream_t s);

struct EmbeddingArgs {
  const void* ids;           // int32 or int64
  int32_t wide_ids;
  int32_t bits, passes;      // of the sort: digits of `bits` bits
  int64_t tokens, vocab, cols;
  float scale;
  const void* table;         // forward
  int32_t table_dtype, accumulate;
  void* y;
  const void* dy;            // backward
  void* dtable;
  int64_t ld_table, ld_y;
  int32_t *keys[2], *slots[2];
  int32_t* hist;             // blocks x kSortBins
  int32_t blocks;
  int64_t per_block;
  uint8_t* touched;          // a byte per row of the table (NULL: not wanted)
  float* partial;            // 2 per chunk x cols
  int32_t chunk;             // sorted tokens that one wave sums: 8 or 32
};
constexpr int kSortBins = 256;
int32_t sort_blocks(int64_t n);
hipError_t launch_embedding(int dtype, const EmbeddingArgs& a, hipStream_t s);
// One block: the whole sort. Several: a pass's counts, then its placing.
hipError_t launch_sort_all(const EmbeddingArgs& a, hipStream_t s);
hipError_t launch_sort_hist(const EmbeddingArgs& a, int pass, hipStream_t s);
hipError_t launch_sort_place(const EmbeddingArgs& a, int pass, hipStream_t s);
hipError_t launch_embedding_sum(int dtype, const EmbeddingArgs& a, hipStream_t s);
hipError_t launch_embedding_join(const EmbeddingArgs& a, hipStream_t s);

// Tensors of one launch, passed by value.
struct ClipTensor {
  const void* in;
  void* out;
  int64_t n;
  int32_t first;             // its first workgroup
  int16_t in_dtype, out_dtype;
};
constexpr int kClipTensors = 120;
struct ClipArgs {
  ClipTensor t[kClipTensors];
  int32_t n, blocks;
  int32_t chunk;             // elements of a workgroup
  float max_norm;
  double* partial;           // a sum per workgroup
  const double* sumsq;
  float* norm;
};
hipError_t launch_grad_sumsq(const ClipArgs& a, hipStream_t s);
hipError_t launch_sum_partials(const double* partial, int64_t n, bool accumulate, double* out, hipStream_t s);
hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t s);

}  // namespace muon
