// Launch interface of the attention kernels (internal to libmuonstep). Every argument is
// checked by the C entry points.
#pragma once

#include "common.hpp"

namespace muon {

constexpr int kAttentionRows = 128;   // queries, or keys, of a workgroup
constexpr int kAttentionFew = 64;     // sequences, one per lane

// Element (token, head, column) at data + token * token_stride + head * head_stride + column.
struct HeadsArg {
  void* data;
  int64_t token_stride, head_stride;
};

struct AttentionArgs {
  HeadsArg q, k, v, o, d_o, dq, dk, dv;
  float* lse_out;              // heads x tokens
  const float* lse;
  float *lse2, *delta;         // heads x tokens: log-sum-exp in units of log 2, rowsum(dO O)
  int64_t tokens;
  const int32_t* offsets;      // NULL: one sequence
  int4* sequence_list;         // per sequence: first token, tokens, first tile
  int4* list;                  // per tile: first token, tokens, tile; NULL: one sequence, or few
  int32_t sequences, tiles;    // tiles: of the list, or of the one sequence
  int32_t heads, kv_heads, group, dim;
  int32_t few;                 // up to kAttentionFew sequences: no list
  int32_t causal, window;      // window >= 1
  int32_t halves, parts;       // see attention_dkv_kernel
  float* partial;              // parts x (dK, dV) x tokens x kv_heads x dim, where parts > 1
  int32_t dtype;
  float scale;
};
hipError_t launch_attention_list(const AttentionArgs& a, hipStream_t s);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s);
hipError_t launch_attention_dq(const AttentionArgs& a, hipStream_t s);    // also lse2 and delta
hipError_t launch_attention_dkv(const AttentionArgs& a, hipStream_t s);   // behind it
void plan_attention_dkv(AttentionArgs& a);
hipError_t launch_attention_join(const AttentionArgs& a, hipStream_t s);   // where there are several parts

}  // namespace muon
