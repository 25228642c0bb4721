// C ABI of the 8-bit operands, their products and the mixture-of-experts operators:
// argument checks (all before the first launch) and launch arguments.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <string>
#include <vector>

#include "capi_util.hpp"
#include "fp8.hpp"
#include "plan.hpp"

using namespace muon;

extern "C" {

int muon_fp8_quantize(const muon_fp8_source_t* src, int32_t blocks, const muon_fp8_t* out, const muon_fp8_t* out_t,
                      void* stream) {
  return guarded([&]() -> int {
    if (src == nullptr) return fail(MUON_ERR_NULL, "the source is NULL");
    if (out == nullptr && out_t == nullptr) return fail(MUON_ERR_NULL, "out and out_t are both NULL");
    int st;
    const int64_t B = src->batch, R = src->out_rows, C = src->cols;
    if (src->rows < 0 || src->rows > MUON_FP8_MAX_SIDE || R < 0 || R > MUON_FP8_MAX_SIDE || C < 0 ||
        C > MUON_FP8_MAX_SIDE)
      return fail(MUON_ERR_BAD_SHAPE, "source: rows, out_rows and cols must lie in [0, MUON_FP8_MAX_SIDE]");
    if (B < 1 || B > MUON_FP8_MAX_BATCH) return fail(MUON_ERR_BAD_SHAPE, "source: batch must lie in [1, MUON_FP8_MAX_BATCH]");
    if (src->row_index != nullptr) {
      if (B != 1) return fail(MUON_ERR_BAD_SHAPE, "source: a row index takes a single matrix");
      if (src->row_div < 1) return fail(MUON_ERR_BAD_SHAPE, "source: row_div must be >= 1");
      if (misaligned(src->row_index, 4)) return fail(MUON_ERR_ALIGN, "row_index is not 4-byte aligned");
    } else {
      if (src->row_div != 1 || src->row_weight != nullptr)
        return fail(MUON_ERR_UNSUPPORTED, "source: row_div and row_weight need a row_index");
      if (R != src->rows) return fail(MUON_ERR_BAD_SHAPE, "source: out_rows must equal rows without a row_index");
    }
    if (src->row_weight != nullptr && (src->n_weights < 0 || misaligned(src->row_weight, 4)))
      return fail(src->n_weights < 0 ? MUON_ERR_BAD_SHAPE : MUON_ERR_ALIGN, "source: bad row_weight");
    // the source is read only, so its matrices may overlap
    const int esz = element_size(src->dtype);
    if (esz == 0) return fail(MUON_ERR_UNSUPPORTED, "source: dtype must be F32, BF16 or F16");
    if (src->rows > 0 && C > 0) {
      if (src->data == nullptr) return fail(MUON_ERR_NULL, "source data is NULL");
      if (misaligned(src->data, esz)) return fail(MUON_ERR_ALIGN, "source is not aligned to its element");
      if (src->ld < 0 || src->ld > kMaxPitch || src->batch_stride < 0 || src->batch_stride > kMaxBatchStride)
        return fail(MUON_ERR_BAD_SHAPE, "source: negative or too large stride");
    }
    const int32_t format = out != nullptr ? out->format : out_t->format;
    std::vector<Span> outs, ins;
    if (out != nullptr) {
      if ((st = check_operand(out, "out")) != MUON_OK) return st;
      if (out->batch != B || out->rows != R || out->cols != C) return fail(MUON_ERR_BAD_SHAPE, "out must be out_rows x cols");
      outs.push_back(span_of(out->data, data_bytes(*out), "out data"));
      outs.push_back(span_of(out->scale, scale_bytes(*out), "out scale"));
    }
    if (out_t != nullptr) {
      if ((st = check_operand(out_t, "out_t")) != MUON_OK) return st;
      if (out_t->batch != B || out_t->rows != C || out_t->cols != R)
        return fail(MUON_ERR_BAD_SHAPE, "out_t must be cols x out_rows");
      if (out_t->format != format) return fail(MUON_ERR_UNSUPPORTED, "out and out_t must have one format");
      outs.push_back(span_of(out_t->data, data_bytes(*out_t), "out_t data"));
      outs.push_back(span_of(out_t->scale, scale_bytes(*out_t), "out_t scale"));
    }
    if (R == 0 || C == 0) return MUON_OK;
    ins.push_back(span_of(src->data, strided_bytes(src->dtype, B, src->rows, C, src->ld, src->batch_stride), "source"));
    if (src->row_index) ins.push_back(span_of(src->row_index, R * 4, "row_index"));
    if (src->row_weight) ins.push_back(span_of(src->row_weight, src->n_weights * 4, "row_weight"));
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;

    QuantArgs a{};
    a.x = src->data;
    a.x_batch = src->batch_stride;
    a.ldx = src->ld;
    a.src_rows = src->rows;
    a.row_index = src->row_index;
    a.row_div = src->row_div;
    a.row_weight = src->row_weight;
    a.n_weights = src->n_weights;
    a.rows = R;
    a.cols = C;
    const int64_t rt = (R + 127) / 128, ct = (C + 127) / 128;
    if (rt * ct * B > 0x7fffffff) return fail(MUON_ERR_BAD_SHAPE, "the matrix has too many 128 x 128 tiles for a launch");
    a.row_tiles = static_cast<int32_t>(rt);
    a.col_tiles = static_cast<int32_t>(ct);
    a.total_tiles = static_cast<int32_t>(rt * ct * B);
    if (out != nullptr) {
      a.q = out->data;
      a.s = out->scale;
      a.qp = fp8_data_pitch(C);
      a.qs = fp8_scale_pitch(C);
    }
    if (out_t != nullptr) {
      a.qt = out_t->data;
      a.st = out_t->scale;
      a.tp = fp8_data_pitch(R);
      a.ts = fp8_scale_pitch(R);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("fp8_quantize", s, launch_fp8_quantize(src->dtype, format, blocks != 0, a, s));
    return MUON_OK;
  });
}

static int check_product(const muon_fp8_t* a, const muon_fp8_t* b) {
  int st;
  if (a == nullptr || b == nullptr) return fail(MUON_ERR_NULL, "a and b must not be NULL");
  if ((st = check_operand(a, "a")) != MUON_OK) return st;
  if ((st = check_operand(b, "b")) != MUON_OK) return st;
  if (a->cols != b->cols) return fail(MUON_ERR_BAD_SHAPE, "a and b must have the same number of columns");
  return MUON_OK;
}

static int check_matmul(const muon_fp8_t* a, const muon_fp8_t* b, bool grouped) {
  const int st = check_product(a, b);
  if (st != MUON_OK) return st;
  if (grouped ? a->batch != 1 : a->batch != b->batch)
    return fail(MUON_ERR_BAD_SHAPE, grouped ? "a grouped product takes one matrix a" : "a and b must have the same batch");
  return MUON_OK;
}

// The fields that every product shares.
static Fp8Gemm gemm_of(const muon_fp8_t* a, const muon_fp8_t* b, const muon_fp8_result_t* c, const int32_t* offsets) {
  Fp8Gemm g{};
  g.a = a->data;
  g.b = b->data;
  g.sa = a->scale;
  g.sb = b->scale;
  g.pitch = fp8_data_pitch(a->cols);
  g.s_pitch = fp8_scale_pitch(a->cols);
  g.a_batch = a->rows * g.pitch;
  g.b_batch = b->rows * g.pitch;
  g.sa_batch = a->rows * g.s_pitch;
  g.sb_batch = b->rows * g.s_pitch;
  g.M = a->rows;
  g.N = b->rows;
  g.kb = static_cast<int32_t>(g.pitch / MUON_FP8_BLOCK);
  g.offsets = offsets;
  g.c = c->data;
  g.c_batch = c->batch_stride;
  g.ldc = c->ld;
  g.c_dtype = c->dtype;
  g.accumulate = c->accumulate != 0;
  return g;
}

static int run_gemm(const muon_fp8_t* a, const muon_fp8_t* b, const Fp8Gemm& g, hipStream_t s) {
  const Fp8Plan p = plan_fp8_gemm(g.M, g.N, g.kb, g.mode, g.batch, g.c_dtype == MUON_DTYPE_F32);
  MUON_LAUNCH(fp8_gemm_kind(p), s, launch_fp8_gemm(a->format, b->format, p, g, s));
  return MUON_OK;
}

int muon_fp8_matmul(const muon_fp8_t* a, const muon_fp8_t* b, const int32_t* group_offsets, const muon_fp8_result_t* c,
                    void* stream) {
  return guarded([&]() -> int {
    const bool grouped = group_offsets != nullptr;
    int st = check_matmul(a, b, grouped);
    if (st != MUON_OK) return st;
    if (c == nullptr) return fail(MUON_ERR_NULL, "c is NULL");
    const int64_t mats = grouped ? 1 : b->batch;
    if ((st = check_strided("c", c->data, c->dtype, mats, a->rows, b->rows, c->ld, c->batch_stride)) != MUON_OK) return st;
    if (misaligned(group_offsets, 4)) return fail(MUON_ERR_ALIGN, "group_offsets is not 4-byte aligned");
    if (a->rows == 0 || b->rows == 0) return MUON_OK;
    std::vector<Span> outs = {span_of(c->data, strided_bytes(c->dtype, mats, a->rows, b->rows, c->ld, c->batch_stride), "c")};
    std::vector<Span> ins = {span_of(a->data, data_bytes(*a), "a data"), span_of(a->scale, scale_bytes(*a), "a scale"),
                             span_of(b->data, data_bytes(*b), "b data"), span_of(b->scale, scale_bytes(*b), "b scale")};
    if (grouped) ins.push_back(span_of(group_offsets, (b->batch + 1) * 4, "group_offsets"));
    Fp8Gemm g = gemm_of(a, b, c, group_offsets);
    g.mode = grouped ? FP8_GROUP_ROWS : FP8_DENSE;
    g.batch = static_cast<int32_t>(b->batch);
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;
    return run_gemm(a, b, g, static_cast<hipStream_t>(stream));
  });
}

int muon_fp8_matmul_grouped_k(const muon_fp8_t* a, const muon_fp8_t* b, const int32_t* group_offsets, int32_t n_groups,
                              const muon_fp8_result_t* c, void* stream) {
  return guarded([&]() -> int {
    int st = check_product(a, b);
    if (st != MUON_OK) return st;
    if (c == nullptr || group_offsets == nullptr) return fail(MUON_ERR_NULL, "c and group_offsets must not be NULL");
    if (a->batch != 1 || b->batch != 1) return fail(MUON_ERR_BAD_SHAPE, "a grouped contraction takes single matrices");
    if (n_groups < 0 || n_groups > MUON_FP8_MAX_BATCH)
      return fail(MUON_ERR_BAD_SHAPE, "n_groups must lie in [0, MUON_FP8_MAX_BATCH]");
    if ((st = check_strided("c", c->data, c->dtype, n_groups, a->rows, b->rows, c->ld, c->batch_stride)) != MUON_OK)
      return st;
    if (misaligned(group_offsets, 4)) return fail(MUON_ERR_ALIGN, "group_offsets is not 4-byte aligned");
    if (a->rows == 0 || b->rows == 0 || n_groups == 0) return MUON_OK;
    const std::vector<Span> outs = {
        span_of(c->data, strided_bytes(c->dtype, n_groups, a->rows, b->rows, c->ld, c->batch_stride), "c")};
    const std::vector<Span> ins = {
        span_of(a->data, data_bytes(*a), "a data"), span_of(a->scale, scale_bytes(*a), "a scale"),
        span_of(b->data, data_bytes(*b), "b data"), span_of(b->scale, scale_bytes(*b), "b scale"),
        span_of(group_offsets, (n_groups + 1) * 4, "group_offsets")};
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;
    Fp8Gemm g = gemm_of(a, b, c, group_offsets);
    g.mode = FP8_GROUP_K;
    g.batch = n_groups;
    return run_gemm(a, b, g, static_cast<hipStream_t>(stream));
  });
}

void muon_default_route_hyper(muon_route_hyper_t* h) {
  if (!h) return;
  *h = muon_route_hyper_t{};
  h->score = MUON_ROUTE_SOFTMAX;
  h->top_k = 1;
  h->n_groups = 1;
  h->top_groups = 1;
  h->group_top = 2;
  h->renormalize = 1;
  h->scale = 1.0f;
}

static int check_route(int64_t tokens, int32_t experts, int32_t dtype, int64_t ld, const muon_route_hyper_t* h) {
  if (h == nullptr) return fail(MUON_ERR_NULL, "hyperparameter pointer is NULL");
  if (h->score != MUON_ROUTE_SOFTMAX && h->score != MUON_ROUTE_SIGMOID)
    return fail(MUON_ERR_BAD_METHOD, "score must be SOFTMAX or SIGMOID");
  if (!std::isfinite(h->scale)) return fail(MUON_ERR_BAD_HYPER, "scale is not finite");
  if (element_size(dtype) == 0) return fail(MUON_ERR_UNSUPPORTED, "logits: dtype must be F32, BF16 or F16");
  if (experts < 1 || experts > MUON_ROUTE_MAX_EXPERTS)
    return fail(MUON_ERR_BAD_SHAPE, "experts must lie in [1, MUON_ROUTE_MAX_EXPERTS]");
  if (h->top_k < 1 || h->top_k > MUON_ROUTE_MAX_TOP_K || h->top_k > experts)
    return fail(MUON_ERR_BAD_SHAPE, "top_k must lie in [1, min(experts, MUON_ROUTE_MAX_TOP_K)]");
  if (h->n_groups < 1 || h->n_groups > MUON_ROUTE_MAX_GROUPS || experts % h->n_groups != 0)
    return fail(MUON_ERR_BAD_SHAPE, "n_groups must lie in [1, MUON_ROUTE_MAX_GROUPS] and divide experts");
  if (h->top_groups < 1 || h->top_groups > h->n_groups)
    return fail(MUON_ERR_BAD_SHAPE, "top_groups must lie in [1, n_groups]");
  if (h->group_top < 1 || h->group_top > 2) return fail(MUON_ERR_BAD_SHAPE, "group_top must be 1 or 2");
  if (tokens < 0 || tokens * h->top_k > 0x7fffffffLL || tokens > 0x7fffffffLL)
    return fail(MUON_ERR_BAD_SHAPE, "tokens * top_k must lie in [0, 2^31)");
  if (tokens > 1 && (ld < experts || ld > kMaxPitch)) return fail(MUON_ERR_BAD_SHAPE, "logits: row pitch outside [experts, 2^28]");
  return MUON_OK;
}

int muon_route(const void* logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t ld, const float* bias,
               const muon_route_hyper_t* h, int32_t* ids, float* weights, void* stream) {
  return guarded([&]() -> int {
    int st = check_route(tokens, experts, dtype, ld, h);
    if (st != MUON_OK) return st;
    if (static_cast<int64_t>(h->top_groups) * (experts / h->n_groups) < h->top_k)
      return fail(MUON_ERR_BAD_SHAPE, "top_groups hold fewer than top_k experts");
    if (tokens == 0) return MUON_OK;
    if (!logits || !ids || !weights) return fail(MUON_ERR_NULL, "logits, ids and weights must not be NULL");
    if (misaligned(logits, element_size(dtype)) || misaligned(ids, 4) || misaligned(weights, 4) || misaligned(bias, 4))
      return fail(MUON_ERR_ALIGN, "a buffer is not aligned to its element");
    std::vector<Span> ins = {span_of(logits, strided_bytes(dtype, 1, tokens, experts, ld, 0), "logits")};
    if (bias) ins.push_back(span_of(bias, experts * 4, "bias"));
    const int64_t n = tokens * h->top_k;
    if ((st = check_outputs({span_of(ids, n * 4, "ids"), span_of(weights, n * 4, "weights")}, ins)) != MUON_OK) return st;
    RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.bias = bias;
    a.experts = experts;
    a.top_k = h->top_k;
    a.n_groups = h->n_groups;
    a.top_groups = h->top_groups;
    a.group_top = h->group_top;
    a.score = h->score;
    a.renormalize = h->renormalize;
    a.scale = h->scale;
    a.ids = ids;
    a.weights = weights;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("route", s, launch_route(dtype, a, s));
    return MUON_OK;
  });
}

int muon_route_backward(const float* dweights, const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                        int64_t ld, const int32_t* ids, const muon_route_hyper_t* h, void* dlogits, int64_t ld_d,
                        void* stream) {
  return guarded([&]() -> int {
    int st = check_route(tokens, experts, dtype, ld, h);
    if (st != MUON_OK) return st;
    if (tokens == 0) return MUON_OK;
    if (!dweights || !logits || !ids || !dlogits)
      return fail(MUON_ERR_NULL, "dweights, logits, ids and dlogits must not be NULL");
    if (misaligned(logits, element_size(dtype)) || misaligned(ids, 4) || misaligned(dweights, 4))
      return fail(MUON_ERR_ALIGN, "a buffer is not aligned to its element");
    if ((st = check_strided("dlogits", dlogits, dtype, 1, tokens, experts, ld_d, 0)) != MUON_OK) return st;
    const int64_t n = tokens * h->top_k;
    if ((st = check_outputs({span_of(dlogits, strided_bytes(dtype, 1, tokens, experts, ld_d, 0), "dlogits")},
                            {span_of(logits, strided_bytes(dtype, 1, tokens, experts, ld, 0), "logits"),
                             span_of(ids, n * 4, "ids"), span_of(dweights, n * 4, "dweights")})) != MUON_OK)
      return st;
    RouteBackArgs a{};
    a.dweights = dweights;
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.ld_d = ld_d;
    a.ids = ids;
    a.experts = experts;
    a.top_k = h->top_k;
    a.score = h->score;
    a.renormalize = h->renormalize;
    a.scale = h->scale;
    a.dlogits = dlogits;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("route_backward", s, launch_route_backward(dtype, a, s));
    return MUON_OK;
  });
}

static int check_order(int64_t n, int32_t experts) {
  if (experts < 1 || experts > MUON_ROUTE_MAX_EXPERTS)
    return fail(MUON_ERR_BAD_SHAPE, "experts must lie in [1, MUON_ROUTE_MAX_EXPERTS]");
  if (n < 0 || n > 0x7fffffffLL) return fail(MUON_ERR_BAD_SHAPE, "n must lie in [0, 2^31)");
  return MUON_OK;
}

static size_t order_workspace(int64_t n, int32_t experts) {
  const int32_t b = order_blocks(n);
  return b > 1 ? static_cast<size_t>(b) * experts * 4 : 0;
}

int muon_expert_order_workspace_size(int64_t n, int32_t experts, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (bytes_out == nullptr) return fail(MUON_ERR_NULL, "bytes_out is NULL");
    const int st = check_order(n, experts);
    if (st != MUON_OK) return st;
    *bytes_out = order_workspace(n, experts);
    return MUON_OK;
  });
}

int muon_expert_order(const int32_t* ids, int64_t n, int32_t experts, int32_t align, int32_t* offsets, int32_t* counts,
                      int32_t* rows, int64_t capacity, int32_t* pos, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return guarded([&]() -> int {
    int st = check_order(n, experts);
    if (st != MUON_OK) return st;
    if (align < 1 || align > 1024) return fail(MUON_ERR_BAD_SHAPE, "align must lie in [1, 1024]");
    if (capacity < n + static_cast<int64_t>(experts) * (align - 1) || capacity > 0x7fffffffLL)
      return fail(MUON_ERR_RANGE, "capacity must lie in [n + experts * (align - 1), 2^31)");
    if (!offsets || !counts || (capacity > 0 && !rows) || (n > 0 && (!ids || !pos)))
      return fail(MUON_ERR_NULL, "ids, offsets, counts, rows and pos must not be NULL");
    if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(counts, 4) || misaligned(rows, 4) || misaligned(pos, 4))
      return fail(MUON_ERR_ALIGN, "a buffer is not 4-byte aligned");
    const size_t need = order_workspace(n, experts);
    if (need > 0 && workspace == nullptr) return fail(MUON_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
      return fail(MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
    if (need > 0 && misaligned(workspace, 4)) return fail(MUON_ERR_ALIGN, "workspace is not 4-byte aligned");
    std::vector<Span> outs = {span_of(offsets, (experts + 1) * 4, "offsets"), span_of(counts, experts * 4, "counts"),
                              span_of(rows, capacity * 4, "rows"), span_of(pos, n * 4, "pos")};
    if (need > 0) outs.push_back(span_of(workspace, static_cast<int64_t>(need), "workspace"));
    if ((st = check_outputs(outs, {span_of(ids, n * 4, "ids")})) != MUON_OK) return st;
    OrderArgs a{};
    a.ids = ids;
    a.n = n;
    a.experts = experts;
    a.align = align;
    a.offsets = offsets;
    a.counts = counts;
    a.rows = rows;
    a.pos = pos;
    a.capacity = capacity;
    a.hist = static_cast<int32_t*>(workspace);
    a.blocks = order_blocks(n);
    a.per_block = (n + a.blocks - 1) / a.blocks;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.blocks > 1) MUON_LAUNCH("order_hist", s, launch_order_hist(a, s));
    MUON_LAUNCH("order_place", s, launch_order_place(a, s));
    return MUON_OK;
  });
}

// Checks and arguments that both directions of the combination share.
static int combine_common(int32_t dtype, int64_t o_rows, int64_t cols, const int32_t* pos, const float* weights,
                          int64_t tokens, int32_t top_k, CombineArgs& a) {
  if (element_size(dtype) == 0) return fail(MUON_ERR_UNSUPPORTED, "dtype must be F32, BF16 or F16");
  if (o_rows < 0 || o_rows > 0x7fffffffLL || cols < 0 || cols > MUON_FP8_MAX_SIDE)
    return fail(MUON_ERR_BAD_SHAPE, "o_rows must lie in [0, 2^31) and cols in [0, MUON_FP8_MAX_SIDE]");
  if (top_k < 1 || top_k > MUON_ROUTE_MAX_TOP_K) return fail(MUON_ERR_BAD_SHAPE, "top_k must lie in [1, MUON_ROUTE_MAX_TOP_K]");
  if (tokens < 0 || tokens > 0x7fffffffLL || tokens * top_k > 0x7fffffffLL)
    return fail(MUON_ERR_BAD_SHAPE, "tokens * top_k must lie in [0, 2^31)");
  if (tokens > 0 && (!pos || !weights)) return fail(MUON_ERR_NULL, "pos and weights must not be NULL");
  if (misaligned(pos, 4) || misaligned(weights, 4)) return fail(MUON_ERR_ALIGN, "pos or weights is not 4-byte aligned");
  a.o_rows = o_rows;
  a.cols = cols;
  a.pos = pos;
  a.weights = weights;
  a.tokens = tokens;
  a.top_k = top_k;
  return MUON_OK;
}

int muon_combine(const void* o, int32_t dtype, int64_t o_rows, int64_t cols, int64_t ld_o, const int32_t* pos,
                 const float* weights, int64_t tokens, int32_t top_k, void* y, int64_t ld_y, void* stream) {
  return guarded([&]() -> int {
    CombineArgs a{};
    int st = combine_common(dtype, o_rows, cols, pos, weights, tokens, top_k, a);
    if (st != MUON_OK) return st;
    if ((st = check_strided("o", o, dtype, 1, o_rows, cols, ld_o, 0)) != MUON_OK) return st;
    if ((st = check_strided("y", y, dtype, 1, tokens, cols, ld_y, 0)) != MUON_OK) return st;
    if (tokens == 0 || cols == 0) return MUON_OK;
    const int64_t n = tokens * top_k;
    if ((st = check_outputs({span_of(y, strided_bytes(dtype, 1, tokens, cols, ld_y, 0), "y")},
                            {span_of(o, strided_bytes(dtype, 1, o_rows, cols, ld_o, 0), "o"), span_of(pos, n * 4, "pos"),
                             span_of(weights, n * 4, "weights")})) != MUON_OK)
      return st;
    a.o = o;
    a.ld_o = ld_o;
    a.y = y;
    a.ld_y = ld_y;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("combine", s, launch_combine(dtype, a, s));
    return MUON_OK;
  });
}

int muon_combine_backward(const void* dy, int32_t dtype, int64_t tokens, int64_t cols, int64_t ld_dy, const void* o,
                          int64_t o_rows, int64_t ld_o, const int32_t* pos, const float* weights, int32_t top_k,
                          float* dweights, void* d_o, int64_t ld_do, void* stream) {
  return guarded([&]() -> int {
    CombineArgs a{};
    int st = combine_common(dtype, o_rows, cols, pos, weights, tokens, top_k, a);
    if (st != MUON_OK) return st;
    if (dweights == nullptr && d_o == nullptr) return fail(MUON_ERR_NULL, "dweights and d_o are both NULL");
    if ((st = check_strided("dy", dy, dtype, 1, tokens, cols, ld_dy, 0)) != MUON_OK) return st;
    const int64_t n = tokens * top_k;
    std::vector<Span> outs, ins = {span_of(dy, strided_bytes(dtype, 1, tokens, cols, ld_dy, 0), "dy"),
                                   span_of(pos, n * 4, "pos"), span_of(weights, n * 4, "weights")};
    if (dweights != nullptr) {
      if (misaligned(dweights, 4)) return fail(MUON_ERR_ALIGN, "dweights is not 4-byte aligned");
      if ((st = check_strided("o", o, dtype, 1, o_rows, cols, ld_o, 0)) != MUON_OK) return st;
      ins.push_back(span_of(o, strided_bytes(dtype, 1, o_rows, cols, ld_o, 0), "o"));
      outs.push_back(span_of(dweights, n * 4, "dweights"));
    }
    if (d_o != nullptr) {
      if ((st = check_strided("d_o", d_o, dtype, 1, o_rows, cols, ld_do, 0)) != MUON_OK) return st;
      outs.push_back(span_of(d_o, strided_bytes(dtype, 1, o_rows, cols, ld_do, 0), "d_o"));
    }
    if (tokens == 0) return MUON_OK;
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.o = o;
    a.ld_o = ld_o;
    a.dweights = dweights;
    a.d_o = d_o;
    a.ld_do = ld_do;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("combine_backward", s, launch_combine_backward(dtype, a, s));
    return MUON_OK;
  });
}

}  // extern "C"
