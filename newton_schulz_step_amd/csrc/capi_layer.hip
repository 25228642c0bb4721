// C ABI of the norm, embedding, clipping and attention operators: argument checks (all before the
// first launch) and launch arguments.
#include <math.h>

#include <algorithm>
#include <string>
#include <vector>

#include "attention.hpp"
#include "capi_util.hpp"
#include "fp8.hpp"
#include "layer.hpp"
#include "plan.hpp"

namespace muon {

// A strided input, whose rows may overlap.
static int check_input(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  const std::string n(name);
  const int esz = element_size(dtype);
  if (esz == 0) return fail(MUON_ERR_UNSUPPORTED, n + ": dtype must be F32, BF16 or F16");
  if (rows == 0 || cols == 0) return MUON_OK;
  if (p == nullptr) return fail(MUON_ERR_NULL, n + " is NULL");
  if (misaligned(p, esz)) return fail(MUON_ERR_ALIGN, n + " is not aligned to its element");
  if (rows > 1 && (ld < 0 || ld > kMaxPitch)) return fail(MUON_ERR_BAD_SHAPE, n + ": row pitch outside [0, 2^28]");
  return MUON_OK;
}

static Span matrix_span(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const char* name) {
  return span_of(p, strided_bytes(dtype, 1, rows, cols, rows > 1 ? ld : cols, 0), name);
}

static int check_workspace(const void* ws, size_t bytes, size_t need, uintptr_t align) {
  if (need > 0 && ws == nullptr) return fail(MUON_ERR_NULL, "workspace is NULL");
  if (bytes < need) return fail(MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  if (need > 0 && misaligned(ws, align)) return fail(MUON_ERR_ALIGN, "workspace is not " + std::to_string(align) + "-byte aligned");
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Norm

static int check_norm_size(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > 0x7fffffffLL) return fail(MUON_ERR_BAD_SHAPE, "rows must lie in [0, 2^31)");
  if (cols < 1 || cols > MUON_NORM_MAX_COLS) return fail(MUON_ERR_BAD_SHAPE, "cols must lie in [1, MUON_NORM_MAX_COLS]");
  return MUON_OK;
}

// What both directions share; the inputs' spans go to `ins`.
static int norm_common(const muon_norm_t* n, NormArgs& a, std::vector<Span>& ins) {
  int st;
  if (n == nullptr) return fail(MUON_ERR_NULL, "the rows' description is NULL");
  if ((st = check_norm_size(n->rows, n->cols)) != MUON_OK) return st;
  if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return fail(MUON_ERR_BAD_HYPER, "eps must be finite and not negative");
  if ((st = check_input("x", n->x, n->dtype, n->rows, n->cols, n->ld_x)) != MUON_OK) return st;
  ins.push_back(matrix_span(n->x, n->dtype, n->rows, n->cols, n->ld_x, "x"));
  if (n->residual != nullptr) {
    if ((st = check_input("residual", n->residual, n->dtype, n->rows, n->cols, n->ld_residual)) != MUON_OK) return st;
    ins.push_back(matrix_span(n->residual, n->dtype, n->rows, n->cols, n->ld_residual, "residual"));
  }
  if (n->weight != nullptr) {
    if ((st = check_input("weight", n->weight, n->weight_dtype, 1, n->cols, n->cols)) != MUON_OK) return st;
    ins.push_back(matrix_span(n->weight, n->weight_dtype, 1, n->cols, n->cols, "weight"));
  }
  a.x = n->x;
  a.ld_x = n->ld_x;
  a.residual = n->residual;
  a.ld_residual = n->ld_residual;
  a.weight = n->weight;
  a.weight_dtype = n->weight_dtype;
  a.rows = n->rows;
  a.cols = n->cols;
  a.eps = n->eps;
  a.inv_cols = 1.0 / static_cast<double>(n->cols);
  return MUON_OK;
}

static size_t norm_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(norm_blocks(rows, cols)) * static_cast<size_t>(cols) * sizeof(float);
}

// ---------------------------------------------------------------------------
// Embedding

static int check_embedding(const muon_embedding_t* e) {
  if (e == nullptr) return fail(MUON_ERR_NULL, "the tokens' description is NULL");
  if (e->tokens < 0 || e->tokens > 0x7fffffffLL) return fail(MUON_ERR_BAD_SHAPE, "tokens must lie in [0, 2^31)");
  if (e->vocab < 1 || e->vocab > MUON_EMBEDDING_MAX_VOCAB)
    return fail(MUON_ERR_BAD_SHAPE, "vocab must lie in [1, MUON_EMBEDDING_MAX_VOCAB]");
  if (e->cols < 0 || e->cols > MUON_FP8_MAX_SIDE) return fail(MUON_ERR_BAD_SHAPE, "cols must lie in [0, MUON_FP8_MAX_SIDE]");
  if (e->id_bytes != 4 && e->id_bytes != 8) return fail(MUON_ERR_UNSUPPORTED, "ids must have 4 or 8 bytes");
  if (element_size(e->table_dtype) == 0) return fail(MUON_ERR_UNSUPPORTED, "table: dtype must be F32, BF16 or F16");
  if (!std::isfinite(e->scale)) return fail(MUON_ERR_BAD_HYPER, "scale is not finite");
  return MUON_OK;
}

static int check_ids(const muon_embedding_t* e) {
  if (e->tokens > 0 && e->ids == nullptr) return fail(MUON_ERR_NULL, "ids is NULL");
  if (misaligned(e->ids, e->id_bytes)) return fail(MUON_ERR_ALIGN, "ids is not aligned to its element");
  return MUON_OK;
}

static EmbeddingArgs embedding_args(const muon_embedding_t* e) {
  EmbeddingArgs a{};
  a.ids = e->ids;
  a.wide_ids = e->id_bytes == 8;
  a.tokens = e->tokens;
  a.vocab = e->vocab;
  a.cols = e->cols;
  a.scale = e->scale;
  a.table_dtype = e->table_dtype;
  a.ld_table = e->ld;
  int bits = 0;   // of the keys 0 .. vocab, the last of them for ids that are no rows
  while (bits < 31 && (e->vocab >> bits) != 0) ++bits;
  a.passes = (bits + 7) / 8;
  a.bits = (bits + a.passes - 1) / a.passes;
  a.blocks = sort_blocks(e->tokens);
  a.per_block = (e->tokens + a.blocks - 1) / a.blocks;
  a.chunk = e->tokens <= (e->cols <= 2048 ? 8192 : 4096) ? 8 : 32;
  return a;
}

// Lays the workspace out from `base`; returns its size.
static size_t embedding_workspace(EmbeddingArgs& a, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base == nullptr ? nullptr : base + at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  const size_t list = static_cast<size_t>(a.tokens) * 4;
  for (int i = 0; i < 2; ++i) {
    a.keys[i] = reinterpret_cast<int32_t*>(take(list));
    a.slots[i] = reinterpret_cast<int32_t*>(take(list));
  }
  a.hist = reinterpret_cast<int32_t*>(take(a.blocks > 1 ? static_cast<size_t>(a.blocks) * kSortBins * 4 : 0));
  a.touched = reinterpret_cast<uint8_t*>(take(static_cast<size_t>(a.vocab)));
  const size_t chunks = static_cast<size_t>((a.tokens + a.chunk - 1) / a.chunk);
  a.partial = reinterpret_cast<float*>(take(2 * chunks * static_cast<size_t>(a.cols) * 4));
  return at;
}

// ---------------------------------------------------------------------------
// Clipping

// Elements of a workgroup: as many as leave 2048 workgroups or more, 8192 to 65536.
static int32_t clip_chunk(int64_t elements) {
  int32_t chunk = 65536;
  while (chunk > 8192 && elements / chunk < 2048) chunk /= 2;
  return chunk;
}

static int check_tensors(const muon_tensor_t* t, int32_t n, const char* name, int64_t& elements) {
  const std::string s(name);
  if (n < 0 || n > MUON_CLIP_MAX_TENSORS) return fail(MUON_ERR_BAD_SHAPE, "n must lie in [0, MUON_CLIP_MAX_TENSORS]");
  if (n > 0 && t == nullptr) return fail(MUON_ERR_NULL, s + " is NULL");
  elements = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int esz = element_size(t[i].dtype);
    if (esz == 0) return fail(MUON_ERR_UNSUPPORTED, s + "[" + std::to_string(i) + "]: dtype must be F32, BF16 or F16");
    if (t[i].numel < 0 || t[i].numel > MUON_MAX_TABLE_ELEMENTS || (elements += t[i].numel) > MUON_MAX_TABLE_ELEMENTS)
      return fail(MUON_ERR_BAD_SHAPE, s + ": more than MUON_MAX_TABLE_ELEMENTS elements, or a negative number");
    if (t[i].numel == 0) continue;
    if (t[i].data == nullptr) return fail(MUON_ERR_NULL, s + "[" + std::to_string(i) + "] is NULL");
    if (misaligned(t[i].data, esz))
      return fail(MUON_ERR_ALIGN, s + "[" + std::to_string(i) + "] is not aligned to its element");
  }
  return MUON_OK;
}

static int64_t clip_blocks(const muon_tensor_t* t, int32_t n, int32_t chunk) {
  int64_t b = 0;
  for (int32_t i = 0; i < n; ++i) b += (t[i].numel + chunk - 1) / chunk;
  return b;
}

// Calls f with the arguments of one launch after the other: up to kClipTensors tensors each.
template <typename F>
static int each_clip_launch(const muon_tensor_t* in, const muon_tensor_t* out, int32_t n, int32_t chunk, F&& f) {
  ClipArgs a{};
  a.chunk = chunk;
  int64_t before = 0;   // workgroups of earlier launches
  for (int32_t i = 0; i < n;) {
    int64_t blocks = 0;
    a.n = 0;
    for (; i < n && a.n < kClipTensors; ++i) {
      if (in[i].numel == 0) continue;
      ClipTensor& t = a.t[a.n++];
      t.in = in[i].data;
      t.out = out[i].data;
      t.n = in[i].numel;
      t.first = static_cast<int32_t>(blocks);
      t.in_dtype = static_cast<int16_t>(in[i].dtype);
      t.out_dtype = static_cast<int16_t>(out[i].dtype);
      blocks += (in[i].numel + chunk - 1) / chunk;
    }
    a.blocks = static_cast<int32_t>(blocks);   // at most 2^36 / 8192 and one per tensor
    if (a.n == 0) continue;
    const int st = f(a, before);
    if (st != MUON_OK) return st;
    before += blocks;
  }
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Attention

static int check_attention(const muon_attention_t* a) {
  if (a == nullptr) return fail(MUON_ERR_NULL, "the attention's description is NULL");
  if (a->tokens < 0 || a->tokens > MUON_ATTENTION_MAX_TOKENS)
    return fail(MUON_ERR_BAD_SHAPE, "tokens must lie in [0, MUON_ATTENTION_MAX_TOKENS]");
  if (a->offsets != nullptr && (a->sequences < 0 || a->sequences > MUON_ATTENTION_MAX_TOKENS))
    return fail(MUON_ERR_BAD_SHAPE, "sequences must lie in [0, MUON_ATTENTION_MAX_TOKENS]");
  if (a->heads < 1 || a->heads > MUON_ATTENTION_MAX_HEADS || a->kv_heads < 1 || a->heads % a->kv_heads != 0)
    return fail(MUON_ERR_BAD_SHAPE, "heads must lie in [1, MUON_ATTENTION_MAX_HEADS] and be a multiple of kv_heads");
  if (a->dim < 8 || a->dim > MUON_ATTENTION_MAX_DIM || a->dim % 8 != 0)
    return fail(MUON_ERR_BAD_SHAPE, "dim must be a multiple of 8 in [8, MUON_ATTENTION_MAX_DIM]");
  if (a->dtype != MUON_DTYPE_BF16 && a->dtype != MUON_DTYPE_F16) return fail(MUON_ERR_UNSUPPORTED, "attention: dtype must be BF16 or F16");
  if (a->window < 0) return fail(MUON_ERR_BAD_SHAPE, "window must not be negative");
  if (a->window > 0 && !a->causal) return fail(MUON_ERR_UNSUPPORTED, "a window needs causal");
  if (!(a->scale > 0.0f) || !(a->scale <= MUON_ATTENTION_MAX_SCALE))
    return fail(MUON_ERR_BAD_HYPER, "scale must lie in (0, MUON_ATTENTION_MAX_SCALE]");
  if (misaligned(a->offsets, 4)) return fail(MUON_ERR_ALIGN, "offsets is not 4-byte aligned");
  return MUON_OK;
}

// The heads of one operand as they lie in memory.
struct HeadsSpan {
  const muon_heads_t* t;
  int64_t tokens, heads, dim;
  const char* name;
  // columns between the first and the last of a token
  int64_t width() const { return (heads - 1) * t->head_stride + dim; }
  const char* lo() const { return static_cast<const char*>(t->data); }
  const char* hi() const { return lo() + ((tokens - 1) * t->token_stride + width()) * 2; }
};

static bool heads_meet(const HeadsSpan& a, const HeadsSpan& b) {
  if (!(a.lo() < b.hi() && b.lo() < a.hi())) return false;
  // parts of the same rows, such as those of a joint projection: of a token's, or of each head's
  const int64_t pitch = a.t->token_stride, head = a.t->head_stride, by = (b.lo() - a.lo()) / 2;
  const bool one = a.tokens == 1;   // whose pitch does not matter
  if ((!one && b.t->token_stride != pitch) || (b.lo() - a.lo()) % 2 != 0) return true;
  auto apart = [&](int64_t wa, int64_t wb, int64_t every) {   // runs of wa and of wb elements, each once in `every`
    const int64_t d = (by % every + every) % every;
    return wa <= every && wb <= every && d >= wa && d + wb <= every;
  };
  if (!one && apart(a.width(), b.width(), pitch)) return false;
  return !(a.heads > 1 && b.heads > 1 && b.t->head_stride == head && head > 0 && (one || pitch % head == 0) &&
           apart(a.dim, b.dim, head));
}

static int check_heads(const HeadsSpan& x, bool output) {
  const std::string n(x.name);
  const muon_heads_t* t = x.t;
  if (t == nullptr) return fail(MUON_ERR_NULL, n + " is NULL");
  if (x.tokens == 0) return MUON_OK;
  if (t->data == nullptr) return fail(MUON_ERR_NULL, n + ": data is NULL");
  if (misaligned(t->data, 16) || t->token_stride % 8 != 0 || t->head_stride % 8 != 0)
    return fail(MUON_ERR_ALIGN, n + ": data must be 16-byte aligned and strides multiples of 8");
  if (t->token_stride < x.dim || t->token_stride > (1 << 22))
    return fail(MUON_ERR_BAD_SHAPE, n + ": token stride outside [dim, 2^22]");
  if (t->head_stride < 0 || t->head_stride > (int64_t(1) << 40)) return fail(MUON_ERR_BAD_SHAPE, n + ": head stride outside [0, 2^40]");
  if (output && x.heads > 1) {   // rows of tokens, each with all heads, or of heads, each with all tokens
    const bool by_token = t->head_stride >= x.dim && t->token_stride >= x.width();
    const bool by_head = t->head_stride >= (x.tokens - 1) * t->token_stride + x.dim;
    if (!by_token && !by_head) return fail(MUON_ERR_BAD_SHAPE, n + ": heads and tokens overlap");
  }
  return MUON_OK;
}

// No output may meet another operand, nor a flat buffer.
static int check_heads_apart(const std::vector<HeadsSpan>& outs, const std::vector<HeadsSpan>& ins, const std::vector<Span>& flat_outs,
                             const std::vector<Span>& flat_ins) {
  auto both = [](const char* x, const char* y) { return fail(MUON_ERR_OVERLAP, std::string("buffers overlap: ") + x + " and " + y); };
  auto hits = [](const HeadsSpan& x, const Span& s) { return s.lo < s.hi && x.lo() < s.hi && s.lo < x.hi(); };
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (heads_meet(outs[i], outs[j])) return both(outs[i].name, outs[j].name);
    for (const HeadsSpan& x : ins)
      if (heads_meet(outs[i], x)) return both(outs[i].name, x.name);
    for (const Span& s : flat_ins)
      if (hits(outs[i], s)) return both(outs[i].name, s.name);
  }
  for (const Span& s : flat_outs) {
    for (const HeadsSpan& x : outs)
      if (hits(x, s)) return both(x.name, s.name);
    for (const HeadsSpan& x : ins)
      if (hits(x, s)) return both(x.name, s.name);
  }
  return check_outputs(flat_outs, flat_ins);
}

static HeadsArg heads_arg(const muon_heads_t* t) { return {t->data, t->token_stride, t->head_stride}; }

static AttentionArgs attention_args(const muon_attention_t* m) {
  AttentionArgs a{};
  a.tokens = m->tokens;
  a.offsets = m->offsets;
  a.sequences = m->offsets != nullptr ? m->sequences : 1;
  // as many tiles as any sequences of so many tokens can have
  const int64_t tiles = m->offsets != nullptr ? m->tokens / kAttentionRows + std::min<int64_t>(m->sequences, m->tokens)
                                              : (m->tokens + kAttentionRows - 1) / kAttentionRows;
  a.tiles = static_cast<int32_t>(tiles);
  a.few = m->offsets != nullptr && m->sequences <= kAttentionFew;
  a.heads = m->heads;
  a.kv_heads = m->kv_heads;
  a.group = m->heads / m->kv_heads;
  a.dim = m->dim;
  a.causal = m->causal != 0;
  a.window = m->window > 0 ? std::min(m->window, 1 << 30) : 1 << 30;
  a.dtype = m->dtype;
  a.scale = m->scale;
  return a;
}

// Lays the workspace out from `base`; returns its size.
static size_t attention_workspace(AttentionArgs& a, bool backward, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base == nullptr ? nullptr : base + at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  if (a.offsets != nullptr && !a.few) {
    a.sequence_list = reinterpret_cast<int4*>(take(static_cast<size_t>(a.sequences) * sizeof(int4)));
    a.list = reinterpret_cast<int4*>(take(static_cast<size_t>(a.tiles) * sizeof(int4)));
  }
  if (backward) {
    const size_t rows = static_cast<size_t>(a.tokens) * static_cast<size_t>(a.heads) * sizeof(float);
    a.lse2 = reinterpret_cast<float*>(take(rows));
    a.delta = reinterpret_cast<float*>(take(rows));
    plan_attention_dkv(a);
    if (a.parts > 1)
      a.partial = reinterpret_cast<float*>(take(static_cast<size_t>(a.parts) * 2 * static_cast<size_t>(a.tokens) *
                                                static_cast<size_t>(a.kv_heads) * static_cast<size_t>(a.dim) * sizeof(float)));
  }
  return at;
}

}  // namespace muon

using namespace muon;

extern "C" {

int muon_rms_norm(const muon_norm_t* n, void* sum, int64_t ld_sum, void* y, int64_t ld_y, const muon_fp8_t* q,
                  float* rstd, void* stream) {
  return guarded([&]() -> int {
    NormArgs a{};
    std::vector<Span> ins, outs;
    int st = norm_common(n, a, ins);
    if (st != MUON_OK) return st;
    if (sum == nullptr && y == nullptr && q == nullptr && rstd == nullptr) return fail(MUON_ERR_NULL, "no output is wanted");
    const int64_t R = n->rows, C = n->cols;
    if (sum != nullptr) {
      if ((st = check_strided("sum", sum, n->dtype, 1, R, C, ld_sum, 0)) != MUON_OK) return st;
      outs.push_back(matrix_span(sum, n->dtype, R, C, ld_sum, "sum"));
    }
    if (y != nullptr) {
      if ((st = check_strided("y", y, n->dtype, 1, R, C, ld_y, 0)) != MUON_OK) return st;
      outs.push_back(matrix_span(y, n->dtype, R, C, ld_y, "y"));
    }
    if (q != nullptr) {
      if ((st = check_operand(q, "q")) != MUON_OK) return st;
      if (q->batch != 1 || q->rows != R || q->cols != C) return fail(MUON_ERR_BAD_SHAPE, "q must be rows x cols, batch 1");
      outs.push_back(span_of(q->data, data_bytes(*q), "q data"));
      outs.push_back(span_of(q->scale, scale_bytes(*q), "q scale"));
      a.q = q->data;
      a.s = q->scale;
      a.qp = fp8_data_pitch(C);
      a.qs = fp8_scale_pitch(C);
      a.format = q->format;
    }
    if (rstd != nullptr) {
      if (misaligned(rstd, 4)) return fail(MUON_ERR_ALIGN, "rstd is not 4-byte aligned");
      outs.push_back(span_of(rstd, R * 4, "rstd"));
    }
    if (R == 0) return MUON_OK;
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;
    a.sum = sum;
    a.ld_sum = ld_sum;
    a.y = y;
    a.ld_y = ld_y;
    a.rstd = rstd;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("rms_norm", s, launch_rms_norm(n->dtype, a, s));
    return MUON_OK;
  });
}

int muon_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (bytes_out == nullptr) return fail(MUON_ERR_NULL, "bytes_out is NULL");
    const int st = check_norm_size(rows, cols);
    if (st != MUON_OK) return st;
    *bytes_out = norm_workspace(rows, cols);
    return MUON_OK;
  });
}

int muon_rms_norm_backward(const muon_norm_t* n, const float* rstd, const void* dy, int64_t ld_dy, const void* dsum,
                           int64_t ld_dsum, void* dx, int64_t ld_dx, void* dweight, int32_t dweight_dtype,
                           int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    NormArgs a{};
    std::vector<Span> ins, outs;
    int st = norm_common(n, a, ins);
    if (st != MUON_OK) return st;
    if (n->residual != nullptr) return fail(MUON_ERR_UNSUPPORTED, "the gradient takes the rows that were normed, without a residual");
    if (dx == nullptr && dweight == nullptr) return fail(MUON_ERR_NULL, "dx and dweight are both NULL");
    const int64_t R = n->rows, C = n->cols;
    if (R > 0 && rstd == nullptr) return fail(MUON_ERR_NULL, "rstd is NULL");
    if (misaligned(rstd, 4)) return fail(MUON_ERR_ALIGN, "rstd is not 4-byte aligned");
    if ((st = check_input("dy", dy, n->dtype, R, C, ld_dy)) != MUON_OK) return st;
    ins.push_back(span_of(rstd, R * 4, "rstd"));
    ins.push_back(matrix_span(dy, n->dtype, R, C, ld_dy, "dy"));
    if (dsum != nullptr) {
      if ((st = check_input("dsum", dsum, n->dtype, R, C, ld_dsum)) != MUON_OK) return st;
      ins.push_back(matrix_span(dsum, n->dtype, R, C, ld_dsum, "dsum"));
    }
    if (dx != nullptr) {
      if ((st = check_strided("dx", dx, n->dtype, 1, R, C, ld_dx, 0)) != MUON_OK) return st;
      outs.push_back(matrix_span(dx, n->dtype, R, C, ld_dx, "dx"));
    }
    if (dweight != nullptr) {
      if ((st = check_strided("dweight", dweight, dweight_dtype, 1, 1, C, C, 0)) != MUON_OK) return st;
      outs.push_back(matrix_span(dweight, dweight_dtype, 1, C, C, "dweight"));
      const size_t need = norm_workspace(R, C);
      if ((st = check_workspace(workspace, workspace_bytes, need, 4)) != MUON_OK) return st;
      outs.push_back(span_of(workspace, static_cast<int64_t>(need), "workspace"));
      a.partial = static_cast<float*>(workspace);
    }
    if ((st = check_outputs(outs, ins)) != MUON_OK) return st;
    a.rstd_in = rstd;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.dsum = dsum;
    a.ld_dsum = ld_dsum;
    a.dx = dx;
    a.ld_dx = ld_dx;
    a.dweight = dweight;
    a.dweight_dtype = dweight_dtype;
    a.accumulate = accumulate != 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // without rows the weight's gradient is still zero
    if (R > 0 || dweight != nullptr) MUON_LAUNCH("rms_norm_backward", s, launch_rms_norm_backward(n->dtype, a, s));
    if (dweight != nullptr) MUON_LAUNCH("norm_weight", s, launch_norm_weight(a, s));
    return MUON_OK;
  });
}

int muon_embedding(const muon_embedding_t* e, const void* table, void* y, int32_t dtype, int64_t ld_y, void* stream) {
  return guarded([&]() -> int {
    int st = check_embedding(e);
    if (st != MUON_OK) return st;
    if ((st = check_ids(e)) != MUON_OK) return st;
    if ((st = check_input("table", table, e->table_dtype, e->vocab, e->cols, e->ld)) != MUON_OK) return st;
    if ((st = check_strided("y", y, dtype, 1, e->tokens, e->cols, ld_y, 0)) != MUON_OK) return st;
    if (e->tokens == 0 || e->cols == 0) return MUON_OK;
    if ((st = check_outputs({matrix_span(y, dtype, e->tokens, e->cols, ld_y, "y")},
                            {matrix_span(table, e->table_dtype, e->vocab, e->cols, e->ld, "table"),
                             span_of(e->ids, e->tokens * e->id_bytes, "ids")})) != MUON_OK)
      return st;
    if (e->tokens * ((e->cols + 2047) / 2048) > 0x7fffffffLL)
      return fail(MUON_ERR_BAD_SHAPE, "too many tokens and columns for a launch");
    EmbeddingArgs a = embedding_args(e);
    a.table = table;
    a.y = y;
    a.ld_y = ld_y;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_LAUNCH("embedding", s, launch_embedding(dtype, a, s));
    return MUON_OK;
  });
}

int muon_embedding_backward_workspace_size(const muon_embedding_t* e, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (bytes_out == nullptr) return fail(MUON_ERR_NULL, "bytes_out is NULL");
    const int st = check_embedding(e);
    if (st != MUON_OK) return st;
    EmbeddingArgs a = embedding_args(e);
    *bytes_out = embedding_workspace(a, nullptr);
    return MUON_OK;
  });
}

int muon_embedding_backward(const muon_embedding_t* e, const void* dy, int32_t dtype, int64_t ld_dy, void* dtable,
                            int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int st = check_embedding(e);
    if (st != MUON_OK) return st;
    if ((st = check_ids(e)) != MUON_OK) return st;
    if ((st = check_input("dy", dy, dtype, e->tokens, e->cols, ld_dy)) != MUON_OK) return st;
    if ((st = check_strided("dtable", dtable, e->table_dtype, 1, e->vocab, e->cols, e->ld, 0)) != MUON_OK) return st;
    EmbeddingArgs a = embedding_args(e);
    const size_t need = embedding_workspace(a, nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, need, 16)) != MUON_OK) return st;
    if (e->cols == 0 || (e->tokens == 0 && accumulate)) return MUON_OK;
    if ((st = check_outputs({matrix_span(dtable, e->table_dtype, e->vocab, e->cols, e->ld, "dtable"),
                             span_of(workspace, static_cast<int64_t>(need), "workspace")},
                            {matrix_span(dy, dtype, e->tokens, e->cols, ld_dy, "dy"),
                             span_of(e->ids, e->tokens * e->id_bytes, "ids")})) != MUON_OK)
      return st;
    const int64_t chunks = (e->tokens + a.chunk - 1) / a.chunk;
    if (chunks * ((e->cols + 511) / 512) + e->vocab > 0x7fffffffLL)
      return fail(MUON_ERR_BAD_SHAPE, "too many tokens and columns for a launch");
    embedding_workspace(a, static_cast<char*>(workspace));
    if (accumulate) a.touched = nullptr;
    a.accumulate = accumulate != 0;
    a.dy = dy;
    a.ld_y = ld_dy;
    a.dtable = dtable;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.blocks == 1) {
      MUON_LAUNCH("sort_all", s, launch_sort_all(a, s));
    } else {
      for (int p = 0; p < a.passes; ++p) {
        MUON_LAUNCH("sort_hist", s, launch_sort_hist(a, p, s));
        MUON_LAUNCH("sort_place", s, launch_sort_place(a, p, s));
      }
    }
    MUON_LAUNCH("embedding_sum", s, launch_embedding_sum(dtype, a, s));
    MUON_LAUNCH("embedding_join", s, launch_embedding_join(a, s));
    return MUON_OK;
  });
}

int muon_grad_sumsq_workspace_size(const muon_tensor_t* grads, int32_t n, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (bytes_out == nullptr) return fail(MUON_ERR_NULL, "bytes_out is NULL");
    int64_t elements;
    const int st = check_tensors(grads, n, "grads", elements);
    if (st != MUON_OK) return st;
    *bytes_out = static_cast<size_t>(clip_blocks(grads, n, clip_chunk(elements))) * sizeof(double);
    return MUON_OK;
  });
}

int muon_grad_sumsq(const muon_tensor_t* grads, int32_t n, int32_t accumulate, double* sumsq, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int64_t elements;
    int st = check_tensors(grads, n, "grads", elements);
    if (st != MUON_OK) return st;
    if (sumsq == nullptr) return fail(MUON_ERR_NULL, "sumsq is NULL");
    if (misaligned(sumsq, 8)) return fail(MUON_ERR_ALIGN, "sumsq is not 8-byte aligned");
    const int32_t chunk = clip_chunk(elements);
    const int64_t blocks = clip_blocks(grads, n, chunk);
    const size_t need = static_cast<size_t>(blocks) * sizeof(double);
    if ((st = check_workspace(workspace, workspace_bytes, need, 8)) != MUON_OK) return st;
    std::vector<Span> ins;
    for (int32_t i = 0; i < n; ++i) ins.push_back(span_of(grads[i].data, grads[i].numel * element_size(grads[i].dtype), "a gradient"));
    if ((st = check_outputs({span_of(sumsq, 8, "sumsq"), span_of(workspace, static_cast<int64_t>(need), "workspace")}, ins)) != MUON_OK)
      return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    st = each_clip_launch(grads, grads, n, chunk, [&](ClipArgs& a, int64_t before) -> int {
      a.partial = static_cast<double*>(workspace) + before;
      MUON_LAUNCH("grad_sumsq", s, launch_grad_sumsq(a, s));
      return MUON_OK;
    });
    if (st != MUON_OK) return st;
    MUON_LAUNCH("sum_partials", s, launch_sum_partials(static_cast<const double*>(workspace), blocks, accumulate != 0, sumsq, s));
    return MUON_OK;
  });
}

int muon_grad_clip(const muon_tensor_t* grads, const muon_tensor_t* outs, int32_t n, const double* sumsq,
                   float max_norm, float* norm, void* stream) {
  return guarded([&]() -> int {
    int64_t elements, other;
    int st = check_tensors(grads, n, "grads", elements);
    if (st != MUON_OK) return st;
    if (outs == nullptr) outs = grads;
    if (outs != grads && (st = check_tensors(outs, n, "outs", other)) != MUON_OK) return st;
    if (!(max_norm >= 0.0f)) return fail(MUON_ERR_BAD_HYPER, "max_norm must not be negative or NaN");
    if (sumsq == nullptr) return fail(MUON_ERR_NULL, "sumsq is NULL");
    if (misaligned(sumsq, 8) || misaligned(norm, 4)) return fail(MUON_ERR_ALIGN, "sumsq or norm is not aligned to its element");
    // outputs may be their own inputs and nothing else: sorted by address, nobody begins
    // before an output in front of it ends, and no output before anybody in front of it does
    struct Part {
      const char *lo, *hi;
      bool out;
    };
    std::vector<Part> parts;
    parts.reserve(2 * static_cast<size_t>(n) + 2);
    auto add = [&](const void* p, int64_t bytes, bool out) {
      if (bytes > 0) parts.push_back({static_cast<const char*>(p), static_cast<const char*>(p) + bytes, out});
    };
    for (int32_t i = 0; i < n; ++i) {
      if (outs[i].numel != grads[i].numel) return fail(MUON_ERR_BAD_SHAPE, "outs[" + std::to_string(i) + "] has another number of elements");
      add(outs[i].data, outs[i].numel * element_size(outs[i].dtype), true);
      if (outs[i].data != grads[i].data || outs[i].dtype != grads[i].dtype)
        add(grads[i].data, grads[i].numel * element_size(grads[i].dtype), false);
    }
    add(sumsq, 8, false);
    if (norm != nullptr) add(norm, 4, true);
    std::sort(parts.begin(), parts.end(), [](const Part& x, const Part& y) { return x.lo < y.lo; });
    const char *end = nullptr, *end_out = nullptr;
    for (const Part& p : parts) {
      if (p.lo < (p.out ? end : end_out)) return fail(MUON_ERR_OVERLAP, "an output overlaps another buffer");
      end = std::max(end, p.hi);
      if (p.out) end_out = std::max(end_out, p.hi);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    bool told = false;   // the first launch writes the norm
    auto launch = [&](ClipArgs& a, int64_t) -> int {
      a.sumsq = sumsq;
      a.max_norm = max_norm;
      a.norm = told ? nullptr : norm;
      MUON_LAUNCH("grad_clip", s, launch_grad_clip(a, s));
      told = true;
      return MUON_OK;
    };
    if ((st = each_clip_launch(grads, outs, n, clip_chunk(elements), launch)) != MUON_OK) return st;
    if (!told && norm != nullptr) {   // no elements at all
      ClipArgs a{};
      return launch(a, 0);
    }
    return MUON_OK;
  });
}

int muon_attention_workspace_size(const muon_attention_t* m, int32_t backward, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (bytes_out == nullptr) return fail(MUON_ERR_NULL, "bytes_out is NULL");
    const int st = check_attention(m);
    if (st != MUON_OK) return st;
    AttentionArgs a = attention_args(m);
    *bytes_out = attention_workspace(a, backward != 0, nullptr);
    return MUON_OK;
  });
}

int muon_attention(const muon_attention_t* m, const muon_heads_t* q, const muon_heads_t* k, const muon_heads_t* v,
                   const muon_heads_t* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int st = check_attention(m);
    if (st != MUON_OK) return st;
    const int64_t T = m->tokens;
    const HeadsSpan sq{q, T, m->heads, m->dim, "q"}, sk{k, T, m->kv_heads, m->dim, "k"}, sv{v, T, m->kv_heads, m->dim, "v"},
        so{o, T, m->heads, m->dim, "o"};
    for (const HeadsSpan* x : {&sq, &sk, &sv})
      if ((st = check_heads(*x, false)) != MUON_OK) return st;
    if ((st = check_heads(so, true)) != MUON_OK) return st;
    if (misaligned(lse, 4)) return fail(MUON_ERR_ALIGN, "lse is not 4-byte aligned");
    AttentionArgs a = attention_args(m);
    const size_t need = attention_workspace(a, false, nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, need, 16)) != MUON_OK) return st;
    if (T == 0 || a.sequences == 0) return MUON_OK;
    std::vector<Span> outs, ins;
    if (lse != nullptr) outs.push_back(span_of(lse, T * m->heads * 4, "lse"));
    if (need > 0) outs.push_back(span_of(workspace, static_cast<int64_t>(need), "workspace"));
    if (m->offsets != nullptr) ins.push_back(span_of(m->offsets, (static_cast<int64_t>(m->sequences) + 1) * 4, "offsets"));
    if ((st = check_heads_apart({so}, {sq, sk, sv}, outs, ins)) != MUON_OK) return st;
    if (static_cast<int64_t>(a.tiles) * a.heads > 0x7fffffffLL) return fail(MUON_ERR_BAD_SHAPE, "too many tokens and heads for a launch");
    attention_workspace(a, false, static_cast<char*>(workspace));
    a.q = heads_arg(q);
    a.k = heads_arg(k);
    a.v = heads_arg(v);
    a.o = heads_arg(o);
    a.lse_out = lse;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.list != nullptr) MUON_LAUNCH("attention_list", s, launch_attention_list(a, s));
    MUON_LAUNCH("attention", s, launch_attention(a, s));
    return MUON_OK;
  });
}

int muon_attention_backward(const muon_attention_t* m, const muon_heads_t* d_o, const muon_heads_t* q,
                            const muon_heads_t* k, const muon_heads_t* v, const muon_heads_t* o, const float* lse,
                            const muon_heads_t* dq, const muon_heads_t* dk, const muon_heads_t* dv, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int st = check_attention(m);
    if (st != MUON_OK) return st;
    const int64_t T = m->tokens;
    const int32_t H = m->heads, K = m->kv_heads, D = m->dim;
    const std::vector<HeadsSpan> ins = {{d_o, T, H, D, "d_o"}, {q, T, H, D, "q"}, {k, T, K, D, "k"}, {v, T, K, D, "v"}, {o, T, H, D, "o"}};
    const std::vector<HeadsSpan> outs = {{dq, T, H, D, "dq"}, {dk, T, K, D, "dk"}, {dv, T, K, D, "dv"}};
    for (const HeadsSpan& x : ins)
      if ((st = check_heads(x, false)) != MUON_OK) return st;
    for (const HeadsSpan& x : outs)
      if ((st = check_heads(x, true)) != MUON_OK) return st;
    if (T > 0 && lse == nullptr) return fail(MUON_ERR_NULL, "lse is NULL");
    if (misaligned(lse, 4)) return fail(MUON_ERR_ALIGN, "lse is not 4-byte aligned");
    AttentionArgs a = attention_args(m);
    const size_t need = attention_workspace(a, true, nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, need, 16)) != MUON_OK) return st;
    if (T == 0 || a.sequences == 0) return MUON_OK;
    std::vector<Span> flat = {span_of(lse, T * H * 4, "lse")};
    if (m->offsets != nullptr) flat.push_back(span_of(m->offsets, (static_cast<int64_t>(m->sequences) + 1) * 4, "offsets"));
    if ((st = check_heads_apart(outs, ins, {span_of(workspace, static_cast<int64_t>(need), "workspace")}, flat)) != MUON_OK) return st;
    if (static_cast<int64_t>(a.tiles) * H > 0x7fffffffLL || T * H > (int64_t(1) << 36) || T * K * D > (int64_t(1) << 38))
      return fail(MUON_ERR_BAD_SHAPE, "too many tokens and heads for a launch");
    attention_workspace(a, true, static_cast<char*>(workspace));
    a.q = heads_arg(q);
    a.k = heads_arg(k);
    a.v = heads_arg(v);
    a.o = heads_arg(o);
    a.d_o = heads_arg(d_o);
    a.dq = heads_arg(dq);
    a.dk = heads_arg(dk);
    a.dv = heads_arg(dv);
    a.lse = lse;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.list != nullptr) MUON_LAUNCH("attention_list", s, launch_attention_list(a, s));
    MUON_LAUNCH("attention_dq", s, launch_attention_dq(a, s));
    MUON_LAUNCH("attention_dkv", s, launch_attention_dkv(a, s));
    if (a.parts > 1) MUON_LAUNCH("attention_join", s, launch_attention_join(a, s));
    return MUON_OK;
  });
}

}  // extern "C"
