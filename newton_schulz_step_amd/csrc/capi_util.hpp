// Helpers shared by the C entry points: the thread's error message, argument
// checks and timed launches.
#pragma once

#include <exception>
#include <string>
#include <vector>

#include "common.hpp"
#include "fp8.hpp"
#include "plan.hpp"

namespace muon {

// Records the calling thread's error message and returns `code`.
int fail(int code, const std::string& msg);
void clear_error();

// Measurement hooks: launches are bracketed with events while profiling is on.
bool prof_active();
hipError_t prof_open(hipStream_t s, hipEvent_t* a, hipEvent_t* b);
void prof_close(const char* kind, hipStream_t s, hipEvent_t a, hipEvent_t b);

template <typename F>
hipError_t timed(const char* kind, hipStream_t s, F&& launch) {
  if (!prof_active()) return launch();
  hipEvent_t a = nullptr, b = nullptr;
  hipError_t r = prof_open(s, &a, &b);
  if (r != hipSuccess) return r;
  r = launch();
  prof_close(kind, s, a, b);
  return r;
}

#define MUON_LAUNCH(kind, stream, expr)                                                        \
  do {                                                                                         \
    const hipError_t _e = timed(kind, stream, [&]() { return (expr); });                      \
    if (_e != hipSuccess)                                                                      \
      return fail(MUON_ERR_HIP, std::string(kind) + " launch failed: " + hipGetErrorString(_e)); \
  } while (0)

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

struct Span {
  const char* lo;
  const char* hi;
  const char* name;
};

inline bool overlapping(const std::vector<Span>& v, std::string& which) {
  for (size_t i = 0; i < v.size(); ++i)
    for (size_t j = i + 1; j < v.size(); ++j)
      if (v[i].lo < v[j].hi && v[j].lo < v[i].hi) {
        which = std::string(v[i].name) + " and " + v[j].name;
        return true;
      }
  return false;
}

// Runs an entry point's body; nothing may throw through the C ABI.
template <typename F>
int guarded(F&& f) noexcept {
  try {
    clear_error();
    return f();
  } catch (...) {   // only host memory can run out here
    clear_error();
    return MUON_ERR_HIP;
  }
}

// Strides beyond these are refused, so that no byte count below overflows.
constexpr int64_t kMaxPitch = int64_t(1) << 28;
constexpr int64_t kMaxBatchStride = int64_t(1) << 48;

inline Span span_of(const void* p, int64_t bytes, const char* name) {
  return {static_cast<const char*>(p), static_cast<const char*>(p) + bytes, name};
}

// No output may overlap another buffer; inputs may share memory with each other.
inline int check_outputs(const std::vector<Span>& outs, const std::vector<Span>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    const Span& a = outs[i];
    auto hits = [&](const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; };
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (hits(outs[j])) return fail(MUON_ERR_OVERLAP, std::string("buffers overlap: ") + a.name + " and " + outs[j].name);
    for (const Span& b : ins)
      if (hits(b)) return fail(MUON_ERR_OVERLAP, std::string("buffers overlap: ") + a.name + " and " + b.name);
  }
  return MUON_OK;
}

// A strided result of `batch` rows x cols matrices that must not overlap each other.
inline int check_strided(const char* name, const void* p, int32_t dtype, int64_t batch, int64_t rows, int64_t cols,
                         int64_t ld, int64_t batch_stride) {
  const std::string n(name);
  const int esz = element_size(dtype);
  if (esz == 0) return fail(MUON_ERR_UNSUPPORTED, n + ": dtype must be F32, BF16 or F16");
  if (rows == 0 || cols == 0 || batch == 0) return MUON_OK;
  if (p == nullptr) return fail(MUON_ERR_NULL, n + " is NULL");
  if (misaligned(p, esz)) return fail(MUON_ERR_ALIGN, n + " is not aligned to its element");
  if (rows > 1 && (ld < cols || ld > kMaxPitch)) return fail(MUON_ERR_BAD_SHAPE, n + ": row pitch outside [cols, 2^28]");
  if (batch > 1 && (batch_stride < (rows - 1) * (rows > 1 ? ld : 0) + cols || batch_stride > kMaxBatchStride))
    return fail(MUON_ERR_BAD_SHAPE, n + ": batch stride too small (matrices overlap) or above 2^48");
  return MUON_OK;
}

inline int64_t strided_bytes(int32_t dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t batch_stride) {
  if (batch == 0 || rows == 0 || cols == 0) return 0;
  return ((batch - 1) * batch_stride + (rows - 1) * ld + cols) * element_size(dtype);
}

// Bytes and checks of a quantised operand.
inline int64_t data_bytes(const muon_fp8_t& t) { return t.batch * t.rows * fp8_data_pitch(t.cols); }
inline int64_t scale_bytes(const muon_fp8_t& t) { return t.batch * t.rows * fp8_scale_pitch(t.cols); }

inline int check_operand(const muon_fp8_t* t, const char* name) {
  const std::string n(name);
  if (t->rows < 0 || t->cols < 0 || t->rows > MUON_FP8_MAX_SIDE || t->cols > MUON_FP8_MAX_SIDE)
    return fail(MUON_ERR_BAD_SHAPE, n + ": rows and cols must lie in [0, MUON_FP8_MAX_SIDE]");
  if (t->batch < 1 || t->batch > MUON_FP8_MAX_BATCH)
    return fail(MUON_ERR_BAD_SHAPE, n + ": batch must lie in [1, MUON_FP8_MAX_BATCH]");
  if (t->format != MUON_FP8_E4M3 && t->format != MUON_FP8_E5M2)
    return fail(MUON_ERR_UNSUPPORTED, n + ": format must be E4M3 or E5M2");
  if (t->rows > 0 && t->cols > 0) {
    if (t->data == nullptr || t->scale == nullptr) return fail(MUON_ERR_NULL, n + ": data and scale must not be NULL");
    if (misaligned(t->data, 16) || misaligned(t->scale, 4))
      return fail(MUON_ERR_ALIGN, n + ": data must be 16-byte and scale 4-byte aligned");
  }
  return MUON_OK;
}

}  // namespace muon
