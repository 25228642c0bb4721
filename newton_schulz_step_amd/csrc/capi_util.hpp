// Helpers shared by the C entry points: the thread's error message, argument
// checks and timed launches.
#pragma once

#include <exception>
#include <string>
#include <vector>

#include "common.hpp"

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

}  // namespace muon
