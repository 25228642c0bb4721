// Routing of rows to experts, the order of routed rows, and the weighted sum of the
// experts' outputs (gfx950).
#include "common.hpp"
#include "fp8.hpp"

namespace muon {

template <int DT> __device__ __forceinline__ float load1(const void* p, int64_t i) { return grad_to_f32<DT>(p, i); }
template <int DT> __device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (DT == MUON_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (DT == MUON_DTYPE_BF16) static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
  else static_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
}

// ---------------------------------------------------------------------------
// Reductions over a team of 64 or 32 neighbouring lanes with row shifts and broadcasts (no
// LDS); the result in all of its lanes. A wave has one team of 64, uniform values for it,
// or two of 32.

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t shifted(uint32_t v, uint32_t other) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(other), static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ bool upper_team() { return (threadIdx.x & 32) != 0; }

template <int TEAM, typename F>
__device__ __forceinline__ uint32_t team_fold(uint32_t v, uint32_t identity, F&& f) {
  v = f(v, shifted<0x111, 0xf>(v, identity));   // lanes 1, 2, 4, 8 before, within 16
  v = f(v, shifted<0x112, 0xf>(v, identity));
  v = f(v, shifted<0x114, 0xf>(v, identity));
  v = f(v, shifted<0x118, 0xf>(v, identity));
  v = f(v, shifted<0x142, 0xa>(v, identity));   // last lane of the 16 before, in the odd ones
  if constexpr (TEAM == 64) {
    v = f(v, shifted<0x143, 0xc>(v, identity));   // last lane of the first 32
    return lane_value(v, 63);
  } else {
    const uint32_t lower = lane_value(v, 31), upper = lane_value(v, 63);
    return upper_team() ? upper : lower;
  }
}
template <int TEAM>
__device__ __forceinline__ uint32_t team_max_u(uint32_t v) {
  return team_fold<TEAM>(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int TEAM>
__device__ __forceinline__ float team_max_f(float v) {   // ignores NaN
  return __uint_as_float(team_fold<TEAM>(__float_as_uint(v), __float_as_uint(-__builtin_huge_valf()), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double add_shifted(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t o = static_cast<uint64_t>(shifted<CTRL, ROWS>(static_cast<uint32_t>(b >> 32), 0u)) << 32 |
                     shifted<CTRL, ROWS>(static_cast<uint32_t>(b), 0u);
  return v + __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double lane_double(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, static_cast<uint64_t>(lane_value(static_cast<uint32_t>(b >> 32), lane)) << 32 |
                                        lane_value(static_cast<uint32_t>(b), lane));
}
template <int TEAM>
__device__ __forceinline__ double team_add(double v) {
  v = add_shifted<0x111, 0xf>(v);
  v = add_shifted<0x112, 0xf>(v);
  v = add_shifted<0x114, 0xf>(v);
  v = add_shifted<0x118, 0xf>(v);
  v = add_shifted<0x142, 0xa>(v);
  if constexpr (TEAM == 64) {
    v = add_shifted<0x143, 0xc>(v);
    return lane_double(v, 63);
  } else {
    const double lower = lane_double(v, 31), upper = lane_double(v, 63);
    return upper_team() ? upper : lower;
  }
}
// The team's lanes for which `p` holds, the first one in bit 0.
template <int TEAM>
__device__ __forceinline__ uint64_t team_ballot(bool p) {
  const uint64_t m = __ballot(p);
  if constexpr (TEAM == 64) return m;
  return upper_team() ? m >> 32 : m & 0xffffffffull;
}

// ---------------------------------------------------------------------------
// Routing: a team of 64 lanes per token, or of 32 for up to 64 experts; expert TEAM i + lane
// in register i of a lane.
//
// Scores and keys are held in 64 bits: which experts a token gets is then the same
// wherever it is computed in 64 bits, while 32-bit exponentials of different libraries
// would order near neighbours differently. What bounds it is the number of steps, not
// memory: choosing takes top_k rounds of one maximum over the wave. Keys are mapped to
// ordered 64-bit integers and the maximum is taken of their upper halves; only lanes that
// tie there compare the lower ones. The lane that holds the chosen expert notes its slot
// and writes it at the end. 16384 tokens, 64 experts, 8 groups, 6 of 64: 12 us with teams of
// 32 (64: 15; 43 us with 64-bit butterflies through LDS).

constexpr double kNone = -__builtin_huge_val();      // not available
constexpr double kLowest = -1.7976931348623157e308;  // a NaN key: below every number

// Ordered key: larger numbers have larger keys, 0 stands for "not available".
struct Key {
  uint32_t hi, lo;
};
__device__ __forceinline__ Key ordered(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t o = b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
  return v == kNone ? Key{0u, 0u} : Key{static_cast<uint32_t>(o >> 32), static_cast<uint32_t>(o)};
}

// Whether this lane holds the team's best key (largest, ties to the lowest TEAM reg + lane);
// in no lane if none is left. `reg` is the register the lane's own best sits in.
template <int TEAM>
__device__ __forceinline__ bool is_best(const Key& k, int reg) {
  auto several = [](uint64_t who) {   // in any team of the wave
    const uint32_t lower = static_cast<uint32_t>(who), upper = static_cast<uint32_t>(who >> 32);
    if constexpr (TEAM == 64) return (who & (who - 1)) != 0;
    else return ((lower & (lower - 1)) | (upper & (upper - 1))) != 0;
  };
  const uint32_t hi = team_max_u<TEAM>(k.hi);   // by all lanes: not behind a condition
  bool in = hi != 0u && k.hi == hi;
  if (several(__ballot(in))) {
    const uint32_t lo = team_max_u<TEAM>(in ? k.lo : 0u);
    in = in && k.lo == lo;
    if (several(__ballot(in))) {
      const uint32_t first = ~team_max_u<TEAM>(in ? ~static_cast<uint32_t>(reg) : 0u);
      in = in && static_cast<uint32_t>(reg) == first;
      const uint64_t who = team_ballot<TEAM>(in);
      in = in && __builtin_ctzll(who) == (threadIdx.x & (TEAM - 1));
    }
  }
  return in;
}

// One softmax or sigmoid score per register; -inf logits score 0, a row of them too.
template <int TEAM, int V>
__device__ __forceinline__ void row_scores(const float (&l)[V], int score, double (&s)[V]) {
  if (score == MUON_ROUTE_SOFTMAX) {
    float most = -__builtin_huge_valf();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      most = fmaxf(most, l[i]);   // ignores NaN
      nan = nan || l[i] != l[i];
    }
    const double m = static_cast<double>(team_max_f<TEAM>(most));
    nan = team_ballot<TEAM>(nan) != 0;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] == -__builtin_huge_valf() ? 0.0 : exp(static_cast<double>(l[i]) - m);
      sum += s[i];
    }
    sum = team_add<TEAM>(sum);
    if (nan) sum = __builtin_nan("");
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = l[i] == -__builtin_huge_valf() ? 0.0 : s[i] / sum;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
  }
}

template <int DT, int TEAM, int V>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  extern __shared__ double keys[];   // experts of each team, where there are groups
  constexpr int TEAMS = 256 / TEAM;
  const int lane = threadIdx.x & (TEAM - 1), team = threadIdx.x / TEAM;
  const int64_t row = static_cast<int64_t>(flat_block()) * TEAMS + team;
  const bool live = row < a.tokens;
  if (__ballot(live) == 0) return;   // no barrier below: a wave is by itself
  const int64_t token = live ? row : a.tokens - 1;
  const int E = a.experts;
  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * TEAM + lane;
    l[i] = e < E ? load1<DT>(a.logits, token * a.ld + e) : -__builtin_huge_valf();
  }
  double s[V], key[V];
  row_scores<TEAM, V>(l, a.score, s);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * TEAM + lane;
    key[i] = s[i];
    if (a.bias != nullptr && e < E) key[i] += static_cast<double>(a.bias[e]);
    if (key[i] != key[i]) key[i] = kLowest;
    if (e >= E || l[i] == -__builtin_huge_valf()) key[i] = kNone;
  }
  Key o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = ordered(key[i]);
  if (a.n_groups > 1) {
    const int per = E / a.n_groups;
    double* mine = keys + team * E;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * TEAM + lane < E) mine[i * TEAM + lane] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // lane g scores group g
    double gk = kNone;
    if (lane < a.n_groups) {
      double t1 = kNone, t2 = kNone;
#pragma unroll 4
      for (int j = 0; j < per; ++j) {
        const double k = mine[lane * per + j];
        t2 = fmax(t2, fmin(t1, k));
        t1 = fmax(t1, k);
      }
      gk = t1;
      if (a.group_top > 1 && t2 > kNone) gk = t1 <= kLowest ? t1 : (t2 <= kLowest ? kLowest : t1 + t2);
    }
    Key k = ordered(gk);
    bool keep = false;
    for (int j = 0; j < a.top_groups; ++j)
      if (is_best<TEAM>(k, 0)) {
        keep = true;
        k = Key{0u, 0u};
      }
    const uint64_t kept = team_ballot<TEAM>(keep);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * TEAM + lane;
      if (e < E && !((kept >> (e / per)) & 1)) o[i] = Key{0u, 0u};
    }
  }
  int slot[V];   // of the expert in register i, -1 if it is not chosen
#pragma unroll
  for (int i = 0; i < V; ++i) slot[i] = -1;
  for (int j = 0; j < a.top_k; ++j) {
    Key k = o[0];
    int reg = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (o[i].hi > k.hi || (o[i].hi == k.hi && o[i].lo > k.lo)) {
        k = o[i];
        reg = i;
      }
    const bool mine = is_best<TEAM>(k, reg);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (mine && reg == i) {
        slot[i] = j;
        o[i] = Key{0u, 0u};
      }
  }
  double sum = 0.0;
  int found = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sum += slot[i] >= 0 ? s[i] : 0.0;
    found += __popcll(team_ballot<TEAM>(slot[i] >= 0));
  }
  double f = static_cast<double>(a.scale);
  if (a.renormalize) f /= team_add<TEAM>(sum) + 1e-20;
  if (!live) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (slot[i] >= 0) {
      a.ids[token * a.top_k + slot[i]] = i * TEAM + lane;
      a.weights[token * a.top_k + slot[i]] = static_cast<float>(s[i] * f);
    }
  if (lane >= found && lane < a.top_k) {   // slots that no expert is left for
    a.ids[token * a.top_k + lane] = -1;
    a.weights[token * a.top_k + lane] = 0.0f;
  }
}

// The gradient: with T = sum of the chosen s + 1e-20 and w_j = scale s_j / T,
//   ds_j = (scale dw_j - sum_i dw_i w_i) / T     (scale dw_j without renormalisation)
//   sigmoid: dl_j = ds_j s_j (1 - s_j);  softmax: dl_i = s_i (ds_i - sum_j ds_j s_j).
// The chosen slots' values reach their experts' registers slot by slot, broadcast to the
// wave (at most 32).
template <int DT, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t token = static_cast<int64_t>(flat_block()) * 4 + wave;
  if (token >= a.tokens) return;
  const int E = a.experts;
  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? load1<DT>(a.logits, token * a.ld + e) : -__builtin_huge_valf();
  }
  int id = -1;
  float dw = 0.0f;
  if (lane < a.top_k) {
    id = a.ids[token * a.top_k + lane];
    if (id < 0 || id >= E) id = -1;
    else dw = a.dweights[token * a.top_k + lane];
  }
  double s[V], ds[V];
  row_scores<64, V>(l, a.score, s);
  bool hit[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ds[i] = 0.0;
    hit[i] = false;
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(dw), j));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == i * 64 + lane) {
        ds[i] = static_cast<double>(d);
        hit[i] = true;
      }
  }
  const double f = static_cast<double>(a.scale);
  if (a.renormalize) {
    double total = 0.0, dot = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      total += hit[i] ? s[i] : 0.0;
      dot += hit[i] ? ds[i] * s[i] : 0.0;
    }
    total = team_add<64>(total) + 1e-20;
    dot = team_add<64>(dot) / total;
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] = hit[i] ? f * (ds[i] - dot) / total : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] *= f;
  }
  double sum = 0.0;
  if (a.score == MUON_ROUTE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += hit[i] ? ds[i] * s[i] : 0.0;
    sum = team_add<64>(sum);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    double d;
    if (a.score == MUON_ROUTE_SOFTMAX) d = s[i] * (ds[i] - sum);
    else d = hit[i] ? ds[i] * s[i] * (1.0 - s[i]) : 0.0;
    if (l[i] == -__builtin_huge_valf()) d = 0.0;
    if (e < E) store1<DT>(a.dlogits, token * a.ld_d + e, static_cast<float>(d));
  }
}

template <int DT, int TEAM, int V>
static hipError_t launch_teams(const RouteArgs& a, hipStream_t s) {
  constexpr int TEAMS = 256 / TEAM;
  const size_t lds = a.n_groups > 1 ? TEAMS * sizeof(double) * a.experts : 0;
  hipLaunchKernelGGL((route_kernel<DT, TEAM, V>), flat_grid((a.tokens + TEAMS - 1) / TEAMS), dim3(256), lds, s, a);
  return hipGetLastError();
}
template <int DT>
static hipError_t route_dt(const RouteArgs& a, hipStream_t s) {
  // Teams of 32 take half the steps per token and twice the scores per lane: 64 experts 15 ->
  // 12 us for 16384 tokens, 3.3 us either way for 16; 128 experts 12.1 -> 11.8 and 18.3 ->
  // 16.4 (8 groups), but 3.3 -> 4.5 and 4.7 -> 6.1 for 16.
  if (a.experts <= 64 && a.n_groups <= 32) return launch_teams<DT, 32, 2>(a, s);   // a lane per group
  if (a.experts <= 64) return launch_teams<DT, 64, 1>(a, s);
  if (a.experts <= 128) return launch_teams<DT, 64, 2>(a, s);
  if (a.experts <= 256) return launch_teams<DT, 64, 4>(a, s);
  return launch_teams<DT, 64, 16>(a, s);
}
hipError_t launch_route(int dtype, const RouteArgs& a, hipStream_t s) {
  if (a.tokens <= 0) return hipSuccess;
  if (dtype == MUON_DTYPE_BF16) return route_dt<MUON_DTYPE_BF16>(a, s);
  if (dtype == MUON_DTYPE_F16) return route_dt<MUON_DTYPE_F16>(a, s);
  return route_dt<MUON_DTYPE_F32>(a, s);
}

template <int DT>
static hipError_t route_backward_dt(const RouteBackArgs& a, hipStream_t s) {
  const dim3 grid = flat_grid((a.tokens + 3) / 4);
  if (a.experts <= 64) hipLaunchKernelGGL((route_backward_kernel<DT, 1>), grid, dim3(256), 0, s, a);
  else if (a.experts <= 128) hipLaunchKernelGGL((route_backward_kernel<DT, 2>), grid, dim3(256), 0, s, a);
  else if (a.experts <= 256) hipLaunchKernelGGL((route_backward_kernel<DT, 4>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((route_backward_kernel<DT, 16>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_route_backward(int dtype, const RouteBackArgs& a, hipStream_t s) {
  if (a.tokens <= 0) return hipSuccess;
  if (dtype == MUON_DTYPE_BF16) return route_backward_dt<MUON_DTYPE_BF16>(a, s);
  if (dtype == MUON_DTYPE_F16) return route_backward_dt<MUON_DTYPE_F16>(a, s);
  return route_backward_dt<MUON_DTYPE_F32>(a, s);
}

// ---------------------------------------------------------------------------
// Expert order: a stable counting sort. Block b owns slots [b P, (b + 1) P). The first
// launch counts each block's slots per expert; in the second every block sums the
// counts of all blocks (the padded offsets) and of the blocks before it (its first row
// of each expert), then places its slots in order. Small inputs take one block and one
// launch. Counting uses integer LDS atomics, whose order does not matter; placing ranks
// the 64 slots of a wave step with ballots, so rows come out in slot order.
constexpr int kOrderThreads = 512, kOrderWaves = kOrderThreads / 64;
constexpr int64_t kOrderBlock = 1024;   // slots of a block, unless that makes too many blocks
constexpr int32_t kOrderBlocks = 256;

int32_t order_blocks(int64_t n) {
  if (n <= 4 * kOrderBlock) return 1;
  return static_cast<int32_t>(std::min<int64_t>((n + kOrderBlock - 1) / kOrderBlock, kOrderBlocks));
}

__device__ __forceinline__ int slot_expert(const OrderArgs& a, int64_t i) {
  const int e = a.ids[i];
  return e >= 0 && e < a.experts ? e : -1;
}

__global__ __launch_bounds__(kOrderThreads) void order_hist_kernel(OrderArgs a) {
  __shared__ int h[MUON_ROUTE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.experts; e += kOrderThreads) h[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.per_block, hi = min(a.n, lo + a.per_block);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kOrderThreads) {
    const int e = slot_expert(a, i);
    if (e >= 0) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kOrderThreads)
    a.hist[static_cast<int64_t>(blockIdx.x) * a.experts + e] = h[e];
}

__global__ __launch_bounds__(kOrderThreads) void order_place_kernel(OrderArgs a) {
  __shared__ int total[MUON_ROUTE_MAX_EXPERTS];              // slots of each expert
  __shared__ int earlier[MUON_ROUTE_MAX_EXPERTS];            // those in earlier blocks
  __shared__ int pad[MUON_ROUTE_MAX_EXPERTS];                // its first padding row
  __shared__ int next[kOrderWaves][MUON_ROUTE_MAX_EXPERTS];  // next row of each expert, per wave
  __shared__ int scan[kOrderWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int E = a.experts;
  const int64_t lo = blockIdx.x * a.per_block, hi = min(a.n, lo + a.per_block);
  // each wave places a contiguous part of the block's slots
  const int64_t part = ((hi - lo + kOrderWaves - 1) / kOrderWaves + 63) / 64 * 64;
  const int64_t wlo = min(hi, lo + wave * part), whi = min(hi, wlo + part);
  for (int e = t; e < E; e += kOrderThreads)
    for (int w = 0; w < kOrderWaves; ++w) next[w][e] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 64) {
    const int e = slot_expert(a, i);
    if (e >= 0) atomicAdd(&next[wave][e], 1);
  }
  __syncthreads();
  // totals, slots before this block and before each wave; the blocks' counts are summed by
  // all threads together
  if (a.blocks > 1) {
    for (int e = t; e < E; e += kOrderThreads) total[e] = earlier[e] = 0;
    __syncthreads();
    const int parts = max(1, kOrderThreads / E);
    for (int e0 = 0; e0 < E; e0 += kOrderThreads) {
      const int e = e0 + (E < kOrderThreads ? t % E : t), part = E < kOrderThreads ? t / E : 0;
      if (e < E && part < parts) {
        int all = 0, before = 0;
#pragma unroll 4
        for (int b = part; b < a.blocks; b += parts) {
          const int c = a.hist[static_cast<int64_t>(b) * E + e];
          before += b < static_cast<int>(blockIdx.x) ? c : 0;
          all += c;
        }
        atomicAdd(&total[e], all);
        atomicAdd(&earlier[e], before);
      }
    }
    __syncthreads();
  }
  for (int e = t; e < E; e += kOrderThreads) {
    int before = a.blocks > 1 ? earlier[e] : 0;
    for (int w = 0; w < kOrderWaves; ++w) {
      const int c = next[w][e];
      next[w][e] = before;
      before += c;
    }
    if (a.blocks == 1) total[e] = before;
  }
  __syncthreads();
  // padded offsets: exclusive scan over the experts, kOrderThreads at a time
  int64_t base = 0;
  for (int e0 = 0; e0 < E; e0 += kOrderThreads) {
    const int e = e0 + t;
    const int n = e < E ? (total[e] + a.align - 1) / a.align * a.align : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    if (lane == 63) scan[wave] = incl;
    __syncthreads();
    int64_t first = base + incl - n;
    int64_t sum = 0;
    for (int w = 0; w < kOrderWaves; ++w) {
      if (w < wave) first += scan[w];
      sum += scan[w];
    }
    if (e < E) {
      for (int w = 0; w < kOrderWaves; ++w) next[w][e] += static_cast<int>(first);
      if (blockIdx.x == 0) {
        a.offsets[e] = static_cast<int>(first);
        a.counts[e] = total[e];
      }
      pad[e] = static_cast<int>(first) + total[e];
    }
    base += sum;
    __syncthreads();
  }
  if (blockIdx.x == 0 && t == 0) a.offsets[E] = static_cast<int>(base);
  // padding rows, a wave per expert; rows behind the last expert
  for (int e = static_cast<int>(blockIdx.x) * kOrderWaves + wave; e < E; e += a.blocks * kOrderWaves) {
    const int n = (a.align - total[e] % a.align) % a.align;
    for (int r = lane; r < n; r += 64) a.rows[pad[e] + r] = -1;
  }
  for (int64_t r = base + static_cast<int64_t>(blockIdx.x) * kOrderThreads + t; r < a.capacity;
       r += static_cast<int64_t>(a.blocks) * kOrderThreads)
    a.rows[r] = -1;
  // placing, 64 slots of the wave at a time
  for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = i < whi ? slot_expert(a, i) : -1;
    unsigned long long same = __ballot(e >= 0);
    for (int bit = 0; (1 << bit) < E; ++bit) {
      const unsigned long long m = __ballot((e >> bit) & 1);
      same &= ((e >> bit) & 1) ? m : ~m;
    }
    int row = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      row = next[wave][e] + rank;
      a.rows[row] = static_cast<int>(i);
    }
    if (i < whi) a.pos[i] = row;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same >> lane) == 1ull) next[wave][e] = row + 1;   // the last of its expert
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

hipError_t launch_order_hist(const OrderArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(order_hist_kernel, dim3(a.blocks), dim3(kOrderThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_order_place(const OrderArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(order_place_kernel, dim3(a.blocks), dim3(kOrderThreads), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combination: one workgroup per token, eight columns per thread and pass, 16 bytes at any
// element-aligned place.

typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int DT>
__device__ __forceinline__ void read8(const void* p, int64_t i, int n, float (&v)[8]) {
  if (n == 8) {
    if constexpr (DT == MUON_DTYPE_F32) {
      const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
      const f32x4 a = q[0], b = q[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    } else {
      const u16x8 u = *reinterpret_cast<const u16x8_any*>(static_cast<const unsigned short*>(p) + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = DT == MUON_DTYPE_BF16 ? bf16_bits_to_f32(u[e]) : f16_bits_to_f32(u[e]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < n ? load1<DT>(p, i + e) : 0.0f;
}

template <int DT>
__device__ __forceinline__ void write8(void* p, int64_t i, int n, const float (&v)[8]) {
  if (n == 8) {
    if constexpr (DT == MUON_DTYPE_F32) {
      f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i);
      q[0] = f32x4{v[0], v[1], v[2], v[3]};
      q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      using T = std::conditional_t<DT == MUON_DTYPE_BF16, __bf16, _Float16>;
      T o[8];
      rne<T, 8>(v, o);
      u16x8 u;
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __builtin_bit_cast(unsigned short, o[e]);
      *reinterpret_cast<u16x8_any*>(static_cast<unsigned short*>(p) + i) = u;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) store1<DT>(p, i + e, v[e]);
}

// Bound by memory: every row of o once. Four rows at a time are in flight. 8192 tokens of 6
// rows of 2048 bf16: 49 us (4.8 TB/s, a large copy reaches 5.1).
constexpr int kCombineRows = 4;

template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t t = flat_block();
  if (t >= a.tokens) return;
  const int32_t* pos = a.pos + t * a.top_k;
  const float* w = a.weights + t * a.top_k;
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += 256 * 8) {
    const int n = static_cast<int>(min<int64_t>(8, a.cols - c));
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
    for (int j0 = 0; j0 < a.top_k; j0 += kCombineRows) {
      float v[kCombineRows][8], wj[kCombineRows];
#pragma unroll
      for (int k = 0; k < kCombineRows; ++k) {
        const int j = j0 + k;
        const int r = j < a.top_k ? pos[j] : -1;
        const bool has = r >= 0 && r < a.o_rows;
        wj[k] = has ? w[j] : 0.0f;
        read8<DT>(a.o, has ? r * a.ld_o + c : 0, has ? n : 0, v[k]);
      }
#pragma unroll
      for (int k = 0; k < kCombineRows; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += wj[k] * v[k][e];
    }
    write8<DT>(a.y, t * a.ld_y + c, n, y);
  }
}

constexpr int kBackRows = 1;   // rows in flight: 2 and 4 were 4% and 19% slower
// Row by row: its product with dy, its gradient, a join over the waves. 8192 tokens of 6 rows
// of 2048 bf16: 95 us (4.6 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineArgs a) {
  __shared__ float red[2][4][kBackRows];
  const int64_t t = flat_block();
  if (t >= a.tokens) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0, turn = 0; j0 < a.top_k; j0 += kBackRows, turn ^= 1) {
    int r[kBackRows];
    float wj[kBackRows], sum[kBackRows];
#pragma unroll
    for (int k = 0; k < kBackRows; ++k) {
      r[k] = j0 + k < a.top_k ? a.pos[t * a.top_k + j0 + k] : -1;
      if (r[k] >= a.o_rows) r[k] = -1;
      wj[k] = r[k] >= 0 ? a.weights[t * a.top_k + j0 + k] : 0.0f;
      sum[k] = 0.0f;
    }
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += 256 * 8) {
      const int n = static_cast<int>(min<int64_t>(8, a.cols - c));
      float d[8], v[kBackRows][8];
      read8<DT>(a.dy, t * a.ld_dy + c, n, d);
      if (a.dweights != nullptr) {
#pragma unroll
        for (int k = 0; k < kBackRows; ++k) read8<DT>(a.o, r[k] >= 0 ? r[k] * a.ld_o + c : 0, r[k] >= 0 ? n : 0, v[k]);
      }
      if (a.d_o != nullptr) {
#pragma unroll
        for (int k = 0; k < kBackRows; ++k) {
          if (r[k] < 0) continue;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = d[e] * wj[k];
          write8<DT>(a.d_o, r[k] * a.ld_do + c, n, x);
        }
      }
      if (a.dweights != nullptr) {
#pragma unroll
        for (int k = 0; k < kBackRows; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[k] += r[k] >= 0 ? d[e] * v[k][e] : 0.0f;
      }
    }
    if (a.dweights != nullptr) {
#pragma unroll
      for (int k = 0; k < kBackRows; ++k) {
        sum[k] = wave_sum(sum[k]);
        if (lane == 0) red[turn][wave][k] = sum[k];
      }
      __syncthreads();   // the other half of `red` is free again: everybody is past its reads
      const int k = threadIdx.x;
      if (k < kBackRows && j0 + k < a.top_k)
        a.dweights[t * a.top_k + j0 + k] = (red[turn][0][k] + red[turn][1][k]) + (red[turn][2][k] + red[turn][3][k]);
    }
  }
}

#define MUON_BY_DTYPE(kernel, grid, a)                                                                      \
  do {                                                                                                      \
    if (dtype == MUON_DTYPE_BF16) hipLaunchKernelGGL((kernel<MUON_DTYPE_BF16>), grid, dim3(256), 0, s, a);  \
    else if (dtype == MUON_DTYPE_F16) hipLaunchKernelGGL((kernel<MUON_DTYPE_F16>), grid, dim3(256), 0, s, a); \
    else hipLaunchKernelGGL((kernel<MUON_DTYPE_F32>), grid, dim3(256), 0, s, a);                            \
  } while (0)

hipError_t launch_combine(int dtype, const CombineArgs& a, hipStream_t s) {
  if (a.tokens <= 0 || a.cols <= 0) return hipSuccess;
  MUON_BY_DTYPE(combine_kernel, flat_grid(a.tokens), a);
  return hipGetLastError();
}
hipError_t launch_combine_backward(int dtype, const CombineArgs& a, hipStream_t s) {
  if (a.tokens <= 0) return hipSuccess;
  MUON_BY_DTYPE(combine_backward_kernel, flat_grid(a.tokens), a);
  return hipGetLastError();
}

}  // namespace muon
