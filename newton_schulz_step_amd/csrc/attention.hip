// Attention over packed sequences and its gradient (gfx950).
//
//   S = c Q K^T,  P = exp(S - lse),  O = P V          (rows of P over the keys that are seen)
//   delta = rowsum(dO O),  dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),
//   dQ = c dS K,  dK = c dS^T Q
//
// Every product runs on the 32x32x16 matrix instructions. A wave owns 32 columns of a
// transposed score tile, one per lane (and its twin 32 lanes on): queries in the forward pass
// and in dQ, keys in dK and dV. The instruction returns 4 consecutive rows of a column in 4
// registers, rows 8 g + 4 (lane / 32) + 0..3, so that, rounded to 16 bits, the tile is the next
// product's right operand as it stands, with the contraction in the order
//   slot 8 h + e  <->  row 4 h + e (e < 4),  8 + 4 h + e - 4 (e >= 4)     of 16 rows,
// and the left operand is read out of LDS in that order by transposed reads. No score leaves the
// registers. The gradient is two kernels, one that walks over keys (dQ) and one that walks over
// queries (dK, dV): scores and dP are computed twice, 7 products instead of 5, and in turn
// every sum has one owner and one order, without atomics, and a group's query heads are
// summed in registers.
#include <algorithm>
#include <type_traits>

#include "attention.hpp"
#include "fp8.hpp"
#include "rows.hpp"

namespace muon {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256, kWaves = 4;
constexpr int kWaveRows = 32;      // columns of the transposed tile that a wave owns
constexpr int kStage = 64;         // rows of a tile in LDS

template <typename T> struct Half;
template <> struct Half<__bf16> {
  typedef bf16x8 v8;
  typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4;
  static constexpr bool narrow = false;   // fp32's range
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ v4 transposed(MUON_LDS const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((MUON_LDS v4*)(p));
  }
};
template <> struct Half<_Float16> {
  typedef f16x8 v8;
  typedef __attribute__((__vector_size__(4 * sizeof(__fp16)))) __fp16 v4;
  static constexpr bool narrow = true;
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ v4 transposed(MUON_LDS const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4f16((MUON_LDS v4*)(p));
  }
};

// x of this lane and of its twin 32 lanes on.
__device__ __forceinline__ float twin_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float twin_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------------------
// Tiles in LDS: rows of 64 or 128 elements, DP of them used, in 16-byte chunks, chunk c of row r at place c ^ swizzle(r).
// A row operand is read with one row per lane and the same chunk in all of them, a transposed
// one with four chunks of four consecutive rows per half wave; in both the swizzle spreads the
// lanes that are served together over all banks.
template <int DP> struct Tile {
  static constexpr int WIDE = DP > 64 ? 128 : 64;   // elements of a row in LDS
  static constexpr int CHUNKS = WIDE / 8, PITCH = WIDE * 2, BYTES = kStage * PITCH;   // of kStage rows
  static constexpr int KS = DP / 16;    // steps of a contraction over the columns
  static constexpr int DB = DP / 32;    // blocks of 32 columns
  static __device__ __forceinline__ int swizzle(int r) {
    return WIDE == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  }
  // Byte offset of row `lane % 32`'s chunk lane / 32; step ks is at ^ (ks * 32).
  static __device__ __forceinline__ int row_offset() {
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    return r * PITCH + ((h ^ swizzle(r)) << 4);
  }
  // Byte offset of the lane's part of a transposed read of rows 0 .. 15 and columns 0 .. 31;
  // part e (slots 4 e ..) is at (^ (e * 32)) + e * 8 * PITCH, column block b at ^ (b * 64).
  static __device__ __forceinline__ int column_offset() {
    const int lane = threadIdx.x & 63, g = lane >> 4, s = lane & 15;
    const int r = 4 * (g >> 1) + (s >> 2), c = (g & 1) * 2 + ((s & 3) >> 1);
    return r * PITCH + ((c ^ swizzle(r)) << 4) + (s & 1) * 8;
  }
};

#define MUON_HEAD_RSRC(p, n) __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, n, 0x00027000)

// The loads of one operand's tiles straight to LDS: columns behind `dim` and rows behind the
// last one arrive as zeros (no bytes there).
template <int DP, int WAVES, int ROWS = kStage> struct TileLoads {
  static constexpr int LOADS = ROWS * Tile<DP>::PITCH / 1024 / WAVES;
  int at[LOADS];
  int stride, dim;   // bytes between rows, elements
  __device__ __forceinline__ void init(int64_t token_stride, int d) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    stride = static_cast<int>(token_stride * 2);
    dim = d;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int place = (wave * LOADS + i) * 64 + lane;
      const int r = place / Tile<DP>::CHUNKS, c = (place % Tile<DP>::CHUNKS) ^ Tile<DP>::swizzle(r);
      at[i] = c * 8 < d ? r * stride + c * 16 : static_cast<int>(0x80000000u);
    }
  }
  // `rows` rows from `from` on (none or fewer than none: zeros)
  __device__ __forceinline__ void issue(const char* from, int rows, MUON_LDS char* to) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    rows = min(rows, ROWS);
    const auto rsrc = MUON_HEAD_RSRC(from, rows > 0 ? (rows - 1) * stride + dim * 2 : 0);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MUON_LDS void*)(to + (wave * LOADS + i) * 1024), 16, at[i], 0, 0, 0);
  }
};

__device__ __forceinline__ void arrived() {   // own loads to LDS and reads of it are done, then everybody's
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename T>
__device__ __forceinline__ typename Half<T>::v8 row_part(MUON_LDS const char* tile, int offset) {
  return *reinterpret_cast<MUON_LDS const typename Half<T>::v8*>(tile + offset);
}
// Rows `16 k` .. of the tile, column block b, as a left operand with the rows contracted.
template <typename T, int DP>
__device__ __forceinline__ typename Half<T>::v8 column_part(MUON_LDS const char* tile, int offset, int k, int b) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const u2 lo = __builtin_bit_cast(u2, Half<T>::transposed(tile + (offset ^ (b * 64)) + k * 16 * Tile<DP>::PITCH));
  const u2 hi = __builtin_bit_cast(u2, Half<T>::transposed(tile + (offset ^ (b * 64) ^ 32) + (k * 16 + 8) * Tile<DP>::PITCH));
  return __builtin_bit_cast(typename Half<T>::v8, u4{lo[0], lo[1], hi[0], hi[1]});
}

// 16 rows (two groups of four registers) of a column as a right operand, rounded to T. The
// products' operands have 16 bits: half a step of T per probability or score gradient, which
// adds up like noise over the keys, while all sums stay in fp32.
template <typename T>
__device__ __forceinline__ typename Half<T>::v8 operand(const f32x16& x, int k) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  f32x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x[8 * k + e];
  return __builtin_convertvector(v, typename Half<T>::v8);
}

// The right operand of a lane's row: 8 columns per step, 16 apart.
template <typename T, int DP>
__device__ __forceinline__ void load_rows(typename Half<T>::v8 (&f)[Tile<DP>::KS], const char* base, int64_t row, bool there,
                                          int64_t stride, int dim) {
  const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
  for (int ks = 0; ks < Tile<DP>::KS; ++ks) {
    const int c = ks * 16 + h * 8;
    if (there && c < dim) {
      f[ks] = *reinterpret_cast<const typename Half<T>::v8*>(base + (row * stride + c) * 2);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[ks][e] = static_cast<T>(0.0f);
    }
  }
}

// A wave's transposed result (rows = columns of the head, one of its 32 rows per lane), rounded
// and written through LDS in whole rows. `lds`: 32 rows of the wave's own.
template <typename T, int DP>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[Tile<DP>::DB], float factor, MUON_LDS char* lds, char* base,
                                           int64_t row, int64_t rows, int64_t stride, int dim) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  constexpr int CH = Tile<DP>::CHUNKS;
  typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int b = 0; b < Tile<DP>::DB; ++b)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[b][4 * g + e] * factor;
      T o[4];
      rne<T, 4>(v, o);
      *reinterpret_cast<MUON_LDS t4*>(lds + r * Tile<DP>::PITCH + (((b * 4 + g) ^ (r & (CH - 1))) << 4) + h * 8) =
          t4{o[0], o[1], o[2], o[3]};
    }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < kWaveRows * CH / 64; ++i) {
    const int place = i * 64 + lane, k = place / CH, c = place % CH;
    const auto v = *reinterpret_cast<MUON_LDS const typename Half<T>::v8*>(lds + k * Tile<DP>::PITCH + ((c ^ (k & (CH - 1))) << 4));
    if (row + k < rows && c * 8 < dim) *reinterpret_cast<typename Half<T>::v8*>(base + ((row + k) * stride + c * 8) * 2) = v;
  }
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// Which rows of which sequence and which head a workgroup takes. Workgroups that follow each
// other go to the 8 XCDs in turn, each with its own L2; with a multiple of 8 heads, a head's
// tiles all go to one XCD, and neighbouring heads, which share keys, with it. The tiles
// with the most work come first. Among up to 64 sequences, one per lane, each wave finds its tile by
// itself; among more a launch before lists them (32 texts, 4095 tokens, 16 heads of 64, fp16:
// 14.0 us a call without the list, 18.0 with it; gradient of 12 texts, 8191 tokens, 32 heads of 128: 311 and 313).
struct Place {
  int64_t start;   // first token of the sequence
  int len;         // its tokens
  int row;         // first row of the tile
  int head;
};

// Inclusive over the lanes up to each one's, of values that are not negative.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lanes_below(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, true);
}
__device__ __forceinline__ int lanes_max(int x) {
  x = max(x, lanes_below<0x111, 0xf>(x));   // 1, 2, 4, 8 lanes back in a row of 16, then the last of rows 0 and 2, of row 1
  x = max(x, lanes_below<0x112, 0xf>(x));
  x = max(x, lanes_below<0x114, 0xf>(x));
  x = max(x, lanes_below<0x118, 0xf>(x));
  x = max(x, lanes_below<0x142, 0xa>(x));
  return max(x, lanes_below<0x143, 0xc>(x));
}
__device__ __forceinline__ int lanes_total(int x) {
  x += lanes_below<0x111, 0xf>(x);
  x += lanes_below<0x112, 0xf>(x);
  x += lanes_below<0x114, 0xf>(x);
  x += lanes_below<0x118, 0xf>(x);
  x += lanes_below<0x142, 0xa>(x);
  x += lanes_below<0x143, 0xc>(x);
  return __builtin_amdgcn_readlane(x, 63);
}

// Up to 64 sequences, one per lane: first token and the token behind the last one.
struct FewSequences {
  int start, end;
  __device__ __forceinline__ explicit FewSequences(const AttentionArgs& a) {
    const int lane = threadIdx.x & 63, tokens = static_cast<int>(a.tokens);
    const int top = min(max(a.offsets[0], 0), tokens);
    end = lane < a.sequences ? min(max(a.offsets[lane + 1], 0), tokens) : 0;
    end = max(lanes_max(end), top);   // an offset that falls counts as the largest before it
    const int before = __shfl_up(end, 1, 64);
    start = lane > 0 ? before : top;
  }
};

// Tile k of few sequences, the most work first: by its place in its sequence (`by_place`), or the
// longest sequence's tiles one after the other. False behind the last one. With causal the place
// is the work, and this order balances best. Queries of one sequence next to each other find its
// keys in L2, which is worth more from two rounds of two workgroups per CU on. Bfloat16, 8192 tokens,
// causal, by place and by sequence: dQ of 4000 workgroups 108 and 103 us, of 608 42 and 46; forward of
// 3000 87 and 76, of 608 30 and 34; dK and dV gain nowhere (1216: 83 and 98).
__device__ __forceinline__ bool tile_of_few(const AttentionArgs& a, int k, bool by_place, Place& p, int& t) {
  const FewSequences f(a);
  const int lane = threadIdx.x & 63, n = (f.end - f.start + kAttentionRows - 1) / kAttentionRows;
  if (k >= lanes_total(n)) return false;
  // the last class of work that, with those behind it, more than k tiles have; class x is the tiles at
  // place x, or all tiles of the sequences of x + 1 tiles
  auto from_class = [&](int x) { return lanes_total(by_place ? max(n - x, 0) : n > x ? n : 0); };
  int cls = 0, hi = __builtin_amdgcn_readlane(lanes_max(n), 63) - 1;
  while (cls < hi) {
    const int mid = (cls + hi + 1) >> 1;
    if (from_class(mid) > k) cls = mid;
    else hi = mid - 1;
  }
  int rank = k - from_class(cls + 1);
  t = cls;
  if (!by_place) {
    t = cls - rank % (cls + 1);
    rank /= cls + 1;
  }
  const bool in = by_place ? n > cls : n == cls + 1;
  const unsigned long long others = __ballot(in), pick = __ballot(in && __popcll(others & ((1ull << lane) - 1)) == rank);
  const int s = __builtin_ctzll(pick);
  const int start = __builtin_amdgcn_readlane(f.start, s);
  p.start = start;
  p.len = __builtin_amdgcn_readlane(f.end, s) - start;
  return true;
}

__device__ __forceinline__ Place place_of(const AttentionArgs& a, int heads, bool keys) {
  Place p;
  const uint32_t b = flat_block();
  uint32_t tile;
  if ((heads & 7) == 0) {
    const uint32_t per = heads >> 3, k = b >> 3;
    tile = k / per;
    p.head = static_cast<int>((b & 7) * per + k % per);
  } else {
    tile = b / heads;
    p.head = static_cast<int>(b % heads);
  }
  int t = 0;
  p.len = 0;
  p.start = p.row = 0;
  if (tile >= static_cast<uint32_t>(a.tiles)) return p;
  if (a.few) {
    if (!tile_of_few(a, static_cast<int>(tile), a.causal && (keys || static_cast<int64_t>(a.tiles) * heads < 1024), p, t)) return p;
  } else if (a.list != nullptr) {
    const int4 e = a.list[tile];
    p.start = e.x;
    p.len = e.y;
    t = e.z;
  } else {
    p.start = 0;
    p.len = static_cast<int>(a.tokens);
    t = a.tiles - 1 - static_cast<int>(tile);
  }
  // a query tile's work grows with its place, a key tile's shrinks
  p.row = (keys && p.len > 0 ? (p.len - 1) / kAttentionRows - t : t) * kAttentionRows;
  return p;
}

// The list, by one workgroup: prefix sums over the sequences' tiles, then the tiles by work. The first
// 1024 sequences stay in LDS, where bisection looks for a tile's; the sequences go to memory too,
// for the join and for bisection among more of them.
constexpr int kListThreads = 1024, kListWaves = kListThreads / 64, kListClasses = 256;

__global__ __launch_bounds__(kListThreads) void attention_list_kernel(AttentionArgs a) {
  __shared__ int wave_top[kListWaves], wave_sum[kListWaves];
  __shared__ int count[kListClasses];
  __shared__ int4 near[kListThreads];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int tokens = static_cast<int>(a.tokens);
  int top = min(max(a.offsets[0], 0), tokens), tiles = 0;   // of the sequences so far
  if (t < kListClasses) count[t] = 0;
  for (int s0 = 0; s0 < a.sequences; s0 += kListThreads) {
    const int s = s0 + t;
    const int waves = min(kListWaves, (a.sequences - s0 + 63) / 64);   // that have sequences
    // an offset that falls counts as the largest before it
    int end = s < a.sequences ? min(max(a.offsets[s + 1], 0), tokens) : 0;
    int incl = end;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl = max(incl, up);
    }
    if (lane == 63) wave_top[wave] = incl;
    __syncthreads();
    int before = top, all = top;
    for (int w = 0; w < waves; ++w) {
      if (w < wave) before = max(before, wave_top[w]);
      all = max(all, wave_top[w]);
    }
    end = max(incl, before);
    const int prev = __shfl_up(end, 1, 64);
    const int start = lane > 0 ? prev : before;
    const int n = s < a.sequences ? (end - start + kAttentionRows - 1) / kAttentionRows : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(sum, o, 64);
      if (lane >= o) sum += up;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int first = tiles + sum - n, total = tiles;
    for (int w = 0; w < waves; ++w) {
      if (w < wave) first += wave_sum[w];
      total += wave_sum[w];
    }
    if (s < a.sequences) {
      const int4 e{start, end - start, first, 0};
      a.sequence_list[s] = e;
      if (s0 == 0) near[t] = e;
    }
    top = all;
    tiles = total;
    __syncthreads();
  }
  __threadfence_block();
  __syncthreads();
  // each tile's sequence by bisection, its work in classes
  const bool few = a.sequences <= kListThreads;
  auto tile_of = [&](int x, int& cls) {
    int lo = 0, hi = a.sequences - 1;   // the last sequence that begins at or before tile x and has tiles
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((few ? near[mid].z : a.sequence_list[mid].z) <= x) lo = mid;
      else hi = mid - 1;
    }
    const int4 s = few ? near[lo] : a.sequence_list[lo];
    const int tile = x - s.z;
    const int64_t keys = a.causal ? min<int64_t>((tile + 1) * static_cast<int64_t>(kAttentionRows), a.window + kAttentionRows) : s.y;
    cls = kListClasses - 1 - static_cast<int>(min<int64_t>(kListClasses - 1, keys * kListClasses / (a.tokens + kAttentionRows)));
    return int4{s.x, s.y, tile, 0};
  };
  int4 own{};   // the thread's first tile
  int own_class = 0;
  for (int x = t; x < tiles; x += kListThreads) {
    int cls;
    const int4 e = tile_of(x, cls);
    if (x == t) {
      own = e;
      own_class = cls;
    }
    atomicAdd(&count[cls], 1);
  }
  __syncthreads();
  if (wave == 0) {   // where each class begins
    int base = 0;
    for (int c0 = 0; c0 < kListClasses; c0 += 64) {
      const int n = count[c0 + lane];
      int sum = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(sum, o, 64);
        if (lane >= o) sum += up;
      }
      count[c0 + lane] = base + sum - n;
      base += __shfl(sum, 63, 64);
    }
  }
  __syncthreads();
  // the order within a class does not matter: every tile has its own results
  for (int x = t; x < tiles; x += kListThreads) {
    int cls = own_class;
    int4 e = own;
    if (x != t) e = tile_of(x, cls);
    a.list[atomicAdd(&count[cls], 1)] = e;
  }
  for (int x = tiles + t; x < a.tiles; x += kListThreads) a.list[x] = int4{0, 0, 0, 0};
}

// Whether every row of [r0, r1] sees every key of [k0, k1].
__device__ __forceinline__ bool all_seen(const AttentionArgs& a, int len, int r0, int r1, int k0, int k1) {
  return k1 < len && (!a.causal || (k1 <= r0 && r1 - k0 < a.window));
}
// The keys that a row sees, or the rows that see a key: low .. low + span.
struct Sight {
  int low;
  uint32_t span;
  __device__ __forceinline__ bool operator()(int x) const { return static_cast<uint32_t>(x - low) <= span; }
};
__device__ __forceinline__ Sight sight_of_row(const AttentionArgs& a, int len, int row) {
  const int low = a.causal ? max(row - a.window + 1, 0) : 0, high = a.causal ? min(row, len - 1) : len - 1;
  return {low, static_cast<uint32_t>(max(high - low, 0))};   // rows behind the end: any key, so that no sum is empty
}
__device__ __forceinline__ Sight sight_of_key(const AttentionArgs& a, int key) {
  return {a.causal ? key : 0, a.causal ? static_cast<uint32_t>(a.window) - 1 : 0x7fffffffu};
}

// What the scheduler is asked for: MFMAS matrix instructions, each with the LDS reads of the one
// AHEAD places on, and with so many exponentials and other vector instructions behind it. A wave
// issues in order: what stands between matrix instructions runs while those do.
template <int MFMAS, int AHEAD, int READS, int EXPS, int OTHERS>
__device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * READS, 0);
#pragma unroll
  for (int i = 0; i < MFMAS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i + AHEAD < MFMAS) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if constexpr (EXPS > 0) __builtin_amdgcn_sched_group_barrier(0x400, EXPS, 0);
    if constexpr (OTHERS > 0) __builtin_amdgcn_sched_group_barrier(0x002, OTHERS, 0);
  }
}

// ---------------------------------------------------------------------------
// Forward: 128 queries per workgroup, keys and values in tiles of 64, two of each in LDS. The
// scores of tile t + 1 are formed while the exponentials of tile t are taken. The running
// maximum that exponents refer to follows the true one only when it is 2^8 behind: the
// exponentials stay below 2^8, and the sums are scaled again a few times per row at most.
// In fp16 they carry 2^7 more, up to 2^15 of the type's 2^16: without it each key with less than
// 2^-25 of a row's maximum would add nothing to the product, though thousands of them count.
// 8192 tokens, 32 query and 8 key heads of 128, causal, bfloat16: 508 us, 1080 TFLOP/s (a large library product
// 1309 on the same GPU). Power holds the clock at 1.73 GHz, where zeros run at 2.4 (381 us); at either the matrix
// units are busy in 56 to 57% of the cycles. Two tiles in LDS leave
// room for two workgroups per CU at dimension 128, which 248 registers allow too.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, 2) void attention_kernel(AttentionArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host's pass needs the kernel's name only
  using H = Half<T>;
  using TL = Tile<DP>;
  __shared__ __align__(1024) char smem[4 * TL::BYTES];   // keys, keys, values, values
  MUON_LDS char* lds = (MUON_LDS char*)smem;
  const Place p = place_of(a, a.heads, false);
  if (p.row >= p.len) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = p.head / a.group;
  const char* q = static_cast<const char*>(a.q.data) + (p.start * a.q.token_stride + p.head * a.q.head_stride) * 2;
  const char* k = static_cast<const char*>(a.k.data) + (p.start * a.k.token_stride + kv * a.k.head_stride) * 2;
  const char* v = static_cast<const char*>(a.v.data) + (p.start * a.v.token_stride + kv * a.v.head_stride) * 2;
  const int r0 = p.row + wave * kWaveRows, row = r0 + (lane & 31);
  // tiles that the workgroup's rows see, and how many of them are not behind the wave's rows
  const int last = min(p.row + kAttentionRows, p.len) - 1;
  const int begin = a.causal ? max(0, p.row - a.window + 1) / kStage : 0;
  const int tiles = (a.causal ? last : p.len - 1) / kStage + 1 - begin;
  const int own = r0 >= p.len ? 0 : a.causal ? min(tiles, (r0 + kWaveRows - 1) / kStage + 1 - begin) : tiles;
  TileLoads<DP, kWaves> lk, lv;
  lk.init(a.k.token_stride, a.dim);
  lv.init(a.v.token_stride, a.dim);
  auto issue_keys = [&](int t) {
    const int j = (begin + t) * kStage;
    lk.issue(k + static_cast<int64_t>(j) * lk.stride, p.len - j, lds + (t & 1) * TL::BYTES);
  };
  auto issue_values = [&](int t) {
    const int j = (begin + t) * kStage;
    lv.issue(v + static_cast<int64_t>(j) * lv.stride, p.len - j, lds + (2 + (t & 1)) * TL::BYTES);
  };
  issue_keys(0);
  typename H::v8 qf[TL::KS];
  load_rows<T, DP>(qf, q, row, row < p.len, a.q.token_stride, a.dim);
  const int ro = TL::row_offset(), co = TL::column_offset();
  const float c = a.scale * kLog2e;
  const Sight sight = sight_of_row(a, p.len, row);
  f32x16 acc[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) acc[b] = f32x16{};
  constexpr float UP = H::narrow ? 7.0f : 0.0f, DOWN = H::narrow ? 0x1p-7f : 1.0f;
  float m = -__builtin_huge_valf(), sum = 0.0f;   // the maximum that exponents refer to; this lane's part of the sum
  float top;                                      // the row's maximum in the tile whose exponentials come next

  auto scores = [&](f32x16 (&s)[2], MUON_LDS const char* kt) {
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      s[jb] = f32x16{};
#pragma unroll
      for (int ks = 0; ks < TL::KS; ++ks)
        s[jb] = H::mfma(row_part<T>(kt, (ro ^ (ks * 32)) + jb * 32 * TL::PITCH), qf[ks], s[jb]);
    }
  };
  auto mask = [&](f32x16 (&s)[2], int t) {
    const int j0 = (begin + t) * kStage;
    if (!all_seen(a, p.len, r0, r0 + kWaveRows - 1, j0, j0 + kStage - 1)) {
      asm volatile("");   // stays a branch
#pragma unroll
      for (int jb = 0; jb < 2; ++jb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          s[jb][e] = sight(j0 + jb * 32 + 8 * (e >> 2) + 4 * h + (e & 3)) ? s[jb][e] : -__builtin_huge_valf();
    }
  };
  auto largest = [&](const f32x16 (&s)[2]) {
    float x = s[0][0];
#pragma unroll
    for (int jb = 0; jb < 2; ++jb)
#pragma unroll
      for (int e = 0; e < 16; ++e) x = fmaxf(x, s[jb][e]);
    return twin_max(x);
  };
  // Tile t: the exponentials of its scores `s` and their product with the values; meanwhile, with
  // `more`, the scores of tile t + 1.
  auto step = [&](auto more, auto parity, int t, f32x16 (&s)[2], f32x16 (&next)[2]) {
    constexpr bool MORE = decltype(more)::value;
    MUON_LDS const char* kt = lds + (1 - decltype(parity)::value) * TL::BYTES;
    MUON_LDS const char* vt = lds + (2 + decltype(parity)::value) * TL::BYTES;
    if (__any((top - m) * c > 8.0f)) {   // also the first keys, after m = -inf
      const float to = fmaxf(m, top);
      const float keep = to == -__builtin_huge_valf() ? 1.0f : exp2f((m - to) * c);
      m = to;
      sum *= keep;
#pragma unroll
      for (int b = 0; b < TL::DB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[b][e] *= keep;
    }
    const float mc = m == -__builtin_huge_valf() ? 0.0f : fmaf(m, c, -UP);   // no key seen so far: every term is 0
    if constexpr (MORE) scores(next, kt);
    typename H::v8 w[4];
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[jb][e] = __builtin_amdgcn_exp2f(fmaf(s[jb][e], c, -mc));
        sum += s[jb][e];
      }
      w[2 * jb] = operand<T>(s[jb], 0);
      w[2 * jb + 1] = operand<T>(s[jb], 1);
    }
    if constexpr (MORE) {
      interleave<2 * TL::KS, 4, 1, 32 / (2 * TL::KS), 80 / (2 * TL::KS)>();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) asm volatile("" : "+v"(w[kk]));   // here, not behind the branch of the mask
      asm volatile("" : "+v"(sum));
      mask(next, t + 1);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int b = 0; b < TL::DB; ++b) acc[b] = H::mfma(column_part<T, DP>(vt, co, kk, b), w[kk], acc[b]);
    if constexpr (MORE) {
      top = largest(next);
      interleave<4 * TL::DB, 3, 2, 0, 1>();
    }
  };

  // Before step t tile t's values and tile t + 1's keys arrive; the places that they leave free
  // take the next ones.
  arrived();
  issue_values(0);
  if (tiles > 1) issue_keys(1);
  f32x16 s0[2], s1[2];
  if (own > 0) {
    scores(s0, lds);
    mask(s0, 0);
    top = largest(s0);
  }
  auto turn = [&](int t) {
    arrived();
    if (t + 1 < tiles) issue_values(t + 1);
    if (t + 2 < tiles) issue_keys(t + 2);
  };
  const std::integral_constant<int, 0> even{};
  const std::integral_constant<int, 1> odd{};
  int t = 0;
  for (; t + 2 < own; t += 2) {
    turn(t);
    step(std::true_type(), even, t, s0, s1);
    turn(t + 1);
    step(std::true_type(), odd, t + 1, s1, s0);
  }
  if (t + 1 < own) {
    turn(t);
    step(std::true_type(), even, t, s0, s1);
    turn(t + 1);
    step(std::false_type(), odd, t + 1, s1, s0);
    t += 2;
  } else if (t < own) {
    turn(t);
    step(std::false_type(), even, t, s0, s1);
    t += 1;
  }
  for (; t < tiles; ++t) turn(t);   // the other waves' tiles
  sum = twin_sum(sum);
  if (a.lse_out != nullptr && h == 0 && row < p.len) {
    // the exponents' reference was rounded: what a score of m had for an exponent beyond UP is in the sum
    const float off = fmaf(m, c, -fmaf(m, c, -UP)) - UP;
    a.lse_out[p.head * a.tokens + p.start + row] = m * a.scale + fmaf(off, -kLn2, logf(sum * DOWN));
  }
  arrived();   // the tiles are read: their place takes the results
  char* o = static_cast<char*>(a.o.data) + (p.start * a.o.token_stride + p.head * a.o.head_stride) * 2;
  store_rows<T, DP>(acc, 1.0f / sum, lds + wave * kWaveRows * TL::PITCH, o, r0, p.len, a.o.token_stride, a.dim);
#endif
}

// ---------------------------------------------------------------------------
// Gradient.

// Score gradients in fp16 would leave its range at either end: they carry a power of two per
// column, found from the first ones and lowered when they grow, which the column's sums
// carry too. bf16 has fp32's range and needs none.
template <typename T> struct ColumnScale {
  float up = 1.0f, down = 1.0f;
  bool set = !Half<T>::narrow;
  template <int N>
  __device__ __forceinline__ void apply(f32x16& x, f32x16 (&acc)[N]) {
    if constexpr (Half<T>::narrow) {
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
      if (__any(set ? top * up > 32768.0f : top > 0.0f)) {
        top = twin_max(top);
        if (top > 0.0f && (!set || top * up > 32768.0f)) {
          // the largest goes to 2^10 .. 2^11
          const int e = min(max(127 + 10 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 1), 253);
          const float to = __uint_as_float(static_cast<uint32_t>(e) << 23);
          const float ratio = set ? to * down : 1.0f;
          up = to;
          down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
          set = true;
#pragma unroll
          for (int b = 0; b < N; ++b)
#pragma unroll
            for (int e2 = 0; e2 < 16; ++e2) acc[b][e2] *= ratio;
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= up;
    }
  }
};

// dQ: 128 queries per workgroup, keys and values in tiles of 64. Each row's delta and log-sum-exp in
// units of log 2 are formed on the way, for dK and dV. Three products per pair: 713 us for the forward
// kernel's case (1160 TFLOP/s; power, at 1.72 GHz, matrix units busy 61%); 150 to 158 for 12 texts of 8191 tokens, 32
// heads of 128: 417 MB that L2 misses, 68 us as reads, and matrix units busy 27%, with 6 key tiles
// per workgroup to hide one behind the other.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, 2) void attention_dq_kernel(AttentionArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host's pass needs the kernel's name only
  using H = Half<T>;
  using TL = Tile<DP>;
  __shared__ __align__(1024) char smem[4 * TL::BYTES];
  MUON_LDS char* lds = (MUON_LDS char*)smem;
  const Place p = place_of(a, a.heads, false);
  if (p.row >= p.len) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = p.head / a.group;
  const char* q = static_cast<const char*>(a.q.data) + (p.start * a.q.token_stride + p.head * a.q.head_stride) * 2;
  const char* g = static_cast<const char*>(a.d_o.data) + (p.start * a.d_o.token_stride + p.head * a.d_o.head_stride) * 2;
  const char* k = static_cast<const char*>(a.k.data) + (p.start * a.k.token_stride + kv * a.k.head_stride) * 2;
  const char* v = static_cast<const char*>(a.v.data) + (p.start * a.v.token_stride + kv * a.v.head_stride) * 2;
  const int r0 = p.row + wave * kWaveRows, row = r0 + (lane & 31);
  typename H::v8 qf[TL::KS], gf[TL::KS];
  load_rows<T, DP>(qf, q, row, row < p.len, a.q.token_stride, a.dim);
  load_rows<T, DP>(gf, g, row, row < p.len, a.d_o.token_stride, a.dim);
  const int64_t stat = p.head * a.tokens + p.start + min(row, p.len - 1);
  const float lse2 = a.lse[stat] * kLog2e;
  float delta = 0.0f;
  {
    typename H::v8 of[TL::KS];
    load_rows<T, DP>(of, static_cast<const char*>(a.o.data) + (p.start * a.o.token_stride + p.head * a.o.head_stride) * 2, row,
                     row < p.len, a.o.token_stride, a.dim);
#pragma unroll
    for (int ks = 0; ks < TL::KS; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf(static_cast<float>(gf[ks][e]), static_cast<float>(of[ks][e]), delta);
  }
  delta = twin_sum(delta);
  if (h == 0 && row < p.len) {
    a.lse2[stat] = lse2;
    a.delta[stat] = delta;
  }

  const int last = min(p.row + kAttentionRows, p.len) - 1;
  const int begin = a.causal ? max(0, p.row - a.window + 1) / kStage : 0;
  const int end = (a.causal ? last : p.len - 1) / kStage + 1;
  TileLoads<DP, kWaves> lk, lv;
  lk.init(a.k.token_stride, a.dim);
  lv.init(a.v.token_stride, a.dim);
  auto issue = [&](int t, int buf) {
    const int j = t * kStage;
    lk.issue(k + static_cast<int64_t>(j) * lk.stride, p.len - j, lds + buf * 2 * TL::BYTES);
    lv.issue(v + static_cast<int64_t>(j) * lv.stride, p.len - j, lds + (buf * 2 + 1) * TL::BYTES);
  };
  const int ro = TL::row_offset(), co = TL::column_offset();
  const float c = a.scale * kLog2e;
  const Sight sight = sight_of_row(a, p.len, row);
  f32x16 acc[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[b][e] = 0.0f;
  ColumnScale<T> cs;

  auto step = [&](bool masked, int buf, int j0) {
    MUON_LDS const char* kt = lds;
    MUON_LDS const char* vt = kt + TL::BYTES;
    // places in LDS with the tile's in them, made anew for each tile (registers)
    int rk = ro + buf * 2 * TL::BYTES, ck = co + buf * 2 * TL::BYTES;
    asm volatile("" : "+v"(rk), "+v"(ck));
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      f32x16 s = {}, d = {};
#pragma unroll
      for (int ks = 0; ks < TL::KS; ++ks) {
        s = H::mfma(row_part<T>(kt, (rk ^ (ks * 32)) + jb * 32 * TL::PITCH), qf[ks], s);
        d = H::mfma(row_part<T>(vt, (rk ^ (ks * 32)) + jb * 32 * TL::PITCH), gf[ks], d);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lse2)) * (d[e] - delta);
      if (masked) {
        asm volatile("");   // stays a branch
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = sight(j0 + jb * 32 + 8 * (e >> 2) + 4 * h + (e & 3)) ? s[e] : 0.0f;
      }
      cs.apply(s, acc);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const auto w = operand<T>(s, kk);
#pragma unroll
        for (int b = 0; b < TL::DB; ++b) acc[b] = H::mfma(column_part<T, DP>(kt, ck, jb * 2 + kk, b), w, acc[b]);
      }
    }
  };

  issue(begin, begin & 1);
  for (int t = begin; t < end; ++t) {
    arrived();
    if (t + 1 < end) issue(t + 1, (t + 1) & 1);
    const int j0 = t * kStage;
    if (r0 >= p.len || (a.causal && (j0 > r0 + kWaveRows - 1 || j0 + kStage - 1 <= r0 - a.window))) continue;
    step(!all_seen(a, p.len, r0, r0 + kWaveRows - 1, j0, j0 + kStage - 1), t & 1, j0);
  }
  arrived();
  char* o = static_cast<char*>(a.dq.data) + (p.start * a.dq.token_stride + p.head * a.dq.head_stride) * 2;
  store_rows<T, DP>(acc, a.scale * cs.down, lds + wave * kWaveRows * TL::PITCH, o, r0, p.len, a.dq.token_stride, a.dim);
#endif
}

// dK and dV: 128 keys per workgroup, the queries of all heads of the group in tiles. The keys' rows
// stay in registers, the values' in LDS, where the registers end.
// With HALVES = 1 four waves own 32 keys each and take tiles of 32 rows: two workgroups fit a CU, and
// one's exponentials, first loads and results pass behind the other's products. With HALVES = 2 two
// waves share 32 keys, each with half of a tile of 64 rows and sums of its own, joined at the end:
// one workgroup per CU that is done in half the time, for fewer workgroups than two per CU fill
// evenly (with causal the longest take twice the average). Bfloat16, dimension 128: 2432 workgroups 219 us
// with 2, 173 with 1; 512 of them 83 us with 2, 110 with 1. The forward kernel's case: 1066 us (1030 TFLOP/s).
// Where there are fewer still, a key tile's queries are cut into parts, whose sums
// attention_join_kernel adds in order (8 workgroups of 1000 tokens: 216 us, in parts 33).
// Rows behind the sequence arrive as zeros (Q, dO, delta and the log-sum-exp), and add nothing.
template <typename T, int DP, int HALVES>
__global__ __launch_bounds__(kThreads * HALVES, 2) void attention_dkv_kernel(AttentionArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host's pass needs the kernel's name only
  using H = Half<T>;
  using TL = Tile<DP>;
  constexpr int ROWS = kWaveRows * HALVES, WAVES = kWaves * HALVES;
  constexpr int BYTES = ROWS * TL::PITCH;
  constexpr int BUF = 2 * BYTES + 512;                     // Q, dO, then log-sum-exp and delta of the rows
  constexpr int VALUES = kAttentionRows * TL::PITCH;
  constexpr int PART = TL::DB * 16 * 256;                  // a wave's sums
  constexpr int USED = VALUES + 2 * BUF, JOINED = HALVES == 2 ? WAVES * PART : 0;
  __shared__ __align__(1024) char smem[USED > JOINED ? USED : JOINED];
  MUON_LDS char* values = (MUON_LDS char*)smem;
  MUON_LDS char* lds = values + VALUES;
  Place p = place_of(a, a.kv_heads * a.parts, true);
  if (p.row >= p.len) return;
  const int part = p.head % a.parts;
  p.head /= a.parts;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = wave % kWaves, half = wave / kWaves;
  const char* k = static_cast<const char*>(a.k.data) + (p.start * a.k.token_stride + p.head * a.k.head_stride) * 2;
  const char* v = static_cast<const char*>(a.v.data) + (p.start * a.v.token_stride + p.head * a.v.head_stride) * 2;
  const int k0 = p.row + kg * kWaveRows, key = k0 + (lane & 31);

  const int last = min(p.row + kAttentionRows, p.len) - 1;   // key of the workgroup
  const int begin = a.causal ? p.row / ROWS : 0;
  const int rows_end = a.causal && a.window < p.len - last ? last + a.window : p.len;   // rows before it see a key
  const int tiles = (rows_end - 1) / ROWS + 1 - begin;
  TileLoads<DP, WAVES, ROWS> lq, lg;
  lq.init(a.q.token_stride, a.dim);
  lg.init(a.d_o.token_stride, a.dim);
  // tile `t` of head `hq`
  auto issue = [&](int hq, int t, int buf) {
    const int i = (begin + t) * ROWS, rows = p.len - i;
    MUON_LDS char* to = lds + buf * BUF;
    lq.issue(static_cast<const char*>(a.q.data) + ((p.start + i) * a.q.token_stride + hq * a.q.head_stride) * 2, rows, to);
    lg.issue(static_cast<const char*>(a.d_o.data) + ((p.start + i) * a.d_o.token_stride + hq * a.d_o.head_stride) * 2, rows,
             to + BYTES);
    if (wave < 2) {
      const float* from = (wave == 0 ? a.lse2 : a.delta) + hq * a.tokens + p.start + i;
      const auto rsrc = MUON_HEAD_RSRC(reinterpret_cast<const char*>(from), min(rows, ROWS) * 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MUON_LDS void*)(to + 2 * BYTES + wave * 256), 4, lane * 4, 0, 0, 0);
    }
  };
  {
    TileLoads<DP, WAVES, ROWS> lv;
    lv.init(a.v.token_stride, a.dim);
#pragma unroll
    for (int i = 0; i < kAttentionRows / ROWS; ++i) {
      const int j = p.row + i * ROWS;
      lv.issue(v + static_cast<int64_t>(j) * lv.stride, p.len - j, values + i * BYTES);
    }
  }
  // tiles of all heads, one head after the other; this part's
  const int64_t all = static_cast<int64_t>(tiles) * a.group;
  const int from = static_cast<int>(all * part / a.parts), to = static_cast<int>(all * (part + 1) / a.parts);
  int hq = p.head * a.group + from / tiles, ahead = from % tiles;   // of the tile that is loaded next
  auto next = [&](int buf) {
    issue(hq, ahead, buf);
    if (++ahead == tiles) {
      ahead = 0;
      ++hq;
    }
  };
  if (from < to) next(from & 1);
  typename H::v8 kf[TL::KS];
  load_rows<T, DP>(kf, k, key, key < p.len, a.k.token_stride, a.dim);
  const int ro = TL::row_offset(), co = TL::column_offset();
  const float c = a.scale * kLog2e;
  // probabilities in fp16 carry 2^14, so that small ones keep their bits; they are 1 at most, but for the
  // rounding of the log-sum-exp, and the type ends at 4
  constexpr float PUP = H::narrow ? 16384.0f : 1.0f;
  const Sight sight = sight_of_key(a, key);
  f32x16 dk[TL::DB], dv[TL::DB];
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) dk[b] = dv[b] = f32x16{};
  ColumnScale<T> cs;

  auto step = [&](bool masked, int buf, int i0) {
    MUON_LDS const char* qt = lds;
    MUON_LDS const char* gt = qt + BYTES;
    MUON_LDS const char* st = lds + buf * BUF + 2 * BYTES + half * kWaveRows * 4 + h * 16;
    // places in LDS with the tile's in them, made anew for each tile: kept from tile to tile, those
    // of all steps would fill the registers
    int rq = ro + buf * BUF + half * kWaveRows * TL::PITCH, cq = co + buf * BUF + half * kWaveRows * TL::PITCH;
    int rv = ro + kg * kWaveRows * TL::PITCH;
    asm volatile("" : "+v"(rq), "+v"(cq), "+v"(rv));
    f32x16 s = {}, d = {};
#pragma unroll
    for (int ks = 0; ks < TL::KS; ++ks) {
      s = H::mfma(row_part<T>(qt, rq ^ (ks * 32)), kf[ks], s);
      d = H::mfma(row_part<T>(gt, rq ^ (ks * 32)), row_part<T>(values, rv ^ (ks * 32)), d);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const f32x4 l = *reinterpret_cast<MUON_LDS const f32x4*>(st + u * 32);
      const f32x4 x = *reinterpret_cast<MUON_LDS const f32x4*>(st + 256 + u * 32);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = __builtin_amdgcn_exp2f(fmaf(s[4 * u + e], c, -l[e]));
        d[4 * u + e] = w * (d[4 * u + e] - x[e]);
        s[4 * u + e] = H::narrow ? w * PUP : w;
      }
    }
    if (masked) {
      asm volatile("");   // stays a branch
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const bool in = sight(i0 + 8 * (e >> 2) + 4 * h + (e & 3));
        s[e] = in ? s[e] : 0.0f;
        d[e] = in ? d[e] : 0.0f;
      }
    }
    cs.apply(d, dk);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const auto wp = operand<T>(s, kk), wd = operand<T>(d, kk);
#pragma unroll
      for (int b = 0; b < TL::DB; ++b) {
        dv[b] = H::mfma(column_part<T, DP>(gt, cq, kk, b), wp, dv[b]);
        dk[b] = H::mfma(column_part<T, DP>(qt, cq, kk, b), wd, dk[b]);
      }
    }
  };

  int now = from % tiles;   // the present tile of its head
  for (int n = from; n < to; ++n) {
    arrived();
    if (n + 1 < to) next((n + 1) & 1);
    const int i0 = (begin + now) * ROWS + half * kWaveRows;
    if (++now == tiles) now = 0;
    if (k0 >= p.len || i0 >= p.len || (a.causal && (i0 + kWaveRows - 1 < k0 || i0 - (k0 + kWaveRows - 1) >= a.window))) continue;
    step(!all_seen(a, 0x7fffffff, i0, i0 + kWaveRows - 1, k0, k0 + kWaveRows - 1), n & 1, i0);
  }
  const float xk = a.scale * cs.down, xv = 1.0f / PUP;
#pragma unroll
  for (int b = 0; b < TL::DB; ++b) {
    dk[b] *= xk;
    dv[b] *= xv;
  }
  arrived();   // the tiles are read: their place takes the results
  if constexpr (HALVES == 2) {
    // a pair of waves: the first one joins dK, the second one dV (in dk)
    MUON_LDS float* mine = (MUON_LDS float*)(values + (kg * 2 + half) * PART) + lane;
#pragma unroll
    for (int b = 0; b < TL::DB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) mine[(b * 16 + e) * 64] = half == 0 ? dv[b][e] : dk[b][e];
    __syncthreads();
    const MUON_LDS float* other = (const MUON_LDS float*)(values + (kg * 2 + 1 - half) * PART) + lane;
#pragma unroll
    for (int b = 0; b < TL::DB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) dk[b][e] = (half == 0 ? dk[b][e] : dv[b][e]) + other[(b * 16 + e) * 64];
    __syncthreads();
  }
  // dK (which = 0) or dV of the wave's keys
  auto store = [&](const f32x16(&x)[TL::DB], int which) {
    if (a.parts > 1) {
      if (key >= p.len) return;
      const int64_t row = static_cast<int64_t>(part * 2 + which) * a.tokens + p.start + key;
      float* to = a.partial + (row * a.kv_heads + p.head) * a.dim;
#pragma unroll
      for (int b = 0; b < TL::DB; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int at = b * 32 + g * 8 + h * 4;
          if (at < a.dim) *reinterpret_cast<f32x4*>(to + at) = f32x4{x[b][4 * g], x[b][4 * g + 1], x[b][4 * g + 2], x[b][4 * g + 3]};
        }
    } else {
      const HeadsArg& out = which == 0 ? a.dk : a.dv;
      store_rows<T, DP>(x, 1.0f, values + wave * kWaveRows * TL::PITCH,
                        static_cast<char*>(out.data) + (p.start * out.token_stride + p.head * out.head_stride) * 2, k0, p.len,
                        out.token_stride, a.dim);
    }
  };
  if constexpr (HALVES == 2) {
    store(dk, half);
  } else {
    store(dk, 0);
    store(dv, 1);
  }
#endif
}

// The parts' sums in order, eight columns per thread. The sequences' tokens are one range.
template <int DT>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
  const int per = a.dim / 8;
  const int64_t n = a.tokens * a.kv_heads * per, item = static_cast<int64_t>(flat_block()) * 256 + threadIdx.x;
  int64_t first = 0, end = a.tokens;
  if (a.few) {
    const FewSequences f(a);
    first = __builtin_amdgcn_readlane(f.start, 0);
    end = __builtin_amdgcn_readlane(f.end, 63);
  } else if (a.list != nullptr) {
    const int4 last = a.sequence_list[a.sequences - 1];
    first = a.sequence_list[0].x;
    end = last.x + last.y;
  }
  if (item >= 2 * n) return;
  const HeadsArg& out = item < n ? a.dk : a.dv;
  const int64_t at = item < n ? item : item - n;
  const int c = static_cast<int>(at % per) * 8, head = static_cast<int>(at / per % a.kv_heads);
  const int64_t token = at / per / a.kv_heads;
  if (token < first || token >= end) return;
  float v[8] = {};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) {
    float x[8];
    read8<MUON_DTYPE_F32>(a.partial, 8 * (2 * p * n + item), 8, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += x[e];
  }
  write8<DT>(out.data, token * out.token_stride + head * out.head_stride + c, 8, v);
}

// ---------------------------------------------------------------------------

// Kernels for heads of up to 32, 64, 96 and 128 columns (8192 tokens, 16 heads, causal, bfloat16, forward and
// gradient: dimension 32 143 and 406 us, 165 and 511 by the one for 64; 96 228 and 735, 257 and 845 by the one for 128).
template <typename F>
static hipError_t with_dim(const AttentionArgs& a, F&& f) {
  auto of = [&](auto type) {
    if (a.dim <= 32) f(type, std::integral_constant<int, 32>());
    else if (a.dim <= 64) f(type, std::integral_constant<int, 64>());
    else if (a.dim <= 96) f(type, std::integral_constant<int, 96>());
    else f(type, std::integral_constant<int, 128>());
    return hipGetLastError();
  };
  return a.dtype == MUON_DTYPE_BF16 ? of(static_cast<__bf16>(0.0f)) : of(static_cast<_Float16>(0.0f));
}

hipError_t launch_attention_list(const AttentionArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(attention_list_kernel, dim3(1), dim3(kListThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s) {
  return with_dim(a, [&](auto type, auto dim) {
    hipLaunchKernelGGL((attention_kernel<decltype(type), decltype(dim)::value>), flat_grid(static_cast<int64_t>(a.tiles) * a.heads),
                       dim3(kThreads), 0, s, a);
  });
}
hipError_t launch_attention_dq(const AttentionArgs& a, hipStream_t s) {
  return with_dim(a, [&](auto type, auto dim) {
    hipLaunchKernelGGL((attention_dq_kernel<decltype(type), decltype(dim)::value>),
                       flat_grid(static_cast<int64_t>(a.tiles) * a.heads), dim3(kThreads), 0, s, a);
  });
}
template <int HALVES>
static hipError_t launch_dkv(const AttentionArgs& a, hipStream_t s) {
  return with_dim(a, [&](auto type, auto dim) {
    hipLaunchKernelGGL((attention_dkv_kernel<decltype(type), decltype(dim)::value, HALVES>),
                       flat_grid(static_cast<int64_t>(a.tiles) * a.kv_heads * a.parts), dim3(kThreads * HALVES), 0, s, a);
  });
}
hipError_t launch_attention_dkv(const AttentionArgs& a, hipStream_t s) {
  return a.halves == 2 ? launch_dkv<2>(a, s) : launch_dkv<1>(a, s);
}
hipError_t launch_attention_join(const AttentionArgs& a, hipStream_t s) {
  const dim3 grid = flat_grid((a.tokens * a.kv_heads * (a.dim / 8) * 2 + 255) / 256);
  if (a.dtype == MUON_DTYPE_BF16) hipLaunchKernelGGL((attention_join_kernel<MUON_DTYPE_BF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attention_join_kernel<MUON_DTYPE_F16>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// How dK and dV are shared out, by the number of key tiles (see the kernel): from 1024 on HALVES = 1,
// below 2; parts where there are fewer than 256, one CU each, as many as give 512 workgroups, with
// at least 512 rows to a part.
void plan_attention_dkv(AttentionArgs& a) {
  const int64_t groups = std::max<int64_t>(1, static_cast<int64_t>(a.tiles) * a.kv_heads);
  a.halves = groups >= 1024 ? 1 : 2;
  a.parts = 1;
  if (groups < 256)
    a.parts = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({32, (512 + groups - 1) / groups, a.tokens * a.group / 512})));
}

}  // namespace muon
