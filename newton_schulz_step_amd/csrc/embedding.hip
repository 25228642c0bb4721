// Embedding lookup and its gradient by sorted tokens (gfx950).
//
//   y[t] = scale table[id_t];   dtable[v] (+)= scale sum over t with id_t = v of dy[t]
// The gradient sorts the tokens by id (stable, so a row's tokens keep their order), sums
// chunks of 32 or 8 sorted tokens, and joins the sums of rows whose tokens span several chunks:
// a fixed order of sums without floating-point atomics, however often a token occurs.
// Bound by memory: dy once, the table's rows once. 16384 tokens, 32000 x 4096 fp32, every row written:
// 150 us (4.4 TB/s; a large copy reaches 5.1), of which the sort 20.
#include <algorithm>

#include "fp8.hpp"
#include "layer.hpp"
#include "quant8.hpp"
#include "rows.hpp"

namespace muon {

// The row of a slot; `vocab` for an id that is none.
__device__ __forceinline__ int token_row(const EmbeddingArgs& a, int64_t i) {
  const int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return static_cast<int>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// A wave takes 2048 columns of a token.
constexpr int kEmbeddingCols = 2048;

template <int TT, int YT>
__global__ __launch_bounds__(256) void embedding_kernel(EmbeddingArgs a, int tiles) {
  const int lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(flat_block()) * 4 + (threadIdx.x >> 6);
  const int64_t t = item / tiles;
  if (t >= a.tokens) return;
  const int64_t c0 = (item - t * tiles) * kEmbeddingCols + lane * 8;
  const int row = __builtin_amdgcn_readfirstlane(token_row(a, t));
  const bool there = row < a.vocab;
  Raw8<TT> x[4];
  Eight c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = Eight(c0 + i * 512, a.cols);
    x[i].load(a.table, there ? row * a.ld_table + c[i].at : 0, there ? c[i].n : 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = there ? x[i].get(e) * a.scale : 0.0f;
    write_own<YT>(a.y, t * a.ld_y, c[i], v);
  }
}

// ---------------------------------------------------------------------------
// The sort: least significant digit first, up to 8 bits per pass, stable. A pass counts each
// block's slots per digit, then every block sums the counts of all blocks (where a digit
// starts) and of those before it, and places its slots in order, 64 of a wave at a time,
// ranked with ballots. Few tokens take one block and one launch for all passes.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int64_t kSortBlock = 1024;    // slots of a block, unless that makes too many blocks (2048: 1.7 us more per pass)
constexpr int32_t kSortBlocks = 256;

int32_t sort_blocks(int64_t n) {
  if (n <= 4 * kSortBlock) return 1;
  return static_cast<int32_t>(std::min<int64_t>((n + kSortBlock - 1) / kSortBlock, kSortBlocks));
}

// The first pass reads the ids themselves, pass p > 0 what p - 1 left in buffer (p - 1) % 2.
__device__ __forceinline__ int sort_key(const EmbeddingArgs& a, int pass, int64_t i) {
  return pass == 0 ? token_row(a, i) : a.keys[(pass - 1) & 1][i];
}
__device__ __forceinline__ int sort_slot(const EmbeddingArgs& a, int pass, int64_t i) {
  return pass == 0 ? static_cast<int>(i) : a.slots[(pass - 1) & 1][i];
}

__device__ __forceinline__ void clear_touched(const EmbeddingArgs& a, int block, int blocks) {
  if (a.touched == nullptr) return;
  const int64_t words = (a.vocab + 3) / 4;
  uint32_t* p = reinterpret_cast<uint32_t*>(a.touched);
  for (int64_t i = static_cast<int64_t>(block) * kSortThreads + threadIdx.x; i < words;
       i += static_cast<int64_t>(blocks) * kSortThreads)
    p[i] = 0;
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(EmbeddingArgs a, int pass) {
  __shared__ int h[kSortBins];
  if (threadIdx.x < kSortBins) h[threadIdx.x] = 0;
  if (pass == 0) clear_touched(a, blockIdx.x, a.blocks);
  __syncthreads();
  const int shift = pass * a.bits, mask = (1 << a.bits) - 1;
  const int64_t lo = blockIdx.x * a.per_block, hi = min(a.tokens, lo + a.per_block);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&h[(sort_key(a, pass, i) >> shift) & mask], 1);
  __syncthreads();
  if (threadIdx.x < kSortBins) a.hist[blockIdx.x * kSortBins + threadIdx.x] = h[threadIdx.x];
}

struct SortShared {
  int next[kSortWaves][kSortBins];   // next place of each digit, per wave
  int total[kSortBins], earlier[kSortBins];
  int scan[kSortBins / 64];
};

__device__ __forceinline__ void sort_place(const EmbeddingArgs& a, int pass, SortShared& sh, int block, int blocks) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int shift = pass * a.bits, mask = (1 << a.bits) - 1;
  const int64_t lo = block * a.per_block, hi = min(a.tokens, lo + a.per_block);
  // each wave places a contiguous part of the block's slots
  const int64_t part = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t wlo = min(hi, lo + wave * part), whi = min(hi, wlo + part);
  for (int i = t; i < kSortWaves * kSortBins; i += kSortThreads) (&sh.next[0][0])[i] = 0;
  if (t < kSortBins) sh.total[t] = sh.earlier[t] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 64) atomicAdd(&sh.next[wave][(sort_key(a, pass, i) >> shift) & mask], 1);
  if (blocks > 1) {
    const int bin = t % kSortBins;
    int all = 0, before = 0;
#pragma unroll 4
    for (int b = t / kSortBins; b < blocks; b += kSortThreads / kSortBins) {
      const int c = a.hist[b * kSortBins + bin];
      before += b < block ? c : 0;
      all += c;
    }
    atomicAdd(&sh.total[bin], all);
    atomicAdd(&sh.earlier[bin], before);
  }
  __syncthreads();
  int incl = 0, n = 0;
  if (t < kSortBins) {
    int before = sh.earlier[t];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = sh.next[w][t];
      sh.next[w][t] = before;
      before += c;
    }
    n = blocks > 1 ? sh.total[t] : before;
    incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    if (lane == 63) sh.scan[wave] = incl;
  }
  __syncthreads();
  if (t < kSortBins) {
    int first = incl - n;
    for (int w = 0; w < wave; ++w) first += sh.scan[w];
    for (int w = 0; w < kSortWaves; ++w) sh.next[w][t] += first;
  }
  __syncthreads();
  int* keys = a.keys[pass & 1];
  int* slots = a.slots[pass & 1];
  for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool in = i < whi;
    const int key = in ? sort_key(a, pass, i) : 0, slot = in ? sort_slot(a, pass, i) : 0;
    const int d = (key >> shift) & mask;
    unsigned long long same = __ballot(in);
    for (int bit = 0; bit < a.bits; ++bit) {
      const unsigned long long m = __ballot((d >> bit) & 1);
      same &= ((d >> bit) & 1) ? m : ~m;
    }
    int to = 0;
    if (in) {
      to = sh.next[wave][d] + __popcll(same & ((1ull << lane) - 1));
      keys[to] = key;
      slots[to] = slot;
      if (pass == 0 && a.touched != nullptr && key < a.vocab) a.touched[key] = 1;   // the same byte from every slot of a row
    }
    __builtin_amdgcn_wave_barrier();
    if (in && (same >> lane) == 1ull) sh.next[wave][d] = to + 1;   // the last of its digit
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(EmbeddingArgs a, int pass) {
  __shared__ SortShared sh;
  sort_place(a, pass, sh, blockIdx.x, a.blocks);
}

__global__ __launch_bounds__(kSortThreads) void sort_all_kernel(EmbeddingArgs a) {
  __shared__ SortShared sh;
  clear_touched(a, 0, 1);
  for (int pass = 0; pass < a.passes; ++pass) {
    sort_place(a, pass, sh, 0, 1);
    __threadfence_block();
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Sums. A wave takes a chunk of sorted tokens and 512 columns. A row whose tokens lie in one chunk is
// finished there. A chunk leaves the sum of a row that began before it in its first partial row,
// and that of one that begins in it and goes on in the second; the next launch joins them, and
// clears the rows without a token where every row of the table is written. Chunks of 32; of 8 for few
// tokens, whose waves would be too few to keep the memory busy, while with many tokens the rows of
// frequent ones span so many chunks that joining them costs more. The narrower the rows, the more tokens
// it takes: whole calls in us with chunks of 8 and of 32, added to an fp32 table, 8192 x 1024 41 and 49, 12000 x
// 1024 48 and 52, 8192 x 2048 48 and 52, 12000 x 2048 63 and 59, 5000 x 2560 40 and 49, 4200 x 4096 46 and 52, 8192 x
// 4096 68 and 61, 3000 x 8192 50 and 53, 5000 x 8192 73 and 68, 2000 x 11008 45 and 53, 4096 x 11008 79 and
// 74; into every row of 32000, 8192 x 2048 77 and 82, 4096 x 4096 128 and 134, 12000 x 4096 145 and 143. One limit for
// all rows of more than 2048 columns stands in their middle: it leaves up to 20% at 2560 columns, 14% at 4096, 7% at 11008.
struct SumArgs {
  EmbeddingArgs e;
  const int* keys;
  const int* slots;
  int64_t chunks, tiles;
  int64_t joins;   // waves that join
};

template <int WT>
__device__ __forceinline__ void finish_row(const EmbeddingArgs& a, int64_t row, const Eight& c, const float (&sum)[8]) {
  float v[8];
  const int64_t at = row * a.ld_table;
  if (a.accumulate) read8<WT>(a.dtable, at + c.at, c.n, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (a.accumulate ? v[e] : 0.0f) + a.scale * sum[e];
  write_own<WT>(a.dtable, at, c, v);
}

template <int DT, int WT, int CHUNK>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs s) {
  constexpr int AHEAD = 8;
  const EmbeddingArgs& a = s.e;
  const int lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(flat_block()) * 4 + (threadIdx.x >> 6);
  if (item >= s.chunks * s.tiles) return;
  const int64_t chunk = item / s.tiles;
  const Eight c((item - chunk * s.tiles) * 512 + lane * 8, a.cols);
  const int64_t first = chunk * CHUNK;
  const int count = static_cast<int>(min<int64_t>(CHUNK, a.tokens - first));
  // keys of the chunk in lanes 0 .. count - 1, those around it for the runs that leave it
  const int none = static_cast<int>(a.vocab);
  const int key = lane < count ? s.keys[first + lane] : none;
  const int slot = lane < count ? s.slots[first + lane] : 0;
  const int before = first > 0 ? s.keys[first - 1] : none;
  const int after = first + count < a.tokens ? s.keys[first + count] : none;
  float sum[8] = {};
  bool began = before != __builtin_amdgcn_readlane(key, 0);   // whether the present row begins in this chunk
  for (int j0 = 0; j0 < count; j0 += AHEAD) {
    Raw8<DT> x[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = __builtin_amdgcn_readlane(key, j0 + j);   // lanes behind the end hold no row
      const int64_t t = __builtin_amdgcn_readlane(slot, j0 + j);
      x[j].load_once(a.dy, k < none ? t * a.ld_y + c.at : 0, k < none ? c.n : 0);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = __builtin_amdgcn_readlane(key, j0 + j);
      if (k >= none) continue;   // the ids that are no rows come last
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += x[j].get(e);
      const bool at_end = j0 + j == count - 1;
      const int next = at_end ? after : __builtin_amdgcn_readlane(key, (j0 + j + 1) & 63);
      if (next == k && !at_end) continue;
      if (began && next != k) finish_row<WT>(a, k, c, sum);
      else write_own<MUON_DTYPE_F32>(a.partial, (2 * chunk + (began ? 1 : 0)) * a.cols, c, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
      began = true;
    }
  }
}

// Zeros into `n` elements at element i by one wave, 16 neighbouring bytes per lane where they are
// aligned, past the caches: left in them, they delay the next call's reads until they are written
// back (16384 tokens, 32000 x 4096 fp32: 165 us through the caches, 155 past them).
template <int WT>
__device__ __forceinline__ void clear_row(void* p, int64_t i, int64_t n) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  constexpr int SIZE = WT == MUON_DTYPE_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  char* to = static_cast<char*>(p) + i * SIZE;
  const int64_t bytes = n * SIZE;
  if (((reinterpret_cast<uintptr_t>(to) | bytes) & 15) == 0) {
    for (int64_t at = lane * 16; at < bytes; at += 1024)
      __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4*>(to + at));
  } else {
    for (int64_t c = lane; c < n; c += 64) store1<WT>(p, i + c, 0.0f);
  }
}

// A wave per chunk and 512 columns: if a row begins in the chunk and goes on, its chunks' sums
// in order. The waves behind them clear the rows without a token.
template <int WT, int CHUNK>
__global__ __launch_bounds__(256) void embedding_join_kernel(SumArgs s) {
  const EmbeddingArgs& a = s.e;
  const int lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(flat_block()) * 4 + (threadIdx.x >> 6);
  if (item >= s.joins) {
    const int64_t row = item - s.joins;
    if (a.touched == nullptr || row >= a.vocab || a.touched[row]) return;
    clear_row<WT>(a.dtable, row * a.ld_table, a.cols);
    return;
  }
  const int64_t chunk = item / s.tiles;
  const int64_t first = chunk * CHUNK, end = first + CHUNK;
  const int key = s.keys[end - 1];
  if (key >= a.vocab || s.keys[end] != key || (first > 0 && s.keys[first - 1] == key)) return;
  const Eight c((item - chunk * s.tiles) * 512 + lane * 8, a.cols);
  float sum[8];
  read8<MUON_DTYPE_F32>(a.partial, (2 * chunk + 1) * a.cols + c.at, c.n, sum);
  for (int64_t d0 = chunk + 1; d0 < s.chunks; d0 += 64) {
    // the chunks that begin with this row's tokens
    const int64_t mine = d0 + lane;
    const unsigned long long more = __ballot(mine < s.chunks && s.keys[min(mine, s.chunks - 1) * CHUNK] == key);
    const int run = more == ~0ull ? 64 : __builtin_ctzll(~more);
    for (int d = 0; d < run; d += 4) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) read8<MUON_DTYPE_F32>(a.partial, 2 * (d0 + d + u) * a.cols + c.at, d + u < run ? c.n : 0, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[u][e];
    }
    if (run < 64) break;
  }
  finish_row<WT>(a, key, c, sum);
}

// ---------------------------------------------------------------------------

template <int TT>
static hipError_t launch_lookup(int dtype, const EmbeddingArgs& a, hipStream_t s) {
  const int tiles = static_cast<int>((a.cols + kEmbeddingCols - 1) / kEmbeddingCols);
  const dim3 grid = flat_grid((a.tokens * tiles + 3) / 4);
  if (dtype == MUON_DTYPE_F32) hipLaunchKernelGGL((embedding_kernel<TT, MUON_DTYPE_F32>), grid, dim3(256), 0, s, a, tiles);
  else if (dtype == MUON_DTYPE_BF16) hipLaunchKernelGGL((embedding_kernel<TT, MUON_DTYPE_BF16>), grid, dim3(256), 0, s, a, tiles);
  else hipLaunchKernelGGL((embedding_kernel<TT, MUON_DTYPE_F16>), grid, dim3(256), 0, s, a, tiles);
  return hipGetLastError();
}
hipError_t launch_embedding(int dtype, const EmbeddingArgs& a, hipStream_t s) {
  if (a.table_dtype == MUON_DTYPE_F32) return launch_lookup<MUON_DTYPE_F32>(dtype, a, s);
  if (a.table_dtype == MUON_DTYPE_BF16) return launch_lookup<MUON_DTYPE_BF16>(dtype, a, s);
  return launch_lookup<MUON_DTYPE_F16>(dtype, a, s);
}

hipError_t launch_sort_all(const EmbeddingArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(sort_all_kernel, dim3(1), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_sort_hist(const EmbeddingArgs& a, int pass, hipStream_t s) {
  hipLaunchKernelGGL(sort_hist_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a, pass);
  return hipGetLastError();
}
hipError_t launch_sort_place(const EmbeddingArgs& a, int pass, hipStream_t s) {
  hipLaunchKernelGGL(sort_place_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a, pass);
  return hipGetLastError();
}

static SumArgs sum_args(const EmbeddingArgs& a) {
  SumArgs s{};
  s.e = a;
  s.keys = a.keys[(a.passes - 1) & 1];
  s.slots = a.slots[(a.passes - 1) & 1];
  s.chunks = (a.tokens + a.chunk - 1) / a.chunk;
  s.tiles = (a.cols + 511) / 512;
  s.joins = std::max<int64_t>(s.chunks - 1, 0) * s.tiles;   // no row goes on from the last chunk
  return s;
}

template <int DT, int WT>
static hipError_t launch_sum(const SumArgs& g, hipStream_t s) {
  const dim3 grid = flat_grid((g.chunks * g.tiles + 3) / 4);
  if (g.e.chunk == 8) hipLaunchKernelGGL((embedding_sum_kernel<DT, WT, 8>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((embedding_sum_kernel<DT, WT, 32>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}
template <int DT>
static hipError_t launch_sum(const EmbeddingArgs& a, hipStream_t s) {
  const SumArgs g = sum_args(a);
  if (g.chunks == 0) return hipSuccess;
  if (a.table_dtype == MUON_DTYPE_F32) return launch_sum<DT, MUON_DTYPE_F32>(g, s);
  if (a.table_dtype == MUON_DTYPE_BF16) return launch_sum<DT, MUON_DTYPE_BF16>(g, s);
  return launch_sum<DT, MUON_DTYPE_F16>(g, s);
}
hipError_t launch_embedding_sum(int dtype, const EmbeddingArgs& a, hipStream_t s) {
  if (dtype == MUON_DTYPE_F32) return launch_sum<MUON_DTYPE_F32>(a, s);
  if (dtype == MUON_DTYPE_BF16) return launch_sum<MUON_DTYPE_BF16>(a, s);
  return launch_sum<MUON_DTYPE_F16>(a, s);
}

template <int WT>
static hipError_t launch_join(const EmbeddingArgs& a, hipStream_t s) {
  const SumArgs g = sum_args(a);
  const int64_t waves = g.joins + (a.touched != nullptr ? a.vocab : 0);
  if (waves == 0) return hipSuccess;
  const dim3 grid = flat_grid((waves + 3) / 4);
  if (a.chunk == 8) hipLaunchKernelGGL((embedding_join_kernel<WT, 8>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((embedding_join_kernel<WT, 32>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}
hipError_t launch_embedding_join(const EmbeddingArgs& a, hipStream_t s) {
  if (a.table_dtype == MUON_DTYPE_F32) return launch_join<MUON_DTYPE_F32>(a, s);
  if (a.table_dtype == MUON_DTYPE_BF16) return launch_join<MUON_DTYPE_BF16>(a, s);
  return launch_join<MUON_DTYPE_F16>(a, s);
}

}  // namespace muon
