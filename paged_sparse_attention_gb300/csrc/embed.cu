// Token embeddings at the front of a model, and their gradient by sorted tokens.
//
//   out[i, :]  = scale * table[t_i, :]                    (0 where there is no token, t_i < 0)
//   dT[t, :]  += scale * sum of d_out[i, :] over the rows i with t_i = t, in row order
//
// Forward: one pass, a row a group of threads; bound by HBM (distinct rows read, all written).
//
// Backward: rows of one token are summed by one owner in row order, so there are no float
// atomics and the gradient is the same bits on every run.  Up to 32 rows: sum_few, whose warps see all
// tokens at once.  More, in three or four launches:
//   rank_tokens   the stable order of a section: a token's place is the number of those that come
//                 before it, counted by a warp's 32 tokens against the section's.  No pass waits for another
//                 and every SM has a part.  8192 tokens in sections of 1024, with the merge: 4 us less than
//                 at once, 14 less than sorted.
//   sort_tokens   instead, for many tokens: a section a block, by a radix sort of 6 bits a pass in
//                 shared memory (20 us for one section or nine).
//   merge_sections  where there are several sections: a key's rank among all keys is the sum of its
//                 places in every section, found by binary search.
//   sum_runs      the sorted rows in windows of kWindow.  The rows of one token in one window are a
//                 piece, summed in fp32 by one block.  A token whose rows lie in one window goes
//                 straight to its row of the table's gradient.
//   join_pieces   tokens whose rows go on into other windows: their pieces, summed in order.
#include <climits>
#include <type_traits>

#include "attn_common.cuh"
#include "embed.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kRankAll = 4096;       // tokens up to which every one is ranked among all
constexpr int kRankSection = 1024, kRankMost = 28 * 1024;  // ranked in sections up to so many, sorted in sections of
constexpr int kSection = 8192;       // these above
constexpr int kRankKeys = 32, kRankWarps = 16;  // of a block of rank_tokens: tokens, warps that share the comparisons
constexpr int kSortThreads = 1024, kSortKeys = kSection / kSortThreads;
constexpr int kDigit = 6;       // bits a pass
constexpr int kWindow = 16;     // sorted rows a piece lies in
constexpr int kNone = INT_MAX;  // key of a row without a token: behind every other
constexpr int kMostRows = 1 << 26;  // of a gradient: each section is searched for every row (2^24 rows take 0.33 s, 2^26 5)

__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Key of a token: itself, kNone where it is none; outside [0, V) is told.
__device__ __forceinline__ int key_of(int64_t t, int V, uint32_t* err) {
  if (t >= V) {
    atomicOr(err, OOMB_DEVERR_TOKEN);
    return kNone;
  }
  return t < 0 ? kNone : (int)t;
}

// E consecutive elements as fp32 and back, 16 bytes an access (E = 1: one element).
template <typename T, int E>
__device__ __forceinline__ void load_e(const T* p, float (&f)[E]) {
  if constexpr (E == 1) {
    f[0] = to_float<T>(*p);
  } else {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < E; i += V) {
      const uint4 w = *reinterpret_cast<const uint4*>(p + i);
      const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int e = 0; e < V; ++e) f[i + e] = to_float<T>(x[e]);
    }
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T* p, const float (&f)[E]) {
  if constexpr (E == 1) {
    *p = from_float<T>(f[0]);
  } else {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < E; i += V) {
      uint4 w;
      T* x = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = from_float<T>(f[i + e]);
      *reinterpret_cast<uint4*>(p + i) = w;
    }
  }
}

// ------------------------------------------------------------------ forward
// A block: `rows` sets of RR rows, blockDim.x / rows threads each, NV vectors of E elements of each row a thread
// asked for at once (element by element, four rows of four against one of eight: 65000 rows of 65 in fp32 in
// 8 us, 14; 8000 of 3001 in bf16 22, 28): many small blocks, whose token, row and stores wait for one another, hide
// each other's.  (Blocks that walk the rows with the next one in flight took 23 us for 8192 rows of
// 3584 in bf16, these 18 at 8 KB a block.)
template <typename T, int E, int NV, int RR>
__global__ void __launch_bounds__(256) embed_rows(const __grid_constant__ EmbedArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int per_row = blockDim.x / a.rows, r = threadIdx.x / per_row, lane = threadIdx.x % per_row;
  const int64_t i = ((int64_t)blockIdx.x * a.rows + r) * RR;
  if (i >= a.n) return;
  const int live = (int)min((int64_t)RR, a.n - i);
  int64_t token[RR];
  const T* in[RR];
  bool has[RR];
#pragma unroll
  for (int q = 0; q < RR; ++q) token[q] = q < live ? a.tokens[i + q] : -1;
#pragma unroll
  for (int q = 0; q < RR; ++q) {
    const int key = key_of(token[q], a.V, a.err);
    has[q] = key != kNone;
    in[q] = reinterpret_cast<const T*>(a.table) + (size_t)(has[q] ? key : 0) * a.D;
  }
  T* out = reinterpret_cast<T*>(a.out) + (size_t)i * a.D;
  const int step = per_row * E;
  for (int c = lane * E; c < a.D; c += NV * step) {
    float f[RR][NV][E];
#pragma unroll
    for (int q = 0; q < RR; ++q)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[q][v][e] = 0.f;
        if (has[q] && c + v * step < a.D) load_e<T, E>(in[q] + c + v * step, f[q][v]);
      }
#pragma unroll
    for (int q = 0; q < RR; ++q)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[q][v][e] *= a.scale;
        if (q < live && c + v * step < a.D) store_e<T, E>(out + (size_t)q * a.D + c + v * step, f[q][v]);
      }
  }
}

// ----------------------------------------------------------------- ordering
// Tokens before the warp's own count when they are not greater, those behind when they are smaller:
// equal tokens keep their order.
template <int SECTION>
__global__ void __launch_bounds__(32 * kRankWarps) rank_tokens(const __grid_constant__ EmbedArgs a) {
  __shared__ __align__(16) int keys[SECTION];
  __shared__ int parts[kRankWarps][kRankKeys];
  constexpr int T = 32 * kRankWarps, K = SECTION / T;
  wait_for_launch_before();
  let_next_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.n_long[0] = a.n_long[1] = 0;
  const int64_t first = (int64_t)blockIdx.x * kRankKeys / SECTION * SECTION;  // of the block's section
  const int m = (int)min((int64_t)SECTION, a.n - first), own = (int)((int64_t)blockIdx.x * kRankKeys - first), m4 = (m + 3) & ~3;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t* tokens = a.tokens + first;
  int64_t token[K];
#pragma unroll
  for (int k = 0; k < K; ++k) token[k] = threadIdx.x + k * T < m ? tokens[threadIdx.x + k * T] : -1;
#pragma unroll
  for (int k = 0; k < K; ++k) keys[threadIdx.x + k * T] = key_of(token[k], a.V, a.err);
  __syncthreads();
  const int mine = keys[own + lane];  // (own + lane < SECTION; behind the last it is kNone and not used)
  // x < y as the sign of x - y: both lie in [0, 2^31)
  auto below = [](int x, int y) { return (unsigned)(x - y) >> 31; };
  unsigned c0 = 0, c1 = 0, c2 = 0, c3 = 0;
  const int4* v = reinterpret_cast<const int4*>(keys);
#pragma unroll 4
  for (int j = warp; j < own / 4; j += kRankWarps) {  // not greater: all but those above
    const int4 x = v[j];
    c0 += 1 - below(mine, x.x);
    c1 += 1 - below(mine, x.y);
    c2 += 1 - below(mine, x.z);
    c3 += 1 - below(mine, x.w);
  }
  for (int j = own + warp; j < min(own + kRankKeys, m); j += kRankWarps)
    c0 += keys[j] < mine || (keys[j] == mine && j < own + lane);
#pragma unroll 4
  for (int j = (own + kRankKeys) / 4 + warp; j < m4 / 4; j += kRankWarps) {
    const int4 x = v[j];
    c0 += below(x.x, mine);
    c1 += below(x.y, mine);
    c2 += below(x.z, mine);
    c3 += below(x.w, mine);
  }
  parts[warp][lane] = (int)((c0 + c1) + (c2 + c3));
  __syncthreads();
  if (warp != 0 || own + lane >= m) return;
  int at = 0;
#pragma unroll
  for (int p = 0; p < kRankWarps; ++p) at += parts[p][lane];
  const bool alone = a.n <= SECTION;
  (alone ? a.sorted : a.sec_sorted)[first + at] = mine;
  (alone ? a.order : a.sec_order)[first + at] = (int)first + own + lane;
}

// One block a section.  Keys and their rows stand in shared memory in the order reached; in a pass a
// warp takes 256 of them in turn, 32 at a time, and counts its digits, equal digits among the 32 by
// ballots, so that equal keys keep their order.
constexpr int kCountPitch = (1 << kDigit) + 1;
struct SortSpace {
  int keys[kSection];
  uint16_t rows[kSection];
  int counts[32 * kCountPitch];  // [warp, digit], so that a warp's digits lie in different banks
  int sums[64];
};
__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens(const __grid_constant__ EmbedArgs a) {
  extern __shared__ __align__(16) uint8_t sort_mem[];
  SortSpace& s = *reinterpret_cast<SortSpace*>(sort_mem);
  wait_for_launch_before();
  let_next_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t first = (int64_t)blockIdx.x * kSection;
  const int m = (int)min((int64_t)kSection, a.n - first);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.n_long[0] = a.n_long[1] = 0;
  int key[kSortKeys], row[kSortKeys];
  int64_t token[kSortKeys];
  auto place = [&](int k) { return warp * (32 * kSortKeys) + k * 32 + lane; };
#pragma unroll
  for (int k = 0; k < kSortKeys; ++k) token[k] = place(k) < m ? a.tokens[first + place(k)] : -1;
#pragma unroll
  for (int k = 0; k < kSortKeys; ++k) {
    row[k] = place(k);
    const int t = key_of(token[k], a.V, a.err);
    key[k] = t == kNone ? a.V : t;  // behind every token; rows behind the section's last stay behind them too
  }
  for (int shift = 0; shift < a.key_bits; shift += kDigit) {
    const int bits = min(kDigit, a.key_bits - shift), digits = 1 << bits;
    for (int i = threadIdx.x; i < 32 * kCountPitch; i += kSortThreads) s.counts[i] = 0;
    __syncthreads();
    int before[kSortKeys];
    unsigned same_of[kSortKeys];  // lanes with the same digit
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
      unsigned same = 0xffffffffu;
#pragma unroll
      for (int b = 0; b < kDigit; ++b) {
        const bool one = (key[k] >> (shift + b)) & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        if (b < bits) same &= one ? ones : ~ones;
      }
      same_of[k] = same;
    }
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
      const int d = (key[k] >> shift) & (digits - 1);
      const unsigned same = same_of[k];
      int* count = &s.counts[warp * kCountPitch + d];
      before[k] = *count + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (lane == __ffs(same) - 1) *count += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // sums of the counts in front, digit after digit and warp after warp
    // a thread: digit `warp` and, of 64, digit `warp` + 32, of the lane's warp
    const int d0 = lane * kCountPitch + warp, d1 = d0 + 32;
    const int n0 = s.counts[d0], n1 = s.counts[d1];
    int i0 = n0, i1 = n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u0 = __shfl_up_sync(0xffffffffu, i0, o), u1 = __shfl_up_sync(0xffffffffu, i1, o);
      if (lane >= o) {
        i0 += u0;
        i1 += u1;
      }
    }
    if (lane == 31) {
      s.sums[warp] = i0;
      s.sums[32 + warp] = i1;
    }
    __syncthreads();
    // of the digits before: lane d holds digits d and d + 32
    int t0 = s.sums[lane], t1 = s.sums[32 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u0 = __shfl_up_sync(0xffffffffu, t0, o), u1 = __shfl_up_sync(0xffffffffu, t1, o);
      if (lane >= o) {
        t0 += u0;
        t1 += u1;
      }
    }
    const int half = __shfl_sync(0xffffffffu, t0, 31);
    const int p0 = __shfl_sync(0xffffffffu, t0, (warp + 31) & 31), p1 = __shfl_sync(0xffffffffu, t1, (warp + 31) & 31);
    s.counts[d0] = (warp == 0 ? 0 : p0) + i0 - n0;
    s.counts[d1] = half + (warp == 0 ? 0 : p1) + i1 - n1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
      const int at = s.counts[warp * kCountPitch + ((key[k] >> shift) & (digits - 1))] + before[k];
      s.keys[at] = key[k];
      s.rows[at] = (uint16_t)row[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) {
      key[k] = s.keys[place(k)];
      row[k] = s.rows[place(k)];
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kSortKeys; ++k) {
    const int j = place(k);
    if (j >= m) continue;
    a.sec_sorted[first + j] = key[k] == a.V ? kNone : key[k];
    a.sec_order[first + j] = (int)first + row[k];
  }
}

// LANES lanes a key share the other sections; four searches of a lane run side by side, as each is a chain of
// dependent loads.
constexpr int kSearches = 4, kMergeThreads = 256;
template <int SECTION, int LANES>
__global__ void __launch_bounds__(kMergeThreads) merge_sections(const __grid_constant__ EmbedArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int64_t j = ((int64_t)blockIdx.x * kMergeThreads + threadIdx.x) / LANES;
  const int part = threadIdx.x % LANES;
  const bool live = j < a.n;
  const int key = live ? a.sec_sorted[j] : 0, mine = (int)(j / SECTION);
  const int sections = live ? (int)((a.n + SECTION - 1) / SECTION) : 0;
  int at = 0;
  for (int s0 = part; s0 < sections; s0 += LANES * kSearches) {
    int lo[kSearches], hi[kSearches];
#pragma unroll
    for (int u = 0; u < kSearches; ++u) {
      const int s = s0 + u * LANES;
      lo[u] = 0;
      hi[u] = s < sections && s != mine ? (int)min((int64_t)SECTION, a.n - (int64_t)s * SECTION) : 0;
    }
    for (int left = SECTION; left > 0; left >>= 1) {  // a section's keys below `key`, up to it in those before
#pragma unroll
      for (int u = 0; u < kSearches; ++u) {
        if (lo[u] >= hi[u]) continue;
        const int s = s0 + u * LANES, mid = (lo[u] + hi[u]) >> 1, x = a.sec_sorted[(int64_t)s * SECTION + mid];
        if (x < key || (s < mine && x == key))
          lo[u] = mid + 1;
        else
          hi[u] = mid;
      }
    }
#pragma unroll
    for (int u = 0; u < kSearches; ++u) at += lo[u];
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
  if (!live || part != 0) return;
  const int64_t to = j % SECTION + at;
  a.sorted[to] = key;
  a.order[to] = a.sec_order[j];
}

// ------------------------------------------------------------------ sums
// Up to 32 rows.  A warp takes 32 E columns; lane i holds token i, and the lanes that hold the same one are
// known to all.  The tokens' sums are dealt out over grid.y.
template <typename T, int E>
__global__ void __launch_bounds__(128) sum_few(const __grid_constant__ EmbedArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int lane = threadIdx.x % 32, c = ((blockIdx.x * 4 + threadIdx.x / 32) * 32 + lane) * E;
  const int key = lane < a.n ? key_of(a.tokens[lane], a.V, a.err) : kNone;
  const unsigned same = __match_any_sync(0xffffffffu, key);
  unsigned firsts = __ballot_sync(0xffffffffu, key != kNone && lane == __ffs(same) - 1);
  for (int k = 0; firsts; firsts &= firsts - 1, ++k) {
    if (k % gridDim.y != blockIdx.y) continue;
    const int first = __ffs(firsts) - 1, token = __shfl_sync(0xffffffffu, key, first);
    unsigned rows = __shfl_sync(0xffffffffu, same, first);
    if (c >= a.D) continue;
    float* to = a.d_table + (size_t)token * a.D + c;
    float old[E], sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) old[e] = sum[e] = 0.f;
    if (a.accumulate) load_e<float, E>(to, old);
    while (rows) {
      constexpr int B = 4;  // asked for together
      float f[B][E];
#pragma unroll
      for (int u = 0; u < B; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[u][e] = 0.f;
        if (rows) load_e<T, E>(reinterpret_cast<const T*>(a.d_out) + (size_t)(__ffs(rows) - 1) * a.D + c, f[u]);
        rows &= rows - 1;  // (0 stays 0)
      }
#pragma unroll
      for (int u = 0; u < B; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] += f[u][e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = fmaf(a.scale, sum[e], old[e]);
    store_e<float, E>(to, sum);
  }
}

// Where the partial sum of a piece of window w is kept: one may come from the window before (it
// starts the window), one more may go on into the next.
__device__ __forceinline__ size_t piece_slot(int64_t w, bool first) { return (size_t)w * 2 + (first ? 1 : 0); }

// Threads of a block, at most.  (Element by element, 512 take 83 us for 8000 rows of 3001 in fp32, 320 take 73;
// longer vectors hold more loads each.)
constexpr int run_threads(int E) { return E == 1 ? 320 : 512; }

// NV vectors of E elements a thread.  A block walks the windows b, b + grid, ...; the next window's
// tokens are on their way while this one's rows are summed.  A batch's rows are all asked for before
// the first is used, held as they are stored.  Rows of the gradient that will be added to are asked
// into L2 at a window's start and from there one piece ahead.  (Additions in L2 instead, which wait for
// nothing, are an element an operation there: 38 us
// against 33 for 8192 tokens of 3584 in bf16, whose bytes take 26.)
template <typename T, int E, int NV>
__global__ void __launch_bounds__(512, 2) sum_runs(const __grid_constant__ EmbedArgs a) {
  constexpr int R = 4;  // rows of a batch
  using Word = typename std::conditional<E == 1, T, uint4>::type;
  __shared__ int rows_of[2][kWindow], keys_of[2][kWindow + 2];  // keys[.][0]: of the row before the window
  wait_for_launch_before();
  let_next_launch();
  const int width = blockDim.x * E * NV, slab = blockIdx.y * width;
  const int c0 = slab + threadIdx.x * E, step = blockDim.x * E;
  const T* d_out = reinterpret_cast<const T*>(a.d_out) + c0;
  auto add_word = [](float (&sum)[E], const Word& w) {
    const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] += to_float<T>(x[e]);
  };
  // thread j: entry j of a window's lists
  int next_key = kNone, next_row = 0;
  auto ask = [&](int64_t w) {
    const int64_t p = w * kWindow + (int)threadIdx.x - 1;
    if (w >= a.windows || threadIdx.x >= kWindow + 2) return;
    next_key = p >= 0 && p < a.n ? a.sorted[p] : kNone;
    next_row = threadIdx.x < kWindow && p + 1 < a.n ? a.order[p + 1] : 0;
  };
  ask(blockIdx.x);
  int buf = 0;
  for (int64_t window = blockIdx.x; window < a.windows; window += gridDim.x, buf ^= 1) {
    int* rows = rows_of[buf];
    int* keys = keys_of[buf];
    if (threadIdx.x < kWindow + 2) keys[threadIdx.x] = next_key;
    if (threadIdx.x < kWindow) rows[threadIdx.x] = next_row;
    __syncthreads();  // (the window before last has been read: its readers have passed the last barrier)
    ask(window + gridDim.x);
    if (E > 1 && a.accumulate && threadIdx.x < kWindow) {
      const int key = keys[threadIdx.x + 1];
      if (key != kNone && key != keys[threadIdx.x])
        prefetch_l2(a.d_table + (size_t)key * a.D + slab, (uint32_t)min(width, a.D - slab) * 4);
    } else if (E == 1 && a.accumulate) {  // rows off 16 bytes: line by line
      for (int j = threadIdx.x / 32; j < kWindow; j += blockDim.x / 32) {
        const int key = keys[j + 1];
        if (key == kNone || key == keys[j]) continue;
        for (int c = slab + threadIdx.x % 32 * 32; c < min(a.D, slab + width); c += 32 * 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.d_table + (size_t)key * a.D + c));
      }
    }
    int live = 0;  // rows that have a token
    while (live < kWindow && keys[live + 1] != kNone) ++live;
    float sum[NV][E], old[NV][E], ahead[NV][E];
    bool first = false;  // the piece being summed is its token's first
    // what the gradient's row holds, for a piece that starts at row j and may be its token's only one
    auto ask_old = [&](int j) {
      const int key = keys[j + 1];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < E; ++e) ahead[v][e] = 0.f;
        if (j < live && a.accumulate && key != keys[j] && c0 + v * step < a.D)
          load_e<float, E>(a.d_table + (size_t)key * a.D + c0 + v * step, ahead[v]);
      }
    };
    if (E > 1) ask_old(0);
    for (int j0 = 0; j0 < live; j0 += R) {
      Word raw[R][NV];
#pragma unroll
      for (int u = 0; u < R; ++u)
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (j0 + u < live && c0 + v * step < a.D)
            raw[u][v] = *reinterpret_cast<const Word*>(d_out + (size_t)rows[j0 + u] * a.D + v * step);
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const int j = j0 + u;
        if (j >= live) continue;
        const int key = keys[j + 1];
        if (j == 0 || key != keys[j]) {  // a piece starts
          first = key != keys[j];
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              sum[v][e] = 0.f;
              if (E > 1) old[v][e] = ahead[v][e];
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (c0 + v * step < a.D) add_word(sum[v], raw[u][v]);
        const bool last = keys[j + 2] != key;
        if (!last && j + 1 < kWindow) continue;
        if (E > 1 && j + 1 < kWindow) ask_old(j + 1);
        const bool only = first && last;
        if (E == 1 && only)
#pragma unroll
          for (int v = 0; v < NV; ++v)
            old[v][0] = a.accumulate && c0 + v * step < a.D ? a.d_table[(size_t)key * a.D + c0 + v * step] : 0.f;
        float* to = only ? a.d_table + (size_t)key * a.D : a.part + piece_slot(window, first) * a.pitch;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (c0 + v * step >= a.D) continue;
#pragma unroll
          for (int e = 0; e < E; ++e) sum[v][e] = only ? fmaf(a.scale, sum[v][e], old[v][e]) : sum[v][e];
          store_e<float, E>(to + c0 + v * step, sum[v]);
        }
        // the token's last piece tells the join about it (in any order: each has a row of its own), with its
        // first window, the last one whose first row does not go on with it, if that is one of the last 32
        if (last && !first && blockIdx.y == 0 && threadIdx.x < 32) {
          const int64_t w = window - (int)threadIdx.x;
          const unsigned stops = __ballot_sync(0xffffffffu, w <= 0 || a.sorted[max(w, (int64_t)1) * kWindow - 1] != key);
          if (threadIdx.x == 0) {
            if (stops)
              a.long_runs[atomicAdd(a.n_long, 1)] = make_int4(key, (int)window - (__ffs(stops) - 1), (int)window, 0);
            else
              a.long_runs[a.windows - 1 - atomicAdd(a.n_long + 1, 1)] = make_int4(key, 0, (int)window, 0);
          }
        }
      }
    }
  }
}

// Joins the tokens whose rows lie in several windows.  Most have a few pieces: a warp takes 128 columns
// of one.  Those with more than 32, which a common token has in a long batch, are taken by whole
// blocks, 32 columns each, whose groups of eight lanes take a share of the pieces each; the shares' sums are added
// in order.
constexpr int kJoinCols = 128, kJoinWarps = 16;
constexpr int kHeavyCols = 32, kGroup = kHeavyCols / 4, kShares = kJoinWarps * 32 / kGroup;
__global__ void __launch_bounds__(32 * kJoinWarps) join_pieces(const __grid_constant__ EmbedArgs a) {
  __shared__ float4 share[kJoinWarps][32];
  wait_for_launch_before();
  const int chunks = (a.D + kJoinCols - 1) / kJoinCols, strips = (a.D + kHeavyCols - 1) / kHeavyCols;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // first window of a run that goes back from window w by more than 32: a search that cuts in 33 at a step
  auto first_window = [&](int key, int w) {
    int lo = 0, hi = w - 31;  // the first row of window hi goes on with the run, that of lo does not
    while (hi - lo > 1) {
      const int x = lo + (int)((int64_t)(hi - lo) * (lane + 1) / 33);
      const bool goes_back = x > 0 && a.sorted[(int64_t)x * kWindow - 1] == key;
      const unsigned back = __ballot_sync(0xffffffffu, goes_back);  // lanes from some one on
      const int from = back ? __ffs(back) - 1 : 32;
      const int low = __shfl_sync(0xffffffffu, x, max(from - 1, 0)), high = __shfl_sync(0xffffffffu, x, min(from, 31));
      if (from > 0) lo = max(lo, low);
      if (from < 32) hi = high;
    }
    return lo;
  };
  auto sum_of = [&](int begin, int from, int to, int c) {  // pieces [from, to) of the run
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c >= a.D) return sum;
    constexpr int B = 8;  // asked for together
    for (int k = from; k < to; k += B) {
      float4 x[B];
#pragma unroll
      for (int u = 0; u < B; ++u)
        x[u] = k + u < to ? *reinterpret_cast<const float4*>(a.part + piece_slot(begin + k + u, k + u == 0) * a.pitch + c)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < B; ++u) {
        sum.x += x[u].x;
        sum.y += x[u].y;
        sum.z += x[u].z;
        sum.w += x[u].w;
      }
    }
    return sum;
  };
  auto read = [&](int key, int c, float (&old)[4]) {
    const float* from = a.d_table + (size_t)key * a.D + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) old[e] = a.accumulate && c + e < a.D ? from[e] : 0.f;
  };
  auto write = [&](int key, int c, const float4& sum, const float (&old)[4]) {
    const float f[4] = {sum.x, sum.y, sum.z, sum.w};
    float* to = a.d_table + (size_t)key * a.D + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < a.D) to[e] = fmaf(a.scale, f[e], old[e]);
  };
  const int64_t heavy = (int64_t)a.n_long[1] * strips, light = (int64_t)a.n_long[0] * chunks;
  for (int64_t it = blockIdx.x; it < heavy; it += gridDim.x) {
    const int4 run = a.long_runs[a.windows - 1 - it / strips];
    const int c = (int)(it % strips) * kHeavyCols + 4 * (lane % kGroup);
    const int begin = first_window(run.x, run.z), pieces = run.z - begin + 1;
    const int per = (pieces + kShares - 1) / kShares, mine = warp * (32 / kGroup) + lane / kGroup;
    float4 sum = sum_of(begin, mine * per, min(pieces, (mine + 1) * per), c);
    auto add = [&](const float4& y) {
      sum.x += y.x;
      sum.y += y.y;
      sum.z += y.z;
      sum.w += y.w;
    };
    share[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && lane < kGroup) {
#pragma unroll 8
      for (int x = 1; x < kShares; ++x) add(share[x / (32 / kGroup)][x % (32 / kGroup) * kGroup + lane]);
      float old[4];
      read(run.x, c, old);
      write(run.x, c, sum, old);
    }
    __syncthreads();
  }
  for (int64_t it = (int64_t)blockIdx.x * kJoinWarps + warp; it < light; it += (int64_t)gridDim.x * kJoinWarps) {
    const int4 run = a.long_runs[it / chunks];
    const int c = (int)(it % chunks) * kJoinCols + 4 * lane;
    float old[4];
    read(run.x, c, old);
    write(run.x, c, sum_of(run.y, 0, run.z - run.y + 1, c), old);
  }
}

template <typename K>
cudaError_t launch_after(K kernel, dim3 grid, int threads, const EmbedArgs& a, cudaStream_t st, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;  // a dependent launch: its set-up overlaps the end of the one before, which it waits for
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int E, int NV, int RR>
cudaError_t forward(EmbedArgs& a, cudaStream_t st) {
  const int vecs = (a.D + E * NV - 1) / (E * NV);
  const int per_row = (int)std::min<size_t>(256, align_up((size_t)vecs, 32));
  const int64_t sets = (a.n + RR - 1) / RR;
  a.rows = 256 / per_row;
  while (a.rows > 1 && (sets + a.rows - 1) / a.rows < 2 * device_sm_count()) a.rows /= 2;
  return launch_after(embed_rows<T, E, NV, RR>, dim3((unsigned)((sets + a.rows - 1) / a.rows)), per_row * a.rows, a, st);
}

size_t sort_smem_set[kMaxDevices] = {};

// The sorted order.  Both sides of the two bounds, gradient of 8 columns, us by the three ways (ranks of
// all, ranks of sections, sorted sections): 4096 tokens 15.1 / 16.4 / 30.6, 6000: 20.3 / 18.0, 8192: 23.5 /
// 19.1 / 33.3, 24000: - / 30.5 / 40.4, 33000: - / 45.7 / 42.7, 65537: - / 97 / 62.
cudaError_t order_tokens(const EmbedArgs& a, cudaStream_t st) {
  auto merge = [&](auto kernel, int lanes) {
    return launch_after(kernel, dim3((unsigned)((a.n * lanes + kMergeThreads - 1) / kMergeThreads)), kMergeThreads, a, st);
  };
  const dim3 rank_grid((unsigned)((a.n + kRankKeys - 1) / kRankKeys));
  if (a.n <= kRankAll) return launch_after(rank_tokens<kRankAll>, rank_grid, 32 * kRankWarps, a, st);
  cudaError_t e;
  if (a.n <= kRankMost) {
    e = launch_after(rank_tokens<kRankSection>, rank_grid, 32 * kRankWarps, a, st);
    return e == cudaSuccess ? merge(merge_sections<kRankSection, 8>, 8) : e;
  }
  e = set_smem_limit((const void*)sort_tokens, sizeof(SortSpace), sort_smem_set);
  if (e != cudaSuccess) return e;
  e = launch_after(sort_tokens, dim3((unsigned)((a.n + kSection - 1) / kSection)), kSortThreads, a, st, sizeof(SortSpace));
  return e == cudaSuccess ? merge(merge_sections<kSection, 2>, 2) : e;
}

template <typename T, int E, int NV>
cudaError_t backward(const EmbedArgs& a, cudaStream_t st) {
  if (a.n <= 32) {
    const int64_t warps = ((int64_t)a.D + 32 * E - 1) / (32 * E);
    return launch_after(sum_few<T, E>, dim3((unsigned)((warps + 3) / 4), (unsigned)std::min<int64_t>(a.n, 16)), 128, a, st);
  }
  cudaError_t e = order_tokens(a, st);
  if (e != cudaSuccess) return e;
  const int vecs = (a.D + E * NV - 1) / (E * NV);
  const int slabs = (vecs + run_threads(E) - 1) / run_threads(E);
  const int threads = std::max(64, (int)align_up((size_t)(vecs + slabs - 1) / slabs, 32));
  const int64_t most = (int64_t)(1024 / threads) * device_sm_count();
  e = launch_after(sum_runs<T, E, NV>,
                   dim3((unsigned)std::min<int64_t>(a.windows, std::max<int64_t>(1, most / slabs)), (unsigned)slabs),
                   threads, a, st);
  if (e != cudaSuccess || a.n <= kWindow) return e;
  // at most a run goes on from each window into the next
  const int64_t items = ((a.n - 1) / kWindow) * ((a.D + kJoinCols - 1) / kJoinCols);
  const int64_t blocks = std::min<int64_t>((items + kJoinWarps - 1) / kJoinWarps, 3 * device_sm_count());
  return launch_after(join_pieces, dim3((unsigned)blocks), 32 * kJoinWarps, a, st);
}

template <typename T>
cudaError_t forward_any(EmbedArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.table) && on16(a.out) ? forward<T, E, 4, 1>(a, st) : forward<T, 1, 4, 4>(a, st);
}
template <typename T>
cudaError_t backward_any(const EmbedArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.d_out) && on16(a.d_table) ? backward<T, E, 1>(a, st) : backward<T, 1, 4>(a, st);
}

// Workspace: order, sorted [n] int each (twice for several sections), the tokens to join, the pieces.
struct EmbedSpace {
  size_t order, sorted, sec_order, sec_sorted, n_long, long_runs, part, bytes;
  int64_t pitch;
};
EmbedSpace embed_space(int64_t n, int D) {
  EmbedSpace s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  s.order = take((size_t)n * 4);
  s.sorted = take((size_t)n * 4);
  s.sec_order = take(n > kRankAll ? (size_t)n * 4 : 0);
  s.sec_sorted = take(n > kRankAll ? (size_t)n * 4 : 0);
  s.n_long = take(8);
  const size_t windows = (size_t)(n + kWindow - 1) / kWindow;
  s.long_runs = take(windows * 16);
  s.pitch = (int64_t)align_up((size_t)D, 4);
  s.part = take(n > kWindow ? windows * 2 * s.pitch * 4 : 0);
  s.bytes = at;
  return s;
}

oomb_status check_embed(const int64_t* tokens, int n, int V, int D, int dtype, float scale, const uint32_t* word) {
  if (!tokens || !word || n <= 0 || V <= 0 || V == INT_MAX || D <= 0 || !(scale - scale == 0.f)) return OOMB_ERR_ARG;
  if (dtype != OOMB_BF16 && dtype != OOMB_FP32) return OOMB_ERR_DTYPE;
  if (D > 1 << 24) return OOMB_ERR_UNSUPPORTED;  // columns are cut over a grid dimension
  if (reinterpret_cast<uintptr_t>(tokens) % 8 || reinterpret_cast<uintptr_t>(word) % 4) return OOMB_ERR_ALIGN;
  return OOMB_OK;
}

}  // namespace
}  // namespace oomb

using namespace oomb;

extern "C" {

oomb_status oomb_embed_fwd(const int64_t* tokens, int n, const void* table, int V, int D, int dtype, float scale,
                           void* out, uint32_t* error_word, void* stream) {
  const oomb_status s = check_embed(tokens, n, V, D, dtype, scale, error_word);
  if (s != OOMB_OK) return s;
  if (!table || !out) return OOMB_ERR_ARG;
  const uintptr_t es = dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(table) % es || reinterpret_cast<uintptr_t>(out) % es) return OOMB_ERR_ALIGN;
  EmbedArgs a = {};
  a.tokens = tokens;
  a.table = table;
  a.out = out;
  a.n = n;
  a.V = V;
  a.D = D;
  a.scale = scale;
  a.err = error_word;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? forward_any<float>(a, st) : forward_any<__nv_bfloat16>(a, st));
}

size_t oomb_embed_workspace(int n, int D) { return n <= 0 || D <= 0 ? 0 : embed_space(n, D).bytes; }

oomb_status oomb_embed_bwd(const int64_t* tokens, int n, const void* d_out, int V, int D, int dtype, float scale,
                           float* d_table, int accumulate, void* workspace, size_t ws_bytes, uint32_t* error_word,
                           void* stream) {
  const oomb_status s = check_embed(tokens, n, V, D, dtype, scale, error_word);
  if (s != OOMB_OK) return s;
  if (!d_out || !d_table) return OOMB_ERR_ARG;
  if (n > kMostRows) return OOMB_ERR_UNSUPPORTED;
  const EmbedSpace w = embed_space(n, D);
  if (!workspace || ws_bytes < w.bytes) return OOMB_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(d_out) % dtype_size(dtype) || reinterpret_cast<uintptr_t>(d_table) % 4 ||
      reinterpret_cast<uintptr_t>(workspace) % 16)
    return OOMB_ERR_ALIGN;
  char* base = reinterpret_cast<char*>(workspace);
  EmbedArgs a = {};
  a.tokens = tokens;
  a.d_out = d_out;
  a.d_table = d_table;
  a.accumulate = accumulate != 0;
  a.n = n;
  a.V = V;
  a.D = D;
  a.scale = scale;
  a.err = error_word;
  a.order = reinterpret_cast<int*>(base + w.order);
  a.sorted = reinterpret_cast<int*>(base + w.sorted);
  a.sec_order = reinterpret_cast<int*>(base + w.sec_order);
  a.sec_sorted = reinterpret_cast<int*>(base + w.sec_sorted);
  a.key_bits = 1;
  while (a.key_bits < 31 && (V >> a.key_bits) != 0) ++a.key_bits;
  a.n_long = reinterpret_cast<int*>(base + w.n_long);
  a.long_runs = reinterpret_cast<int4*>(base + w.long_runs);
  a.part = reinterpret_cast<float*>(base + w.part);
  a.pitch = w.pitch;
  a.windows = (n + kWindow - 1) / kWindow;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? backward_any<float>(a, st) : backward_any<__nv_bfloat16>(a, st));
}

}  // extern "C"
