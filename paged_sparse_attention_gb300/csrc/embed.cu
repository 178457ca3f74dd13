// Token embeddings at the front of a model, and their gradient by sorted tokens.
//
//   out[i, :]  = scale * table[t_i, :]                    (0 where there is no token, t_i < 0)
//   dT[t, :]  += scale * sum of d_out[i, :] over the rows i with t_i = t, in row order
//
// Forward: one pass, a row a group of threads; bound by HBM (distinct rows read, all written).
//
// Backward: rows of one token are summed by one owner in row order, so there are no float
// atomics and the gradient is the same bits on every run.  Three or four launches:
//   rank_tokens   the stable order of the tokens.  A key's rank among the keys of its section is
//                 counted directly, as the number of keys that come before it: sorting by passes
//                 would need several dependent launches for a chunk of a few thousand tokens.
//   merge_ranks   where there are several sections: a key's rank among all keys is the sum of its
//                 places in every section, found by binary search.
//   sum_runs      the sorted rows in windows of kWindow.  The rows of one token in one window are a
//                 piece, summed in fp32 by the block in whose tile it starts.  A token whose rows
//                 lie in one window goes straight to its row of the table's gradient.
//   join_pieces   tokens whose rows go on into other windows: their pieces, summed in order.
#include <climits>

#include "attn_common.cuh"
#include "embed.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kSection = 8192;  // most keys ranked against each other: 32 KB of shared memory
constexpr int kRankKeys = 32;   // keys a block ranks
constexpr int kRankParts = 16;  // warps that share the comparisons of one key
constexpr int kWindow = 64;     // sorted rows a piece lies in
constexpr int kNone = INT_MAX;  // key of a row without a token: behind every other

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
// Rows of a block: `rows` of them at a time, blockDim.x / rows threads each, NV vectors of E elements
// a thread at a time.
template <typename T, int E, int NV>
__global__ void __launch_bounds__(256) embed_rows(const __grid_constant__ EmbedArgs a) {
  const int per_row = blockDim.x / a.rows, r = threadIdx.x / per_row, lane = threadIdx.x % per_row;
  const int64_t i = (int64_t)blockIdx.x * a.rows + r;
  if (r >= a.rows || i >= a.n) return;
  const int key = key_of(a.tokens[i], a.V, a.err);
  T* out = reinterpret_cast<T*>(a.out) + (size_t)i * a.D;
  const T* in = reinterpret_cast<const T*>(a.table) + (size_t)(key == kNone ? 0 : key) * a.D;
  const int step = per_row * E;
  for (int c = lane * E; c < a.D; c += NV * step) {
    float f[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[v][e] = 0.f;
      if (key != kNone && c + v * step < a.D) load_e<T, E>(in + c + v * step, f[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[v][e] *= a.scale;
      if (c + v * step < a.D) store_e<T, E>(out + c + v * step, f[v]);
    }
  }
}

// ----------------------------------------------------------------- ordering
// Ranks kRankKeys keys of one section, a warp a share of the section's keys.  Keys before the
// block's own count when they are not greater, those behind when they are smaller: equal tokens keep
// their order.
__global__ void __launch_bounds__(kRankKeys * kRankParts) rank_tokens(const __grid_constant__ EmbedArgs a) {
  __shared__ int keys[kSection];
  __shared__ int parts[kRankParts][kRankKeys];
  const int blocks_each = a.section / kRankKeys;
  const int64_t first = (int64_t)(blockIdx.x / blocks_each) * a.section;
  const int m = (int)min((int64_t)a.section, a.n - first);
  const int own = (blockIdx.x % blocks_each) * kRankKeys;
  let_next_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_long = 0;
  const int m4 = (m + 3) & ~3;
#pragma unroll 4
  for (int j = threadIdx.x; j < m4; j += kRankKeys * kRankParts)
    keys[j] = j < m ? key_of(a.tokens[first + j], a.V, a.err) : kNone;
  __syncthreads();
  const int k = threadIdx.x % kRankKeys, part = threadIdx.x / kRankKeys;
  const int mine = own + k < m ? keys[own + k] : kNone;
  int c0 = 0, c1 = 0, c2 = 0, c3 = 0;
  const int4* v = reinterpret_cast<const int4*>(keys);
#pragma unroll 4
  for (int j = part; j < own / 4; j += kRankParts) {
    const int4 x = v[j];
    c0 += x.x <= mine;
    c1 += x.y <= mine;
    c2 += x.z <= mine;
    c3 += x.w <= mine;
  }
  for (int j = own + part; j < min(own + kRankKeys, m); j += kRankParts)
    c0 += keys[j] < mine || (keys[j] == mine && j < own + k);
#pragma unroll 4
  for (int j = min(own + kRankKeys, m4) / 4 + part; j < m4 / 4; j += kRankParts) {
    const int4 x = v[j];
    c0 += x.x < mine;
    c1 += x.y < mine;
    c2 += x.z < mine;
    c3 += x.w < mine;
  }
  parts[part][k] = (c0 + c1) + (c2 + c3);
  __syncthreads();
  if (part != 0 || own + k >= m) return;
  int before = 0;
#pragma unroll
  for (int p = 0; p < kRankParts; ++p) before += parts[p][k];
  const int64_t at = first + before;
  if (a.n <= a.section) {
    a.sorted[at] = mine;
    a.order[at] = own + k;
  } else {
    a.sec_sorted[at] = mine;
    a.sec_order[at] = (int)first + own + k;
  }
}

// Four sections' searches run side by side: each is a chain of dependent loads.
constexpr int kSearches = 4;
__global__ void __launch_bounds__(128) merge_ranks(const __grid_constant__ EmbedArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= a.n) return;
  const int key = a.sec_sorted[j], mine = (int)(j / a.section);
  const int sections = (int)((a.n + a.section - 1) / a.section);
  int64_t at = j % a.section;
  for (int s0 = 0; s0 < sections; s0 += kSearches) {
    int lo[kSearches], hi[kSearches];
#pragma unroll
    for (int u = 0; u < kSearches; ++u) {
      const int s = s0 + u;
      lo[u] = 0;
      hi[u] = s < sections && s != mine ? (int)min((int64_t)a.section, a.n - (int64_t)s * a.section) : 0;
    }
    for (int left = a.section; left > 0; left >>= 1) {  // a section's keys below `key`, up to it in those before
#pragma unroll
      for (int u = 0; u < kSearches; ++u) {
        if (lo[u] >= hi[u]) continue;
        const int mid = (lo[u] + hi[u]) >> 1, x = a.sec_sorted[(int64_t)(s0 + u) * a.section + mid];
        if (x < key || (s0 + u < mine && x == key))
          lo[u] = mid + 1;
        else
          hi[u] = mid;
      }
    }
#pragma unroll
    for (int u = 0; u < kSearches; ++u) at += lo[u];
  }
  a.sorted[at] = key;
  a.order[at] = a.sec_order[j];
}

// ------------------------------------------------------------------ sums
// Where the partial sum of a piece of window w is kept: one may come from the window before (it
// starts the window), one more may go on into the next.
__device__ __forceinline__ size_t piece_slot(int64_t w, bool first) { return (size_t)w * 2 + (first ? 1 : 0); }

// NV vectors of E elements a thread.  The rows of the tile and the rows of the gradient that they
// will be added to are all asked for before the first is used.
template <typename T, int E, int NV>
__global__ void __launch_bounds__(512) sum_runs(const __grid_constant__ EmbedArgs a) {
  constexpr int R = kTileRows;
  __shared__ int rows[kWindow], keys[kWindow + 2];  // from the tile's first row to its window's end; keys[0]: before it
  wait_for_launch_before();
  let_next_launch();
  const int64_t tile = (int64_t)blockIdx.x * R;
  const int64_t window = tile / kWindow;
  const int with = (int)(min((window + 1) * kWindow, a.n) - tile), here = min(R, with);
  for (int j = threadIdx.x; j < with + 2; j += blockDim.x) {
    const int64_t p = tile + j - 1;
    keys[j] = p >= 0 && p < a.n ? a.sorted[p] : kNone;
    if (j < with) rows[j] = a.order[tile + j];
  }
  __syncthreads();
  const int c0 = blockIdx.y * blockDim.x * E * NV + threadIdx.x * E, step = blockDim.x * E;
  if (c0 >= a.D) return;
  const T* d_out = reinterpret_cast<const T*>(a.d_out);
  // row j starts a piece: another token than before, or the first row of a window
  auto starts = [&](int j) { return keys[j + 1] != keys[j] || (j == 0 && tile % kWindow == 0); };
  auto row_ptr = [&](int j, int v) { return d_out + (size_t)rows[j] * a.D + c0 + v * step; };
  float raw[R][NV][E], old[R][NV][E];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const bool has = j < here && keys[j + 1] != kNone;
    // whether a piece that starts here is its token's only one cannot be known yet: if it is not, its old
    // row is read for nothing
    const bool direct = has && a.accumulate && keys[j + 1] != keys[j];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < E; ++e) raw[j][v][e] = old[j][v][e] = 0.f;
      if (has && c0 + v * step < a.D) load_e<T, E>(row_ptr(j, v), raw[j][v]);
      if (direct && c0 + v * step < a.D) load_e<float, E>(a.d_table + (size_t)keys[j + 1] * a.D + c0 + v * step, old[j][v]);
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j >= here || keys[j + 1] == kNone || !starts(j)) continue;
    const int key = keys[j + 1];
    float sum[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[v][e] = raw[j][v][e];
    int end = j + 1;
#pragma unroll
    for (int u = j + 1; u < R; ++u) {
      if (end != u || u >= here || keys[u + 1] != key) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[v][e] += raw[u][v][e];
      end = u + 1;
    }
    if (end == R) {  // on behind the tile
      int stop = end;
      while (stop < with && keys[stop + 1] == key) ++stop;
      for (; end < stop; end += 4) {
        float f[4][NV][E];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int e = 0; e < E; ++e) f[u][v][e] = 0.f;
            if (end + u < stop && c0 + v * step < a.D) load_e<T, E>(row_ptr(end + u, v), f[u][v]);
          }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) sum[v][e] += f[u][v][e];
      }
      end = stop;
    }
    const bool first = keys[j] != key, last = keys[end + 1] != key;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (c0 + v * step >= a.D) continue;
      if (first && last) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum[v][e] = fmaf(a.scale, sum[v][e], old[j][v][e]);
        store_e<float, E>(a.d_table + (size_t)key * a.D + c0 + v * step, sum[v]);
      } else {
        store_e<float, E>(a.part + piece_slot(window, first) * a.pitch + c0 + v * step, sum[v]);
      }
    }
    // the token's last piece tells the join about it (in any order: each has a row of its own)
    if (last && !first && blockIdx.y == 0 && threadIdx.x == 0)
      a.long_runs[atomicAdd(a.n_long, 1)] = make_int2(key, (int)window);
  }
}

// An item is 64 columns of one token with pieces in several windows.  Each of the block's groups of
// threads sums a share of the pieces, the shares are added in order.
constexpr int kJoinCols = 64, kJoinGroups = 8;
__global__ void __launch_bounds__(kJoinCols * kJoinGroups) join_pieces(const __grid_constant__ EmbedArgs a) {
  __shared__ float share[kJoinGroups][kJoinCols];
  wait_for_launch_before();
  const int chunks = (a.D + kJoinCols - 1) / kJoinCols;
  const int64_t items = (int64_t)*a.n_long * chunks;
  const int g = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols, lane = threadIdx.x % 32;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int2 run = a.long_runs[it / chunks];
    const int key = run.x, c = (int)(it % chunks) * kJoinCols + col;
    // first window: the one before the last whose first row is not a continuation (every warp for itself)
    int begin = run.y;
    for (;;) {
      const int w = begin - lane;
      const bool goes_back = w > 0 && a.sorted[(int64_t)w * kWindow - 1] == key;
      const unsigned stops = __ballot_sync(0xffffffffu, !goes_back);
      if (stops) {
        begin -= __ffs(stops) - 1;
        break;
      }
      begin -= 32;
    }
    const int pieces = run.y - begin + 1, per = (pieces + kJoinGroups - 1) / kJoinGroups;
    float sum = 0.f;
    if (c < a.D) {
      const int end = min(pieces, (g + 1) * per);
#pragma unroll 4
      for (int k = g * per; k < end; ++k) sum += a.part[piece_slot(begin + k, k == 0) * a.pitch + c];
    }
    share[g][col] = sum;
    __syncthreads();
    if (g == 0 && c < a.D) {
#pragma unroll
      for (int x = 1; x < kJoinGroups; ++x) sum += share[x][col];
      float* to = a.d_table + (size_t)key * a.D + c;
      *to = fmaf(a.scale, sum, a.accumulate ? *to : 0.f);
    }
    __syncthreads();
  }
}

template <typename K>
cudaError_t launch_after(K kernel, dim3 grid, int threads, const EmbedArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;  // a dependent launch: its set-up overlaps the end of the one before
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int E, int NV>
cudaError_t forward(EmbedArgs& a, cudaStream_t st) {
  const int vecs = (a.D + E * NV - 1) / (E * NV);
  const int per_row = (int)std::min<size_t>(256, align_up((size_t)vecs, 32));
  a.rows = 256 / per_row;
  while (a.rows > 1 && (a.n + a.rows - 1) / a.rows < 2 * device_sm_count()) a.rows /= 2;
  count_launches(1);
  embed_rows<T, E, NV><<<(unsigned)((a.n + a.rows - 1) / a.rows), per_row * a.rows, 0, st>>>(a);
  return cudaGetLastError();
}

// Keys ranked against each other: all of a chunk's where that is one launch less, else half as many,
// which halves the comparisons.
int section_of(int64_t n) { return n <= kSection ? kSection : kSection / 2; }

template <typename T, int E, int NV>
cudaError_t backward(const EmbedArgs& a, cudaStream_t st) {
  const int64_t sections = (a.n + a.section - 1) / a.section;
  const int64_t last = a.n - (sections - 1) * a.section;
  const unsigned ranks = (unsigned)((sections - 1) * (a.section / kRankKeys) + (last + kRankKeys - 1) / kRankKeys);
  count_launches(1);
  rank_tokens<<<ranks, kRankKeys * kRankParts, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (sections > 1) {
    e = launch_after(merge_ranks, dim3((unsigned)((a.n + 127) / 128)), 128, a, st);
    if (e != cudaSuccess) return e;
  }
  const int vecs = (a.D + E * NV - 1) / (E * NV);
  const int slabs = (vecs + 511) / 512;
  const int threads = (int)align_up((size_t)(vecs + slabs - 1) / slabs, 32);
  e = launch_after(sum_runs<T, E, NV>, dim3((unsigned)((a.n + kTileRows - 1) / kTileRows), (unsigned)slabs), threads, a,
                   st);
  if (e != cudaSuccess || a.n <= kWindow) return e;
  // at most a run goes on from each window into the next
  const int64_t most = ((a.n - 1) / kWindow) * ((a.D + kJoinCols - 1) / kJoinCols);
  return launch_after(join_pieces, dim3((unsigned)std::min<int64_t>(most, 4 * device_sm_count())),
                      kJoinCols * kJoinGroups, a, st);
}

template <typename T>
cudaError_t forward_any(EmbedArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.table) && on16(a.out) ? forward<T, E, 2>(a, st) : forward<T, 1, 4>(a, st);
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
  s.sec_order = take(n > section_of(n) ? (size_t)n * 4 : 0);
  s.sec_sorted = take(n > section_of(n) ? (size_t)n * 4 : 0);
  s.n_long = take(4);
  const size_t windows = (size_t)(n + kWindow - 1) / kWindow;
  s.long_runs = take(windows * 8);
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
  a.section = section_of(n);
  a.n_long = reinterpret_cast<int*>(base + w.n_long);
  a.long_runs = reinterpret_cast<int2*>(base + w.long_runs);
  a.part = reinterpret_cast<float*>(base + w.part);
  a.pitch = w.pitch;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? backward_any<float>(a, st) : backward_any<__nv_bfloat16>(a, st));
}

}  // extern "C"
