// Token embeddings at the front of a model, and their gradient by sorted tokens.
//
//   out[i, :]  = scale * table[t_i, :]                    (0 where there is no token, t_i < 0)
//   dT[t, :]  += scale * sum of d_out[i, :] over the rows i with t_i = t, in row order
//
// Forward: one pass, a row a group of threads; bound by HBM (distinct rows read, all written).
//
// Backward: rows of one token are summed by one owner in row order, so there are no float
// atomics and the gradient is the same bits on every run.  Three launches:
//   rank_tokens   the stable order of the tokens.  A key's rank among the keys of its section
//                 (up to kSection rows) is counted directly, the number of keys that come before
//                 it: sorting by passes would need several dependent launches for a chunk of a
//                 few thousand tokens.
//   merge_ranks   where there are several sections: a key's rank among all keys is the sum of its
//                 places in every section, found by binary search.
//   sum_runs      sorted rows are cut into runs of one token and these into pieces of kPiece
//                 rows.  A piece is summed in fp32 by the block in whose tile it starts; a run of
//                 one piece goes straight to its row of the table's gradient.
//   join_pieces   the pieces of longer runs, summed in order.
#include <climits>

#include "attn_common.cuh"
#include "embed.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kSection = 8192;  // keys ranked against each other: 32 KB of shared memory
constexpr int kRankKeys = 64;   // keys a block ranks
constexpr int kRankParts = 4;   // threads that share the comparisons of one key
constexpr int kPiece = 64;      // rows a piece has at most
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
// Rows of a block: `rows` of them at a time, blockDim.x / rows threads each.
template <typename T, int E>
__global__ void __launch_bounds__(512) embed_rows(const __grid_constant__ EmbedArgs a) {
  const int per_row = blockDim.x / a.rows, r = threadIdx.x / per_row, lane = threadIdx.x % per_row;
  const int64_t i = (int64_t)blockIdx.x * a.rows + r;
  if (r >= a.rows || i >= a.n) return;
  const int key = key_of(a.tokens[i], a.V, a.err);
  T* out = reinterpret_cast<T*>(a.out) + (size_t)i * a.D;
  const T* in = reinterpret_cast<const T*>(a.table) + (size_t)(key == kNone ? 0 : key) * a.D;
  for (int c = lane * E; c < a.D; c += per_row * E) {
    float f[E];
    if (key == kNone) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.f;
    } else {
      load_e<T, E>(in + c, f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] *= a.scale;
    }
    store_e<T, E>(out + c, f);
  }
}

// ----------------------------------------------------------------- ordering
// Ranks kRankKeys keys of one section.  Keys before the block's own count when they are not
// greater, those behind when they are smaller: equal tokens keep their order.
__global__ void __launch_bounds__(kRankKeys * kRankParts) rank_tokens(const __grid_constant__ EmbedArgs a) {
  __shared__ int keys[kSection];
  __shared__ int parts[kRankParts][kRankKeys];
  const int blocks_each = kSection / kRankKeys;
  const int64_t first = (int64_t)(blockIdx.x / blocks_each) * kSection;
  const int m = (int)min((int64_t)kSection, a.n - first);
  const int own = (blockIdx.x % blocks_each) * kRankKeys;
  let_next_launch();
  const int m4 = (m + 3) & ~3;
  for (int j = threadIdx.x; j < m4; j += blockDim.x) keys[j] = j < m ? key_of(a.tokens[first + j], a.V, a.err) : kNone;
  __syncthreads();
  const int k = threadIdx.x % kRankKeys, part = threadIdx.x / kRankKeys;
  const int mine = own + k < m ? keys[own + k] : kNone;
  int before = 0;
  const int4* v = reinterpret_cast<const int4*>(keys);
  for (int j = part; j < own / 4; j += kRankParts) {
    const int4 x = v[j];
    before += (x.x <= mine) + (x.y <= mine) + (x.z <= mine) + (x.w <= mine);
  }
  const int end = min(own + kRankKeys, m4);
  for (int j = own + part; j < min(own + kRankKeys, m); j += kRankParts)
    before += keys[j] < mine || (keys[j] == mine && j < own + k);
  for (int j = end / 4 + part; j < m4 / 4; j += kRankParts) {
    const int4 x = v[j];
    before += (x.x < mine) + (x.y < mine) + (x.z < mine) + (x.w < mine);
  }
  parts[part][k] = before;
  __syncthreads();
  if (part != 0 || own + k >= m) return;
#pragma unroll
  for (int p = 1; p < kRankParts; ++p) before += parts[p][k];
  const int64_t at = first + before;
  if (a.n <= kSection) {
    a.sorted[at] = mine;
    a.order[at] = own + k;
  } else {
    a.sec_sorted[at] = mine;
    a.sec_order[at] = (int)first + own + k;
  }
}

// Number of keys of the ascending list v[0, m) below `key` (or_equal: not above it).
__device__ __forceinline__ int count_below(const int* v, int m, int key, bool or_equal) {
  int lo = 0, hi = m;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] < key || (or_equal && v[mid] == key))
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(256) merge_ranks(const __grid_constant__ EmbedArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= a.n) return;
  const int key = a.sec_sorted[j], mine = (int)(j / kSection);
  const int sections = (int)((a.n + kSection - 1) / kSection);
  int64_t at = j % kSection;
  for (int s = 0; s < sections; ++s) {
    if (s == mine) continue;
    const int64_t first = (int64_t)s * kSection;
    at += count_below(a.sec_sorted + first, (int)min((int64_t)kSection, a.n - first), key, s < mine);
  }
  a.sorted[at] = key;
  a.order[at] = a.sec_order[j];
}

// ------------------------------------------------------------------ sums
// Where the partial sum of a piece is kept: of the long runs, at most one starts in 64 rows and
// at most one is continued there by a piece that starts in them.
__device__ __forceinline__ size_t piece_slot(int64_t start, bool first) { return (size_t)(start / kPiece) * 2 + (first ? 1 : 0); }

// First sorted row of the run that row p belongs to.
__device__ __forceinline__ int64_t run_start(const int* sorted, int64_t p, int key) {
  if (p == 0 || sorted[p - 1] != key) return p;
  int64_t lo = 0, hi = p - 1;  // sorted[hi] == key
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (sorted[mid] < key)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <typename T, int E>
__global__ void __launch_bounds__(512) sum_runs(const __grid_constant__ EmbedArgs a) {
  __shared__ int rows[kTileRows + kPiece], keys[kTileRows + kPiece + 1];
  __shared__ int64_t s_begin;
  wait_for_launch_before();
  let_next_launch();
  const int64_t tile = (int64_t)blockIdx.x * kTileRows;
  const int here = (int)min((int64_t)kTileRows, a.n - tile), with = (int)min((int64_t)(kTileRows + kPiece), a.n - tile);
  for (int j = threadIdx.x; j <= with; j += blockDim.x) {
    keys[j] = tile + j < a.n ? a.sorted[tile + j] : kNone;
    if (j < with) rows[j] = a.order[tile + j];
  }
  if (threadIdx.x == 0) {
    const int k = a.sorted[tile];
    s_begin = k == kNone ? tile : run_start(a.sorted, tile, k);
  }
  __syncthreads();
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  if (c >= a.D) return;
  const T* d_out = reinterpret_cast<const T*>(a.d_out) + c;
  int64_t begin = s_begin;  // of the run at j
  int j = (int)((kPiece - (tile - begin) % kPiece) % kPiece);  // first piece that starts in this tile
  // the run may end before that row
  if (j > 0) {
    const int k0 = keys[0];
    int e = 1;
    while (e < j && e < here && keys[e] == k0) ++e;
    if (e < j) {
      j = e;
      begin = tile + e;
    } else if (j < here && keys[j] != k0) {
      begin = tile + j;
    }
  }
  while (j < here) {
    const int key = keys[j];
    if (key == kNone) return;
    int e = j + 1;  // end of the piece
    while (e - j < kPiece && e < with && keys[e] == key) ++e;
    const int64_t start = tile + j;
    const bool first = start == begin, last = keys[e] != key;
    float* to = a.d_table + (size_t)key * a.D + c;
    float old[E], sum[E];
#pragma unroll
    for (int x = 0; x < E; ++x) old[x] = sum[x] = 0.f;
    if (first && last && a.accumulate) load_e<float, E>(to, old);
    int r = j;
    for (; r + 4 <= e; r += 4) {
      float f[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) load_e<T, E>(d_out + (size_t)rows[r + u] * a.D, f[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < E; ++x) sum[x] += f[u][x];
    }
    for (; r < e; ++r) {
      float f[E];
      load_e<T, E>(d_out + (size_t)rows[r] * a.D, f);
#pragma unroll
      for (int x = 0; x < E; ++x) sum[x] += f[x];
    }
    if (first && last) {
#pragma unroll
      for (int x = 0; x < E; ++x) old[x] = fmaf(a.scale, sum[x], old[x]);
      store_e<float, E>(to, old);
    } else {
      store_e<float, E>(a.part + piece_slot(start, first) * a.pitch + c, sum);
    }
    j = e;
    if (last) begin = tile + e;
  }
}

// One block a window of kPiece sorted rows: joins the long run that starts there, if one does.
// Each of the block's groups of threads sums a share of the pieces, the shares are added in order.
constexpr int kJoinCols = 64, kJoinGroups = 8;
__global__ void __launch_bounds__(kJoinCols * kJoinGroups) join_pieces(const __grid_constant__ EmbedArgs a) {
  __shared__ int64_t s_start, s_end;
  __shared__ float share[kJoinGroups][kJoinCols];
  if (threadIdx.x == 0) s_start = -1;
  __syncthreads();
  wait_for_launch_before();
  const int64_t window = (int64_t)blockIdx.x * kPiece;
  if (threadIdx.x < kPiece) {
    const int64_t p = window + threadIdx.x;
    if (p + kPiece < a.n) {
      const int key = a.sorted[p];
      if (key != kNone && (p == 0 || a.sorted[p - 1] != key) && a.sorted[p + kPiece] == key) {  // more than a piece
        int64_t lo = p + kPiece + 1, hi = a.n;  // end of the run
        while (lo < hi) {
          const int64_t mid = (lo + hi) >> 1;
          if (a.sorted[mid] == key)
            lo = mid + 1;
          else
            hi = mid;
        }
        s_start = p;
        s_end = lo;
      }
    }
  }
  __syncthreads();
  if (s_start < 0) return;
  const int64_t start = s_start;
  const int pieces = (int)((s_end - start + kPiece - 1) / kPiece);
  const int g = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols, per = (pieces + kJoinGroups - 1) / kJoinGroups;
  for (int c0 = blockIdx.y * kJoinCols; c0 < a.D; c0 += gridDim.y * kJoinCols) {
    const int c = c0 + col;
    float sum = 0.f;
    if (c < a.D) {
      const int end = min(pieces, (g + 1) * per);
#pragma unroll 4
      for (int k = g * per; k < end; ++k)
        sum += a.part[piece_slot(start + (int64_t)k * kPiece, k == 0) * a.pitch + c];
    }
    share[g][col] = sum;
    __syncthreads();
    if (g == 0 && c < a.D) {
#pragma unroll
      for (int x = 1; x < kJoinGroups; ++x) sum += share[x][col];
      float* to = a.d_table + (size_t)a.sorted[start] * a.D + c;
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

template <typename T, int E>
cudaError_t forward(EmbedArgs& a, cudaStream_t st) {
  const int vecs = (a.D + E - 1) / E;
  const int per_row = (int)std::min<size_t>(256, align_up((size_t)vecs, 32));
  a.rows = 256 / per_row;
  while (a.rows > 1 && (a.n + a.rows - 1) / a.rows < 2 * device_sm_count()) a.rows /= 2;
  count_launches(1);
  embed_rows<T, E><<<(unsigned)((a.n + a.rows - 1) / a.rows), per_row * a.rows, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int E>
cudaError_t backward(const EmbedArgs& a, cudaStream_t st) {
  const int64_t sections = (a.n + kSection - 1) / kSection;
  const int64_t last = a.n - (sections - 1) * kSection;
  const unsigned ranks = (unsigned)((sections - 1) * (kSection / kRankKeys) + (last + kRankKeys - 1) / kRankKeys);
  count_launches(1);
  rank_tokens<<<ranks, kRankKeys * kRankParts, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (sections > 1) {
    e = launch_after(merge_ranks, dim3((unsigned)((a.n + 255) / 256)), 256, a, st);
    if (e != cudaSuccess) return e;
  }
  const int vecs = (a.D + E - 1) / E;
  const int slabs = (vecs + 511) / 512;
  const int threads = (int)align_up((size_t)(vecs + slabs - 1) / slabs, 32);
  e = launch_after(sum_runs<T, E>, dim3((unsigned)((a.n + kTileRows - 1) / kTileRows), (unsigned)slabs), threads, a, st);
  if (e != cudaSuccess || a.n <= kPiece) return e;
  const int windows = (int)((a.n + kPiece - 1) / kPiece);
  return launch_after(join_pieces, dim3((unsigned)windows, (unsigned)std::min(16, (a.D + kJoinCols - 1) / kJoinCols)),
                      kJoinCols * kJoinGroups, a, st);
}

template <typename T>
cudaError_t forward_any(EmbedArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.table) && on16(a.out) ? forward<T, E>(a, st) : forward<T, 1>(a, st);
}
template <typename T>
cudaError_t backward_any(const EmbedArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.d_out) && on16(a.d_table) ? backward<T, E>(a, st) : backward<T, 1>(a, st);
}

// Workspace: order, sorted [n] int each (twice for several sections), then the pieces' sums.
struct EmbedSpace {
  size_t order, sorted, sec_order, sec_sorted, part, bytes;
  int64_t pitch;
};
EmbedSpace embed_space(int64_t n, int D) {
  EmbedSpace s;
  const size_t list = align_up((size_t)n * 4, 256);
  s.order = 0;
  s.sorted = list;
  s.sec_order = 2 * list;
  s.sec_sorted = 3 * list;
  s.part = n > kSection ? 4 * list : 2 * list;
  s.pitch = (int64_t)align_up((size_t)D, 4);
  s.bytes = s.part + (n > kPiece ? ((size_t)n / kPiece + 1) * 2 * s.pitch * 4 : 0);
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
  a.part = reinterpret_cast<float*>(base + w.part);
  a.pitch = w.pitch;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? backward_any<float>(a, st) : backward_any<__nv_bfloat16>(a, st));
}

}  // extern "C"
