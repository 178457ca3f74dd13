// Softmax cross entropy of the output projection over a large vocabulary, without the logits.
//
//   z = x W^T, z' = c tanh(z / c) with a cap c;  lse_i = log sum_v exp z'_iv;  loss_i = lse_i - z'_i,t
//   dz = g_i (exp(z' - lse) - [v = t]) (1 - (z'/c)^2);  dx = s dz W;  dW (+)= s dz^T x
//
// The rows that have a target are gathered first (rows without one cost nothing and what they hold
// is never read).  Forward: one product, whose tiles leave a maximum and a sum of exponentials for
// every row and 128 columns (head_gemm.cuh), and a join of those.  Backward, piece by piece of the
// vocabulary: the logits again with dz stored in bf16, then dx += dz W and dw = dz^T x.  A piece is
// as many columns as keep dz within kDzBytes, so that the sums of dx go through memory a few times
// only.  W is read in place by the copy engines; fp32, and rows off 16 bytes, in staged pieces.
#include <climits>
#include <cmath>

#include "head_gemm.cuh"
#include "head_plan.h"

namespace oomb {
namespace head {
namespace {

constexpr int kMaxWidth = 65536;
// Row tiles that share the columns' tiles in L2: 4096 and 8192 rows on 131072 x 3584, 4 2497 and 19528
// us, 8 2366 and 19152, 16 2313 and 18903, 32 2312 and 19813.
constexpr int kGroup = 16;
// Steps of 64 columns summed on the tensor cores: the loss of 4096 such rows is 1.4e-7, 2.0e-7 and
// 3.4e-7 of its size off after 8, 16 and 28 steps (2.5e-6 after all 56), in 2343, 2288 and 2243 us.
// fp32 operands have six products a step and fewer steps, an eighth of a short K for the logits: dx and dw of 300
// rows on 1000 x 256 are off by 7.9e-7 of their size, by four steps 2.6e-6 (82 us, 80); 951 on 32001 x 1000 by
// 6.4e-7, 8.6e-7 (1097 us, 1061).
// Gradients of bf16 operands: a dw in fp32 has its rows summed in such pieces too (65536 rows of one sign are off by
// 4e-4 of their sum without; backward of 8192 rows on 131072 x 3584, dw added in fp32: 13890 to 14160 us, 13870 in
// one sum, 2500 on 57899 x 1664 1140, 1085); what is rounded to bf16 has only sums of more than kChunkBf16 steps, which are cut by less
// than a quarter of a step of bf16 below it.  dz's logits of bf16 operands are one sum up to kDzSteps: it is cut by 5e-6 of a
// logit at most, which is a quarter of a step of dz for logits of 200 (in pieces, 8192 rows on 131072 x 3584 both ways
// 18570 to 18770 us, 1600 of 4001 on 50001 x 2048 under a cap 958 to 984).  Wider rows would form other logits than the
// forward did: probabilities were 1 % off at logits of 160 over 8192 columns, 7 % over 65536.
constexpr int kChunk = 28, kChunkParts = 4, kChunkBf16 = 2048, kDzSteps = 2 * kChunk;

__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ staging
// Three bf16 parts of an fp32 value: their sum is the value (24 bits in parts of 8).
__device__ __forceinline__ void split3(float v, float (&h)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    h[i] = __bfloat162float(__float2bfloat16_rn(v));
    v -= h[i];
  }
}

// Columns [lane E .. of every `lanes` lanes] of a row into its bf16 parts, `plane` elements apart.
template <typename T, bool VEC>
__device__ __forceinline__ void stage_row(const T* in, __nv_bfloat16* out, size_t plane, int D, int lane, int lanes) {
  if constexpr (VEC && sizeof(T) == 2) {
#pragma unroll 4
    for (int c = lane * 8; c < D; c += lanes * 8)
      *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(in + c);
  } else if constexpr (VEC) {
#pragma unroll 2
    for (int c = lane * 8; c < D; c += lanes * 8) {
      const float4 a = *reinterpret_cast<const float4*>(in + c), b = *reinterpret_cast<const float4*>(in + c + 4);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      float h[8][3];
#pragma unroll
      for (int e = 0; e < 8; ++e) split3(v[e], h[e]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint4*>(out + p * plane + c) =
            make_uint4(pack_bf16x2(h[0][p], h[1][p]), pack_bf16x2(h[2][p], h[3][p]), pack_bf16x2(h[4][p], h[5][p]),
                       pack_bf16x2(h[6][p], h[7][p]));
    }
  } else {
    constexpr int B = 8;  // asked for together
    for (int c0 = lane; c0 < D; c0 += lanes * B) {
      T x[B];
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (c0 + u * lanes < D) x[u] = in[c0 + u * lanes];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int c = c0 + u * lanes;
        if (c >= D) continue;
        if constexpr (sizeof(T) == 2) {
          out[c] = x[u];
        } else {
          float h[3];
          split3(x[u], h);
#pragma unroll
          for (int p = 0; p < 3; ++p) out[p * plane + c] = __float2bfloat16_rn(h[p]);
        }
      }
    }
  }
}

struct GatherArgs {
  const void* in;         // x [n, D], or W's rows of the piece
  __nv_bfloat16* out;     // [parts, n, pitch]
  int n, D, pitch;
  // x only
  const int64_t* targets;
  int V;
  int* rows;
  int* count;
  const void* w;          // forward: W and the cap, for the logits of the targets
  int w_vec;
  float cap;
  float* at;              // [n]
  float* loss;            // forward: written in rows without a target
  float* lse;
  void* dx;               // backward: the same
  int most_splits, clusters, tns, steps0;  // backward: parts K of dx may be cut into, clusters of the GPU, tiles of
                                           // columns, steps of K
  uint32_t* err;
};

// A lane's share of the product of a row and its target's row of W; the same columns for every alignment.
template <typename T, bool VEC>
__device__ __forceinline__ float dot_share(const T* x, const T* w, int D, int lane, int lanes) {
  constexpr int E = 16 / sizeof(T);
  float s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = 0.f;
#pragma unroll 4
  for (int c = lane * E; c < D; c += lanes * E) {
    if constexpr (VEC) {
      const uint4 a = *reinterpret_cast<const uint4*>(x + c), b = *reinterpret_cast<const uint4*>(w + c);
#pragma unroll
      for (int e = 0; e < E; ++e)
        s[e] = fmaf(to_float<T>(reinterpret_cast<const T*>(&a)[e]), to_float<T>(reinterpret_cast<const T*>(&b)[e]), s[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + e < D) s[e] = fmaf(to_float<T>(x[c + e]), to_float<T>(w[c + e]), s[e]);
    }
  }
  float v = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) v += s[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Gathers the rows of x that have a target; forward: forms the targets' logits.  A block takes a
// contiguous range of rows; how many rows before it have a target it counts itself, so that one launch is
// enough.
// ROW_WARPS: warps that share a row (all of them where there are few rows).
constexpr int kStageThreads = 256;
template <typename T, bool VEC, int ROW_WARPS>
__global__ void __launch_bounds__(kStageThreads) stage_x(const __grid_constant__ GatherArgs a) {
  __shared__ int warp_sum[kStageThreads / 32], place[kStageThreads];
  __shared__ float shares[kStageThreads / 32];
  wait_for_launch_before();
  let_next_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int begin = (int)((int64_t)a.n * blockIdx.x / gridDim.x), end = (int)((int64_t)a.n * (blockIdx.x + 1) / gridDim.x);
  // sum of one flag a thread over the block; `before`: over the threads before
  auto block_count = [&](int v, int& before) {
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int all = 0, off = 0;
#pragma unroll
    for (int w = 0; w < kStageThreads / 32; ++w) {
      if (w < warp) off += warp_sum[w];
      all += warp_sum[w];
    }
    before = off + inc - v;
    return all;
  };
  int mine = 0, unused;
  constexpr int B = 8;  // asked for together
  for (int i = threadIdx.x; i < begin; i += B * kStageThreads) {
    int64_t t[B];
#pragma unroll
    for (int u = 0; u < B; ++u) t[u] = i + u * kStageThreads < begin ? a.targets[i + u * kStageThreads] : -1;
#pragma unroll
    for (int u = 0; u < B; ++u) mine += t[u] >= 0 && t[u] < a.V;
  }
  int at = block_count(mine, unused);
  const size_t plane = (size_t)a.n * a.pitch;
  for (int i0 = begin; i0 < end; i0 += kStageThreads) {
    const int i = i0 + threadIdx.x;
    const int64_t t = i < end ? a.targets[i] : -1;
    if (t >= a.V) atomicOr(a.err, OOMB_DEVERR_TOKEN);
    const int has = t >= 0 && t < a.V;
    int before;
    const int all = block_count(has, before);
    place[threadIdx.x] = has ? at + before : -1;
    if (has) a.rows[at + before] = i;
    if (i < end && !has && a.loss) a.loss[i] = a.lse[i] = 0.f;
    __syncthreads();
    constexpr int kGroups = kStageThreads / 32 / ROW_WARPS, kLanes = 32 * ROW_WARPS;
    const int member = threadIdx.x % kLanes;
    for (int j = threadIdx.x / kLanes; j < min(kStageThreads, end - i0); j += kGroups) {
      const int to = place[j];
      if (to >= 0) {
        const T* x = reinterpret_cast<const T*>(a.in) + (size_t)(i0 + j) * a.D;
        stage_row<T, VEC>(x, a.out + (size_t)to * a.pitch, plane, a.D, member, kLanes);
        if (a.at) {
          const T* w = reinterpret_cast<const T*>(a.w) + (size_t)a.targets[i0 + j] * a.D;
          float z = VEC && a.w_vec ? dot_share<T, VEC>(x, w, a.D, member, kLanes)
                                   : dot_share<T, false>(x, w, a.D, member, kLanes);
          if constexpr (ROW_WARPS > 1) {
            __syncthreads();
            if (lane == 0) shares[warp] = z;
            __syncthreads();
            z = 0.f;
#pragma unroll
            for (int u = 0; u < ROW_WARPS; ++u) z += shares[u];
          }
          if (a.cap > 0.f) z = a.cap * tanhf(z / a.cap);
          if (member == 0) a.at[to] = z;
        }
      } else if (a.dx) {
        T* d = reinterpret_cast<T*>(a.dx) + (size_t)(i0 + j) * a.D;
        for (int c = member; c < a.D; c += kLanes) d[c] = from_float<T>(0.f);
      }
    }
    at += all;
  }
  if (blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x == 0) a.count[0] = at;
    if (warp == 0 && a.most_splits > 0) {
      // parts that K of dx is cut into: those that leave the clusters idle for the least time, of 8 steps at
      // least; a lane tries two
      const int dx_tiles = (at + kTile - 1) / kTile * a.tns;
      float least = 1e30f;
      int best = 1;
      for (int s = lane + 1; s <= a.most_splits; s += 32) {
        if (s > 1 && s * 8 > a.steps0) break;
        // rounds of the parts, and what writing and adding one more of them costs
        const float cost = (float)((dx_tiles * s + a.clusters - 1) / a.clusters) / (float)s + 0.004f * (float)s;
        if (cost < least) {
          least = cost;
          best = s;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float c2 = __shfl_xor_sync(0xffffffffu, least, o);
        const int b2 = __shfl_xor_sync(0xffffffffu, best, o);
        if (c2 < least || (c2 == least && b2 < best)) {
          least = c2;
          best = b2;
        }
      }
      if (lane == 0) a.count[1] = best;
    }
    // rows up to the next step of K are read by the product over rows
    const int tail = min(a.n, (at + kStep - 1) / kStep * kStep);
    const size_t many = (size_t)(tail - at) * a.pitch / 8;  // rows of a multiple of 8 elements, on 16 bytes
    for (int p = 0; p < (sizeof(T) == 2 ? 1 : 3); ++p)
      for (size_t k = threadIdx.x; k < many; k += kStageThreads)
        reinterpret_cast<uint4*>(a.out + p * plane + (size_t)at * a.pitch)[k] = make_uint4(0, 0, 0, 0);
  }
}

// Rows of W that are not read in place, a warp 1024 columns of one.
constexpr int kStageCols = 1024;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) stage_w(const __grid_constant__ GatherArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int chunks = (a.D + kStageCols - 1) / kStageCols, lane = threadIdx.x % 32;
  const int64_t items = (int64_t)a.n * chunks;
  for (int64_t it = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t r = it / chunks;
    const int c = (int)(it % chunks) * kStageCols;
    stage_row<T, VEC>(reinterpret_cast<const T*>(a.in) + (size_t)r * a.D + c, a.out + (size_t)r * a.pitch + c,
                      (size_t)a.n * a.pitch, min(kStageCols, a.D - c), lane, 32);
  }
}

// ------------------------------------------------------------------ joins
// Log-sum-exp of a row from its columns' parts, a warp a row.
__global__ void __launch_bounds__(256) join_lse(const __grid_constant__ GemmArgs a, float* loss, float* lse) {
  wait_for_launch_before();
  let_next_launch();
  const int count = *a.count, lane = threadIdx.x % 32;
  for (int r = blockIdx.x * 8 + threadIdx.x / 32; r < count; r += gridDim.x * 8) {
    const float2* part = a.part + (size_t)r * a.parts;
    float m = -INFINITY, s = 0.f;
#pragma unroll 4
    for (int i = lane; i < a.parts; i += 32) {
      const float2 p = part[i];
      const float to = fmaxf(m, p.x), ref = to == -INFINITY ? 0.f : to;
      s = s * ex2_approx(m - ref) + p.y * ex2_approx(p.x - ref);
      m = to;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.f : to;
      // the same order in both lanes of a pair: every lane gets the same bits
      const float lo = s * ex2_approx(m - ref), hi = s2 * ex2_approx(m2 - ref);
      s = lo + hi;
      m = to;
    }
    if (lane == 0) {
      const int row = a.rows[r];
      loss_of(a.at[r], m, s, loss[row], lse[row]);
    }
  }
}

// Four columns of the splits' sums, added in order, and stored.  (Sums in splits are few enough for 32-bit indices:
// kAccBytes, or a tile a cluster.)  951 rows of
// 1000 in fp32: 10 us, a column a thread 18.
template <typename T>
__device__ __forceinline__ void join_four(const GemmArgs& a, int splits, int64_t plane, const float* acc, T* to, int left,
                                          bool add) {
  constexpr int B = 8;  // asked for together
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < splits; s0 += B) {
    float4 x[B];
#pragma unroll
    for (int u = 0; u < B; ++u)
      x[u] = s0 + u < splits ? *reinterpret_cast<const float4*>(acc + (s0 + u) * plane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < B; ++u) {
      v.x += x[u].x;
      v.y += x[u].y;
      v.z += x[u].z;
      v.w += x[u].w;
    }
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (a.out_vec) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(a.scale * v.x, a.scale * v.y),
                                                 pack_bf16x2(a.scale * v.z, a.scale * v.w));
    } else {
      const float4 o = add ? *reinterpret_cast<const float4*>(to) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(to) = make_float4(fmaf(a.scale, v.x, o.x), fmaf(a.scale, v.y, o.y),
                                                   fmaf(a.scale, v.z, o.z), fmaf(a.scale, v.w, o.w));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) to[e] = from_float<T>(fmaf(a.scale, f[e], add ? to_float<T>(to[e]) : 0.f));
}

// dw of a small piece.
template <typename TW>
__global__ void __launch_bounds__(256) join_dw(const __grid_constant__ GemmArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int quads = (a.out_cols + 3) / 4, total = a.cols * quads;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const int r = i / quads, c = i % quads * 4;
    join_four<TW>(a, a.dw_splits, (int64_t)a.cols * a.acc_pitch, a.acc + (size_t)r * a.acc_pitch + c,
                  reinterpret_cast<TW*>(a.out) + (size_t)(a.v0 + r) * a.out_cols + c, a.out_cols - c, a.accumulate != 0);
  }
}

// dx of few rows.
template <typename T>
__global__ void __launch_bounds__(256) join_dx(const __grid_constant__ GemmArgs a) {
  wait_for_launch_before();
  let_next_launch();
  const int count = a.count[0], splits = a.count[1];
  if (splits == 1) return;  // written already
  const int quads = (a.out_cols + 3) / 4, total = count * quads;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const int r = i / quads, c = i % quads * 4;
    join_four<T>(a, splits, (int64_t)a.n * a.acc_pitch, a.acc + (size_t)r * a.acc_pitch + c,
                 reinterpret_cast<T*>(a.out) + (size_t)a.rows[r] * a.out_cols + c, a.out_cols - c, false);
  }
}

// ------------------------------------------------------------------ host side
int clusters() { return std::max(1, device_sm_count() / 2); }
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Map of a [planes, rows, cols] bf16 array with rows of `pitch` elements, boxes of 64 columns.
bool make_map(CUtensorMap* m, const void* base, uint64_t planes, uint64_t rows, uint64_t cols, uint64_t pitch, int box) {
  auto enc = tc::tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, planes};
  cuuint64_t strides[2] = {pitch * 2, (planes > 1 ? rows : 1) * pitch * 2};
  cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename... A>
cudaError_t launch_after(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;  // a dependent launch: its set-up overlaps the end of the one before
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MODE, bool CHUNKED, int TN>
cudaError_t gemm_of(const CUtensorMap& a, const CUtensorMap& b, const GemmArgs& p, int64_t most_tiles, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)head_gemm<MODE, CHUNKED, TN>, Shape<TN>::smem, set);
  if (e != cudaSuccess) return e;
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(clusters(), most_tiles);
  return launch_after(head_gemm<MODE, CHUNKED, TN>, grid, (unsigned)kThreads, Shape<TN>::smem, st, a, b, p);
}
// chunked: K in pieces of p.chunk steps (the row sums always are).
template <int MODE>
cudaError_t gemm(const CUtensorMap& a, const CUtensorMap& b, const GemmArgs& p, int64_t most_tiles, bool narrow, bool chunked,
                 cudaStream_t st) {
  constexpr bool always = MODE == kLse;
  if constexpr (MODE == kLse || MODE == kDz)
    if (narrow)
      return always || chunked ? gemm_of<MODE, true, kNarrow>(a, b, p, most_tiles, st)
                               : gemm_of<MODE, always, kNarrow>(a, b, p, most_tiles, st);
  return always || chunked ? gemm_of<MODE, true, 256>(a, b, p, most_tiles, st)
                           : gemm_of<MODE, always, 256>(a, b, p, most_tiles, st);
}
// What both directions share: the rows with a target, gathered.  (8192 rows of 3584, with their targets' logits: 31 us by
// four blocks an SM, 49 by two, 46 by six, which take two rounds.)
template <typename T>
cudaError_t gather(const void* x, const GatherArgs& s, cudaStream_t st) {
  const unsigned grid = (unsigned)std::min(s.n, 4 * device_sm_count());
  const bool vec = s.D % 8 == 0 && on16(x), few = s.n <= 4 * (int)grid;
  if (few)
    return vec ? launch_after(stage_x<T, true, 8>, grid, kStageThreads, 0, st, s)
               : launch_after(stage_x<T, false, 8>, grid, kStageThreads, 0, st, s);
  return vec ? launch_after(stage_x<T, true, 1>, grid, kStageThreads, 0, st, s)
             : launch_after(stage_x<T, false, 1>, grid, kStageThreads, 0, st, s);
}

// The map of the piece's rows of W, in place or staged here; row_b: where the piece starts in it.
template <typename T>
cudaError_t weights(const void* w, const Plan& pl, char* ws, int D, int V, int v0, int cols, bool narrow,
                    CUtensorMap* m128, CUtensorMap* m64, int* row_b, cudaStream_t st) {
  const void* base = w;
  uint64_t rows = V, planes = 1, pitch = D;
  *row_b = v0;
  if (pl.staged) {
    GatherArgs s = {};
    s.in = reinterpret_cast<const T*>(w) + (size_t)v0 * D;
    s.out = reinterpret_cast<__nv_bfloat16*>(ws + pl.w);
    s.n = cols;
    s.D = D;
    s.pitch = pl.pitch_d;
    const unsigned grid = (unsigned)std::min(tiles((int64_t)cols * tiles(D, kStageCols), 8), 8 * device_sm_count());
    const cudaError_t e = D % 8 == 0 && on16(s.in) ? launch_after(stage_w<T, true>, grid, 256u, 0, st, s)
                                                   : launch_after(stage_w<T, false>, grid, 256u, 0, st, s);
    if (e != cudaSuccess) return e;
    base = s.out;
    rows = cols;
    planes = pl.parts_of;
    pitch = pl.pitch_d;
    *row_b = 0;
  }
  if (!make_map(m128, base, planes, rows, D, pitch, narrow ? kNarrow / 2 : kHalf)) return cudaErrorInvalidValue;
  if (m64 && !make_map(m64, base, planes, rows, D, pitch, kStep)) return cudaErrorInvalidValue;
  return cudaSuccess;
}

template <typename T>
cudaError_t forward(GemmArgs g, GatherArgs s, const void* w, const Plan& pl, char* ws, int V, float* loss, float* lse,
                    cudaStream_t st) {
  const RowParts of = row_parts(s.n, V, pl.piece, clusters());
  const bool narrow = of.narrow;
  const int tn = narrow ? kNarrow : kTile;
  g.parts = of.parts;
  if (pl.part + (size_t)s.n * g.parts * 8 > pl.bytes) return cudaErrorInvalidValue;  // (never, by the plan)
  cudaError_t e = gather<T>(s.in, s, st);
  if (e != cudaSuccess) return e;
  CUtensorMap mx, mw;
  if (!make_map(&mx, s.out, pl.parts_of, s.n, s.D, s.pitch, kHalf)) return cudaErrorInvalidValue;
  g.steps = tiles(s.D, kStep);
  for (int v0 = 0; v0 < V; v0 += pl.piece) {
    g.v0 = v0;
    g.cols = std::min(pl.piece, V - v0);
    e = weights<T>(w, pl, ws, s.D, V, v0, g.cols, narrow, &mw, nullptr, &g.row_b, st);
    if (e != cudaSuccess) return e;
    g.tns = tiles(g.cols, tn);
    g.part0 = v0 / (tn / 2);
    e = gemm<kLse>(mx, mw, g, (int64_t)tiles(s.n, kTile) * g.tns, narrow, true, st);
    if (e != cudaSuccess) return e;
  }
  return launch_after(join_lse, (unsigned)std::min(tiles(s.n, 8), 8 * device_sm_count()), 256u, 0, st, g, loss, lse);
}

template <typename T>
cudaError_t backward(GemmArgs g, GatherArgs s, const void* w, const Plan& pl, char* ws, int V, void* dx, void* dw,
                     int dw_dtype, int accumulate, cudaStream_t st) {
  s.most_splits = most_splits(s.n, s.D);
  s.clusters = clusters();
  s.tns = tiles(s.D, kTile);
  s.steps0 = tiles(pl.piece, kStep);
  cudaError_t e = gather<T>(s.in, s, st);
  if (e != cudaSuccess) return e;
  const int D = s.D;
  CUtensorMap mx, mx64, mw, mw64, mz, mz64;
  if (!make_map(&mx, s.out, pl.parts_of, s.n, D, s.pitch, kHalf) ||
      !make_map(&mx64, s.out, pl.parts_of, s.n, D, s.pitch, kStep))
    return cudaErrorInvalidValue;
  const int tms = tiles(s.n, kTile), tds = tiles(D, kTile);
  g.pitch = pl.pitch_z;
  GemmArgs gx = g, gw = g;
  gx.chunk = gw.chunk = pl.parts_of > 1 ? kChunkParts : kChunk;  // of a K of their own
  // Whether a sum of `steps` is cut in pieces: always in parts, else where it is longer than a piece and stays fp32, or
  // so long that the cuts come near a half of a step of bf16 all the same.
  auto chunked = [&](int steps, bool fp32) { return pl.parts_of > 1 || steps > (fp32 ? kChunk : kChunkBf16); };
  for (int v0 = 0; v0 < V; v0 += pl.piece) {
    const int cols = std::min(pl.piece, V - v0);
    int row_b;
    const bool narrow = is_narrow(s.n, cols, clusters());
    e = weights<T>(w, pl, ws, D, V, v0, cols, narrow, &mw, &mw64, &row_b, st);
    if (e != cudaSuccess) return e;
    if (!make_map(&mz, g.dz, pl.parts_of, s.n, cols, g.pitch, kHalf) ||
        !make_map(&mz64, g.dz, pl.parts_of, s.n, cols, g.pitch, kStep))
      return cudaErrorInvalidValue;
    for (GemmArgs* a : {&g, &gx, &gw}) {
      a->v0 = v0;
      a->cols = cols;
    }
    g.steps = tiles(D, kStep);
    g.row_b = row_b;
    g.tns = tiles(cols, narrow ? kNarrow : kTile);
    e = gemm<kDz>(mx, mw, g, (int64_t)tms * g.tns, narrow, pl.parts_of > 1 || g.steps > kDzSteps, st);
    if (e != cudaSuccess) return e;
    if (dx) {
      const bool last = v0 + cols == V;
      gx.steps = tiles(cols, kStep);
      gx.row_b = row_b;
      gx.tns = tds;
      gx.add = v0 > 0;
      gx.last = last;
      gx.out = dx;
      gx.out_cols = D;
      gx.out_fp32 = sizeof(T) == 4;
      gx.out_vec = D % (16 / (int)sizeof(T)) == 0 && on16(dx);
      e = gemm<kDx>(mz, mw64, gx, (int64_t)tms * tds * s.most_splits, false, chunked(gx.steps, false), st);
      if (e != cudaSuccess) return e;
      if (last && s.most_splits > 1) {
        e = launch_after(join_dx<T>, (unsigned)std::min<int64_t>(((int64_t)s.n * tiles(D, 4) + 255) / 256, 8 * device_sm_count()),
                         256u, 0, st, gx);
        if (e != cudaSuccess) return e;
      }
    }
    if (dw) {
      gw.tms = tiles(cols, kTile);
      gw.tns = tds;
      gw.out = dw;
      gw.out_cols = D;
      gw.out_fp32 = dw_dtype == OOMB_FP32;
      gw.out_vec = D % (16 / (int)dtype_size(dw_dtype)) == 0 && on16(dw);
      gw.accumulate = accumulate;
      gw.dw_splits = dw_splits(s.n, D, cols, clusters());
      gw.acc = reinterpret_cast<float*>(ws + pl.acc_w);
      e = gemm<kDw>(mz64, mx64, gw, (int64_t)gw.tms * tds * gw.dw_splits, false,
                    chunked(tiles(tiles(s.n, kStep), gw.dw_splits), gw.out_fp32), st);
      if (e == cudaSuccess && gw.dw_splits > 1) {
        const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)cols * tiles(D, 4) + 255) / 256, 8 * device_sm_count());
        e = dw_dtype == OOMB_FP32 ? launch_after(join_dw<float>, grid, 256u, 0, st, gw)
                                  : launch_after(join_dw<__nv_bfloat16>, grid, 256u, 0, st, gw);
      }
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

GemmArgs arguments(const void* x, const int64_t* targets, int n, int D, int V, int dtype, float cap, const Plan& pl,
                   char* ws, uint32_t* err, GatherArgs* s) {
  *s = {};
  s->in = x;
  s->out = reinterpret_cast<__nv_bfloat16*>(ws + pl.x);
  s->n = n;
  s->D = D;
  s->pitch = pl.pitch_d;
  s->targets = targets;
  s->V = V;
  s->rows = reinterpret_cast<int*>(ws + pl.rows);
  s->count = reinterpret_cast<int*>(ws + pl.count);
  s->err = err;
  GemmArgs g = {};
  g.count = s->count;
  g.rows = s->rows;
  g.n = n;
  g.passes = pl.parts_of == 1 ? 1 : 6;
  // about equal pieces of K
  const int steps = tiles(D, kStep), pieces = tiles(steps, kChunk);
  g.chunk = pl.parts_of == 1 ? tiles(steps, pieces) : std::max(1, std::min(kChunkParts, steps / 8));
  g.group = kGroup;
  g.targets = targets;
  g.cap = cap;
  g.part = reinterpret_cast<float2*>(ws + pl.part);
  g.at = reinterpret_cast<const float*>(ws + pl.at);
  g.dz = reinterpret_cast<__nv_bfloat16*>(ws + pl.dz);
  g.acc = reinterpret_cast<float*>(ws + pl.acc);
  g.acc_pitch = (int)align_up((size_t)D, 4);
  g.err = err;
  return g;
}

SmallArgs small_arguments(const void* x, const void* w, const int64_t* targets, int n, int D, int V, float cap,
                          bool backward, char* ws, uint32_t* err) {
  SmallSpace s = {};
  small_space(n, D, V, backward, &s);
  SmallArgs a = {};
  a.x = x;
  a.w = w;
  a.targets = targets;
  a.n = n;
  a.D = D;
  a.V = V;
  a.cap = cap;
  a.err = err;
  a.part = reinterpret_cast<float2*>(ws + s.part);
  a.parts = s.parts;
  a.at = reinterpret_cast<float*>(ws + s.at);
  a.dz = reinterpret_cast<float*>(ws + s.dz);
  a.pitch = s.pitch;
  a.acc = reinterpret_cast<float*>(ws + s.acc);
  a.acc_pitch = s.acc_pitch;
  return a;
}

oomb_status check(const void* x, const void* w, const int64_t* targets, int n, int D, int V, int dtype, float cap,
                  const void* lse, const void* ws, const uint32_t* word) {
  if (!x || !w || !targets || !lse || !word || n <= 0 || D <= 0 || V <= 0 || V > INT_MAX - 1024) return OOMB_ERR_ARG;
  if (!(cap >= 0.f) || cap > 1e30f || (cap > 0.f && cap < 1e-30f)) return OOMB_ERR_ARG;
  if (dtype != OOMB_BF16 && dtype != OOMB_FP32) return OOMB_ERR_DTYPE;
  if (D > kMaxWidth) return OOMB_ERR_UNSUPPORTED;
  const uintptr_t es = dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(w) % es ||
      reinterpret_cast<uintptr_t>(targets) % 8 || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(ws) % 256 || reinterpret_cast<uintptr_t>(word) % 4)
    return OOMB_ERR_ALIGN;
  return OOMB_OK;
}

}  // namespace
}  // namespace head
}  // namespace oomb

using namespace oomb;
using namespace oomb::head;

extern "C" {

size_t oomb_head_loss_workspace(int n, int D, int V, int dtype, int backward) {
  if (n <= 0 || D <= 0 || D > kMaxWidth || V <= 0 || V > INT_MAX - 1024 || (dtype != OOMB_BF16 && dtype != OOMB_FP32)) return 0;
  // grows with n: fewer rows may go either way
  SmallSpace s;
  const int few = std::min(n, small_rows(D, V, dtype));
  return std::max(make_plan(n, D, V, dtype, backward != 0, true, clusters()).bytes,
                  few > 0 ? small_space(few, D, V, backward != 0, &s) : 0);
}

oomb_status oomb_head_loss_fwd(const void* x, const void* w, const int64_t* targets, int n, int D, int V, int dtype,
                               float softcap, float* loss, float* lse, void* workspace, size_t ws_bytes,
                               uint32_t* error_word, void* stream) {
  const oomb_status s = check(x, w, targets, n, D, V, dtype, softcap, lse, workspace, error_word);
  if (s != OOMB_OK) return s;
  if (!loss) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(loss) % 4) return OOMB_ERR_ALIGN;
  if (!workspace || ws_bytes < oomb_head_loss_workspace(n, D, V, dtype, 0)) return OOMB_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  if (n <= small_rows(D, V, dtype)) {
    SmallArgs a = small_arguments(x, w, targets, n, D, V, softcap, false, ws, error_word);
    a.loss = loss;
    a.lse = lse;
    return cuda_status(launch_small_fwd(a, dtype, (cudaStream_t)stream));
  }
  const Plan pl = make_plan(n, D, V, dtype, false, on16(w), clusters());
  GatherArgs st;
  GemmArgs g = arguments(x, targets, n, D, V, dtype, softcap, pl, ws, error_word, &st);
  st.loss = loss;
  st.lse = lse;
  st.w = w;
  st.w_vec = on16(w);
  st.cap = softcap;
  st.at = reinterpret_cast<float*>(ws + pl.at);
  cudaStream_t on = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? forward<float>(g, st, w, pl, ws, V, loss, lse, on)
                                        : forward<__nv_bfloat16>(g, st, w, pl, ws, V, loss, lse, on));
}

oomb_status oomb_head_loss_bwd(const void* x, const void* w, const int64_t* targets, const float* lse,
                               const float* d_loss, float scale, int n, int D, int V, int dtype, float softcap,
                               void* dx, void* dw, int dw_dtype, int accumulate, void* workspace, size_t ws_bytes,
                               uint32_t* error_word, void* stream) {
  const oomb_status s = check(x, w, targets, n, D, V, dtype, softcap, lse, workspace, error_word);
  if (s != OOMB_OK) return s;
  if ((!dx && !dw) || !(scale - scale == 0.f)) return OOMB_ERR_ARG;
  if (dw && dw_dtype != OOMB_FP32 && dw_dtype != dtype) return OOMB_ERR_DTYPE;
  if (accumulate && dw && dw_dtype != OOMB_FP32) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(dx) % dtype_size(dtype) || reinterpret_cast<uintptr_t>(d_loss) % 4 ||
      (dw && reinterpret_cast<uintptr_t>(dw) % dtype_size(dw_dtype)))
    return OOMB_ERR_ALIGN;
  if (!workspace || ws_bytes < oomb_head_loss_workspace(n, D, V, dtype, 1)) return OOMB_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  if (n <= small_rows(D, V, dtype)) {
    SmallArgs a = small_arguments(x, w, targets, n, D, V, softcap, true, ws, error_word);
    a.scale = scale;
    a.lse_in = lse;
    a.d_loss = d_loss;
    a.dx = dx;
    a.dw = dw;
    a.accumulate = accumulate != 0;
    return cuda_status(launch_small_bwd(a, dtype, dw_dtype, (cudaStream_t)stream));
  }
  const Plan pl = make_plan(n, D, V, dtype, true, on16(w), clusters());
  GatherArgs st;
  GemmArgs g = arguments(x, targets, n, D, V, dtype, softcap, pl, ws, error_word, &st);
  st.dx = dx;
  g.lse = lse;
  g.d_loss = d_loss;
  g.scale = scale;
  cudaStream_t on = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? backward<float>(g, st, w, pl, ws, V, dx, dw, dw_dtype, accumulate, on)
                                        : backward<__nv_bfloat16>(g, st, w, pl, ws, V, dx, dw, dw_dtype, accumulate, on));
}

oomb_status oomb_word_check(uint32_t* error_word, void* stream, uint32_t* bits_out) {
  if (!error_word) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(error_word) % 4) return OOMB_ERR_ALIGN;
  uint32_t bits = 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(&bits, error_word, sizeof(bits), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && bits) e = cudaMemsetAsync(error_word, 0, sizeof(bits), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (bits_out) *bits_out = bits;
  if (e != cudaSuccess) return cuda_status(e);
  return bits & OOMB_DEVERR_TIMEOUT ? OOMB_ERR_TIMEOUT : bits ? OOMB_ERR_KERNEL : OOMB_OK;
}

}  // extern "C"
