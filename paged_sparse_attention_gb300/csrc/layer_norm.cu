// Layer norm with weight and bias over rows of D elements.
//
//   mean = sum x / D,  r = 1 / sqrt(sum (x - mean)^2 / D + eps),  xn = (x - mean) r
//   out  = xn w + b
// and, with dy the gradient of out and dx' one that reaches x by another way,
//   t  = dy w,   dx = dx' + r (t - mean(t) - xn mean(t xn))
//   dw = sum dy xn,  db = sum dy   over the rows
// The deviations are squared after the mean is known, from registers, so that a mean that is large against the
// spread costs the variance nothing.  The mean itself is a sum in fp32 and off by a few 2^-24 of itself, which moves
// every deviation alike (a constant row of 33333 came out 1.6 off its bias): the deviations are summed beside their
// squares, or where the row proves far from 0, and their mean is taken off them.  The backward has the mean rounded to
// fp32, and does the same in rows that are further than kFar spreads from 0.
//
// A row is held by one thread block in registers from its load to its stores, so every tensor is
// read once and written once.  A block walks the rows b, b + grid, ... with the next ones' loads in
// flight.  The bytes are HBM's, but the instructions come close behind (a row of 3584 is 14 KB in
// bf16 and at eight columns a thread 3000 warp instructions of an SM that issues 4 a cycle), so a
// thread holds 16 columns, which halves what the two sums of a row cost, and works on pairs of
// fp32.  Backward: the parameter gradients of a block's columns stay in registers and go to the
// workspace once; they are added there in block order, the same bits on every run.
#include <cmath>
#include <type_traits>

#include "attn_common.cuh"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kMaxWidth = 16384;
// |mean| / spread from which a row counts as far from 0: below, a rounded mean is off by 2.4e-7 of a spread, a summed one
// by a few times that.
constexpr float kFar = 4.f;

struct LnArgs {
  const void* x;
  const float* w;
  const float* b;
  void* out;
  float* mean;
  float* rstd;
  const void* dy;
  const void* dx_in;
  void* dx;
  float* dw;
  float* db;
  float* part;  // [2, blocks, D]
  int64_t n;
  int D, accumulate;
  int param_vec;  // w and b start on 16 bytes
  float eps, inv_D;
};

__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Sum of N values over the block; every thread gets them.  `b`: 32 x N floats that no thread still reads from the sum
// before, the entries behind the last warp 0.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* b) {
  const int warps = blockDim.x / 32;
  if constexpr (N == 2) {  // one half of the warp adds the first, the other the second
    const bool up = threadIdx.x & 16;
    float t = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (warps == 1) {
      v[0] = __shfl_sync(0xffffffffu, t, 0);
      v[1] = __shfl_sync(0xffffffffu, t, 16);
      return;
    }
    if (threadIdx.x % 16 == 0) b[(threadIdx.x & 16) * 2 + threadIdx.x / 32] = t;
  } else {
    static_assert(N == 1, "one or two sums");
    v[0] = warp_sum(v[0]);
    if (warps == 1) return;
    if (threadIdx.x % 32 == 0) b[threadIdx.x / 32] = v[0];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < warps; w += 4) {
      const float4 x = *reinterpret_cast<const float4*>(b + i * 32 + w);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    v[i] = (s.x + s.y) + (s.z + s.w);
  }
}
// The same with 2 x 32 x N floats used in turns, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf, int& turn) {
  block_sums<N>(v, buf + turn * 32 * N);
  turn ^= 1;
}

__device__ __forceinline__ uint64_t both(float v) { return f32x2(v, v); }
__device__ __forceinline__ float halves(uint64_t v) {
  float a, b;
  f32x2_split(v, a, b);
  return a + b;
}

// C columns a thread in vectors of E: vector v starts at column (v T + threadIdx.x) E.
template <typename T, int E, int C>
struct Row {
  static constexpr int NV = C / E;
  // the elements as they are stored, so that a row in flight takes few registers
  using Word = typename std::conditional<E == 1, T, uint4>::type;
  Word raw[NV];
  static __device__ __forceinline__ int col(int v) { return (v * (int)blockDim.x + (int)threadIdx.x) * E; }
  __device__ __forceinline__ void clear() {
    unsigned char* p = reinterpret_cast<unsigned char*>(raw);
#pragma unroll
    for (int i = 0; i < (int)sizeof(raw); ++i) p[i] = 0;
  }
  // columns behind the last keep what they hold: 0 from clear()
  __device__ __forceinline__ void load(const T* row, int D) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (col(v) < D) raw[v] = *reinterpret_cast<const Word*>(row + col(v));
  }
  __device__ __forceinline__ void get(uint64_t (&f)[C / 2]) const {
    if constexpr (E == 1) {
#pragma unroll
      for (int k = 0; k < C / 2; ++k) f[k] = f32x2(to_float<T>(raw[2 * k]), to_float<T>(raw[2 * k + 1]));
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint32_t x[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[v * 4 + k] = f32x2(x[k] << 16, x[k] & 0xffff0000u);
        } else {
          f[v * 2] = f32x2(x[0], x[1]);
          f[v * 2 + 1] = f32x2(x[2], x[3]);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T* row, int D, const uint64_t (&f)[C / 2]) {
    float x[C];
#pragma unroll
    for (int k = 0; k < C / 2; ++k) f32x2_split(f[k], x[2 * k], x[2 * k + 1]);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (col(v) >= D) continue;
      if constexpr (E == 1)
        row[col(v)] = from_float<T>(x[v]);
      else if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint4*>(row + col(v)) =
            make_uint4(pack_bf16x2(x[v * 8], x[v * 8 + 1]), pack_bf16x2(x[v * 8 + 2], x[v * 8 + 3]),
                       pack_bf16x2(x[v * 8 + 4], x[v * 8 + 5]), pack_bf16x2(x[v * 8 + 6], x[v * 8 + 7]));
      else
        *reinterpret_cast<float4*>(row + col(v)) = make_float4(x[v * 4], x[v * 4 + 1], x[v * 4 + 2], x[v * 4 + 3]);
    }
  }
};
// fp32 parameters at the same columns
template <int E, int C>
__device__ __forceinline__ void load_param(const float* p, int D, bool vec, uint64_t (&f)[C / 2], float absent) {
  float x[C];
#pragma unroll
  for (int v = 0; v < C / E; ++v) {
    const int c = (v * (int)blockDim.x + (int)threadIdx.x) * E;
    if (E >= 4 && vec && p && c < D) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(p + c + e));
        const float t[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < (E < 4 ? E : 4); ++k) x[v * E + e + k] = t[k];
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[v * E + e] = p && c + e < D ? __ldg(p + c + e) : absent;
    }
  }
#pragma unroll
  for (int k = 0; k < C / 2; ++k) f[k] = f32x2(x[2 * k], x[2 * k + 1]);
}

// AGAIN: the deviations are summed, and squared again, in rows further than kFar spreads from 0 alone.
template <typename T, int E, int C, int THREADS, int MIN_BLOCKS, bool AGAIN>
__global__ void __launch_bounds__(THREADS, MIN_BLOCKS) ln_fwd(const __grid_constant__ LnArgs a) {
  constexpr int H = C / 2;
  using R = Row<T, E, C>;
  __shared__ __align__(16) float buf1[32], buf2[64];  // (a row's two sums: a barrier lies between two uses of either)
  for (int i = threadIdx.x; i < 64; i += blockDim.x) buf1[i % 32] = buf2[i] = 0.f;
  wait_for_launch_before();
  let_next_launch();
  R next;
  next.clear();
  if (blockIdx.x < a.n) next.load(reinterpret_cast<const T*>(a.x) + (size_t)blockIdx.x * a.D, a.D);
  uint64_t w[H], b[H];
  load_param<E, C>(a.w, a.D, a.param_vec, w, 1.f);
  load_param<E, C>(a.b, a.D, a.param_vec, b, 0.f);
  if (blockDim.x > 32) __syncthreads();
  int turn = 0;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    uint64_t x[H];
    next.get(x);
    if (i + gridDim.x < a.n) next.load(reinterpret_cast<const T*>(a.x) + (size_t)(i + gridDim.x) * a.D, a.D);
    uint64_t t = 0;
#pragma unroll
    for (int k = 0; k < H; ++k) t = add2(t, x[k]);
    float s[1] = {halves(t)};
    block_sums<1>(s, buf1);
    float mean = s[0] * a.inv_D;
    uint64_t u;
    auto center = [&](uint64_t by) {  // deviations, 0 behind the last column; t: their squares, u: themselves, summed
      t = u = 0;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        x[k] = add2(x[k], by);
        if constexpr (E == 1) {
          if (R::col(2 * k + 1) >= a.D) x[k] = R::col(2 * k) < a.D ? f32x2((uint32_t)x[k], 0u) : 0;
        } else {
          if (R::col(2 * k / E) >= a.D) x[k] = 0;
        }
        t = fma2(x[k], x[k], t);
        if constexpr (!AGAIN) u = add2(u, x[k]);
      }
    };
    float r;
    if constexpr (AGAIN) {
      float shift = -mean;
#pragma unroll 1
      for (bool again = false;; again = true) {
        center(both(shift));
        s[0] = halves(t);
        block_sums<1>(s, buf2);
        r = rsqrtf(fmaf(s[0], a.inv_D, a.eps));
        if (again || !(fabsf(mean) * r > kFar)) break;  // (the same in every thread of the block)
#pragma unroll
        for (int k = 0; k < H; ++k) u = add2(u, x[k]);
        s[0] = halves(u);
        block_sums<1>(s, buf1);
        shift = -s[0] * a.inv_D;
        mean -= shift;
      }
      const uint64_t rr = both(r);
#pragma unroll
      for (int k = 0; k < H; ++k) x[k] = fma2(mul2(x[k], rr), w[k], b[k]);
    } else {
      center(both(-mean));
      float q[2] = {halves(t), halves(u)};
      block_sums<2>(q, buf2);
      const float off = q[1] * a.inv_D, var = fmaf(-off, off, q[0] * a.inv_D);
      r = rsqrtf((var < 0.f ? 0.f : var) + a.eps);
      mean += off;
      const uint64_t rr = both(r), less = both(-off * r);
#pragma unroll
      for (int k = 0; k < H; ++k) x[k] = fma2(fma2(x[k], rr, less), w[k], b[k]);
    }
    R::store(reinterpret_cast<T*>(a.out) + (size_t)i * a.D, a.D, x);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[i] = mean;
      if (a.rstd) a.rstd[i] = r;
    }
  }
}

// SHARED: the sums of the parameter gradients are in shared memory, where registers are short.
template <typename T, int E, int C, int THREADS, int MIN_BLOCKS, bool SHARED>
__global__ void __launch_bounds__(THREADS, MIN_BLOCKS) ln_bwd(const __grid_constant__ LnArgs a) {
  constexpr int H = C / 2;
  using R = Row<T, E, C>;
  extern __shared__ __align__(16) uint64_t acc[];  // SHARED: [2 H, T]
  __shared__ __align__(16) float buf[128];
  for (int i = threadIdx.x; i < 128; i += blockDim.x) buf[i] = 0.f;
  wait_for_launch_before();
  let_next_launch();
  R nx, ny, nz;
  float n_mean = 0.f, n_rstd = 0.f;
  auto fetch = [&](int64_t i) {
    const size_t at = (size_t)i * a.D;
    nx.load(reinterpret_cast<const T*>(a.x) + at, a.D);
    ny.load(reinterpret_cast<const T*>(a.dy) + at, a.D);
    if (a.dx_in) nz.load(reinterpret_cast<const T*>(a.dx_in) + at, a.D);
    n_mean = a.mean[i];
    n_rstd = a.rstd[i];
  };
  nx.clear();
  ny.clear();
  nz.clear();
  if (blockIdx.x < a.n) fetch(blockIdx.x);
  uint64_t w[H], dw[SHARED ? 1 : H], db[SHARED ? 1 : H];
  load_param<E, C>(a.w, a.D, a.param_vec, w, 1.f);
#pragma unroll
  for (int k = 0; k < H; ++k) {
    if constexpr (SHARED)
      acc[k * blockDim.x + threadIdx.x] = acc[(H + k) * blockDim.x + threadIdx.x] = 0;
    else
      dw[k] = db[k] = 0;
  }
  __syncthreads();
  int turn = 0;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    uint64_t xn[H], t[H];
    nx.get(xn);
    ny.get(t);
    const R z = nz;
    const float mean = n_mean, r = n_rstd;
    if (i + gridDim.x < a.n) fetch(i + gridDim.x);
    const uint64_t rr = both(r), shift = both(-mean);
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      xn[k] = mul2(add2(xn[k], shift), rr);  // columns behind the last: t is 0 there
      if constexpr (SHARED) {
        uint64_t* aw = acc + k * blockDim.x + threadIdx.x;
        uint64_t* ab = acc + (H + k) * blockDim.x + threadIdx.x;
        *aw = fma2(t[k], xn[k], *aw);
        *ab = add2(t[k], *ab);
      } else {
        dw[k] = fma2(t[k], xn[k], dw[k]);
        db[k] = add2(t[k], db[k]);
      }
      t[k] = mul2(t[k], w[k]);
      s0 = add2(s0, t[k]);
      s1 = fma2(t[k], xn[k], s1);
    }
    float s[2] = {halves(s0), halves(s1)};
    block_sums<2>(s, buf, turn);
    if (fabsf(mean) * r > kFar) {  // the rounded mean's share of xn is taken off it, and off what was summed of it
      uint64_t t0 = 0;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int c0 = R::col(2 * k / E) + 2 * k % E, c1 = E == 1 ? R::col(2 * k + 1) : c0;
        if (c0 < a.D) t0 = add2(t0, c1 < a.D ? xn[k] : f32x2((uint32_t)xn[k], 0u));
      }
      float u[2] = {halves(t0), 0.f};  // (two sums, as the buffers are of one size)
      block_sums<2>(u, buf, turn);
      const uint64_t off = both(-u[0] * a.inv_D);
      s[1] = fmaf(-u[0] * a.inv_D, s[0], s[1]);
      const T* y = reinterpret_cast<const T*>(a.dy) + (size_t)i * a.D;  // again: dw has the sum of y xn so far
      auto take_off = [&](int k, uint64_t f) {
        xn[k] = add2(xn[k], off);
        if constexpr (SHARED) {
          uint64_t* aw = acc + k * blockDim.x + threadIdx.x;
          *aw = fma2(off, f, *aw);
        } else {
          dw[k] = fma2(off, f, dw[k]);
        }
      };
      if constexpr (sizeof(T) == 2 && E > 1) {
#pragma unroll
        for (int v = 0; v < R::NV; ++v) {
          asm volatile("" ::: "memory");  // one vector after another, for few registers
          const int c = R::col(v);
          const uint4 q = c < a.D ? *reinterpret_cast<const uint4*>(y + c) : make_uint4(0, 0, 0, 0);
          const uint32_t f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int p = 0; p < 4; ++p) take_off(4 * v + p, f32x2(f[p] << 16, f[p] & 0xffff0000u));
        }
      } else {
#pragma unroll
        for (int k = 0; k < H; ++k) {
          const int c0 = R::col(2 * k / E) + 2 * k % E, c1 = E == 1 ? R::col(2 * k + 1) : c0 + 1;
          take_off(k, f32x2(c0 < a.D ? to_float<T>(y[c0]) : 0.f, c1 < a.D ? to_float<T>(y[c1]) : 0.f));
        }
      }
    }
    const uint64_t m0 = both(-s[0] * a.inv_D), m1 = both(-s[1] * a.inv_D);
#pragma unroll
    for (int k = 0; k < H; ++k) t[k] = mul2(fma2(xn[k], m1, add2(t[k], m0)), rr);
    if (a.dx_in) {
      z.get(xn);
#pragma unroll
      for (int k = 0; k < H; ++k) t[k] = add2(t[k], xn[k]);
    }
    R::store(reinterpret_cast<T*>(a.dx) + (size_t)i * a.D, a.D, t);
  }
  // one block has the whole sums, several leave theirs in the workspace
  const bool whole = gridDim.x == 1;
  float* to[2] = {whole ? a.dw : a.dw ? a.part + (size_t)blockIdx.x * a.D : nullptr,
                  whole ? a.db : a.db ? a.part + ((size_t)gridDim.x + blockIdx.x) * a.D : nullptr};
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (!to[g]) continue;
    uint64_t f[H];
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if constexpr (SHARED)
        f[k] = acc[(g * H + k) * blockDim.x + threadIdx.x];
      else
        f[k] = g == 0 ? dw[k] : db[k];
    }
    float x[C];
#pragma unroll
    for (int k = 0; k < H; ++k) f32x2_split(f[k], x[2 * k], x[2 * k + 1]);
#pragma unroll
    for (int v = 0; v < C / E; ++v)
      if (R::col(v) < a.D)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* p = to[g] + R::col(v) + e;
          *p = whole && a.accumulate ? *p + x[v * E + e] : x[v * E + e];
        }
  }
}

// Adds the blocks' parts of 32 columns, a strip of the parts a warp, the strips in order.
constexpr int kStrips = 16;
__global__ void __launch_bounds__(32 * kStrips) ln_join(const __grid_constant__ LnArgs a, int parts) {
  __shared__ float strip[kStrips][33];
  wait_for_launch_before();
  float* to = blockIdx.y == 0 ? a.dw : a.db;
  if (!to) return;
  const int col = threadIdx.x % 32, s = threadIdx.x / 32, c = blockIdx.x * 32 + col;
  const int per = (parts + kStrips - 1) / kStrips, end = min(parts, (s + 1) * per);
  const float* p = a.part + (size_t)blockIdx.y * parts * a.D;
  float sum = 0.f;
  if (c < a.D) {
#pragma unroll 8
    for (int i = s * per; i < end; ++i) sum += p[(size_t)i * a.D + c];
  }
  strip[s][col] = sum;
  __syncthreads();
  if (s != 0 || c >= a.D) return;
#pragma unroll
  for (int k = 1; k < kStrips; ++k) sum += strip[k][col];
  to[c] = a.accumulate ? to[c] + sum : sum;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int threads_for(int D, int cols) { return (int)align_up((size_t)(D + cols - 1) / cols, 32); }

// A dependent launch: its set-up overlaps the end of the one before, which the kernel waits for.
template <typename K, typename... A>
cudaError_t launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Columns of a thread: 8 in narrow rows, which have threads to spare.
int cols_of(int D) { return D <= 2048 ? 8 : 16; }
// Blocks on an SM: 512 threads, 256 of which have 128 registers each.
int blocks_per_sm(int T) { return std::max(1, std::min(16, 512 / T)); }
// Blocks of the backward, each with its own parts of the parameter gradients.  Few rows take one, and a
// launch less (a row after another takes it 0.6 us).
constexpr int kOneBlock = 16;
int bwd_blocks(int64_t n, int D) {
  if (n <= kOneBlock) return 1;
  return (int)std::min<int64_t>(n, (int64_t)blocks_per_sm(threads_for(D, cols_of(D))) * device_sm_count());
}

template <typename T, int E, int C, int THREADS, int MIN_BLOCKS>
cudaError_t fwd(const LnArgs& a, int threads, cudaStream_t st) {
  // as many blocks as are resident: each walks its rows with the next one in flight
  constexpr int kRegisters = 65536 / (THREADS * MIN_BLOCKS);
  const int64_t most = (int64_t)std::min(16, 65536 / (kRegisters * threads)) * device_sm_count();
  // what is always summed costs the narrower vectors of fp32 nothing and these registers more than it saves: 8192 rows of
  // 3584 in bf16 23.8 us by AGAIN, 26.0 without, in fp32 48 and 44
  constexpr bool again = sizeof(T) == 2 && E > 1 && C == 16 && THREADS == 256;
  return launch_after(ln_fwd<T, E, C, THREADS, MIN_BLOCKS, again>, dim3((unsigned)std::min<int64_t>(a.n, most)), threads, 0, st, a);
}
template <typename T, int E>
cudaError_t fwd_width(const LnArgs& a, cudaStream_t st) {
  const int threads = threads_for(a.D, cols_of(a.D));
  if (cols_of(a.D) == 8) return fwd<T, E, 8, 256, 4>(a, threads, st);
  // (element by element, two blocks' registers: 8192 rows of 2049 in bf16 46 us, three's 74)
  if (threads <= 256) return fwd<T, E, 16, 256, E == 1 ? 2 : 3>(a, threads, st);
  return threads <= 512 ? fwd<T, E, 16, 512, 1>(a, threads, st) : fwd<T, E, 16, 1024, 1>(a, threads, st);
}
template <typename T>
cudaError_t fwd_any(const LnArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  return a.D % E == 0 && on16(a.x) && on16(a.out) ? fwd_width<T, E>(a, st) : fwd_width<T, 1>(a, st);
}

template <typename T, int E, int C, int THREADS, int MIN_BLOCKS, bool SHARED>
cudaError_t bwd(const LnArgs& a, int threads, int blocks, cudaStream_t st) {
  size_t smem = 0;
  if constexpr (SHARED) {
    static size_t set[kMaxDevices] = {};
    const cudaError_t e =
        set_smem_limit((const void*)ln_bwd<T, E, C, THREADS, MIN_BLOCKS, SHARED>, (size_t)C * THREADS * 8, set);
    if (e != cudaSuccess) return e;
    smem = (size_t)C * threads * 8;
  }
  return launch_after(ln_bwd<T, E, C, THREADS, MIN_BLOCKS, SHARED>, dim3((unsigned)blocks), threads, smem, st, a);
}
template <typename T, int E>
cudaError_t bwd_width(const LnArgs& a, int blocks, cudaStream_t st) {
  const int threads = threads_for(a.D, cols_of(a.D));
  if (cols_of(a.D) == 8) return bwd<T, E, 8, 256, 2, false>(a, threads, blocks, st);
  if (threads <= 256) return bwd<T, E, 16, 256, 2, false>(a, threads, blocks, st);
  if (threads <= 512) return bwd<T, E, 16, 512, 1, true>(a, threads, blocks, st);
  return bwd<T, E, 16, 1024, 1, true>(a, threads, blocks, st);
}
template <typename T>
cudaError_t bwd_any(const LnArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const int blocks = bwd_blocks(a.n, a.D);
  const bool vec = a.D % E == 0 && on16(a.x) && on16(a.dy) && on16(a.dx_in) && on16(a.dx);
  const cudaError_t e = vec ? bwd_width<T, E>(a, blocks, st) : bwd_width<T, 1>(a, blocks, st);
  if (e != cudaSuccess || (!a.dw && !a.db) || blocks == 1) return e;
  return launch_after(ln_join, dim3((a.D + 31) / 32, 2), 32 * kStrips, 0, st, a, blocks);
}

oomb_status check_ln(const void* x, const float* w, int n, int D, int dtype) {
  if (!x || n <= 0 || D <= 0) return OOMB_ERR_ARG;
  if (dtype != OOMB_BF16 && dtype != OOMB_FP32) return OOMB_ERR_DTYPE;
  if (D > kMaxWidth) return OOMB_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(x) % dtype_size(dtype) || reinterpret_cast<uintptr_t>(w) % 4) return OOMB_ERR_ALIGN;
  return OOMB_OK;
}

}  // namespace
}  // namespace oomb

using namespace oomb;

extern "C" {

oomb_status oomb_layer_norm_fwd(const void* x, const float* w, const float* b, float eps, int n, int D, int dtype,
                                void* out, float* mean, float* rstd, void* stream) {
  const oomb_status s = check_ln(x, w, n, D, dtype);
  if (s != OOMB_OK) return s;
  if (!out || !(eps >= 0.f)) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(out) % dtype_size(dtype) || reinterpret_cast<uintptr_t>(b) % 4 ||
      reinterpret_cast<uintptr_t>(mean) % 4 || reinterpret_cast<uintptr_t>(rstd) % 4)
    return OOMB_ERR_ALIGN;
  LnArgs a = {};
  a.x = x;
  a.w = w;
  a.b = b;
  a.param_vec = on16(w) && on16(b);
  a.eps = eps;
  a.n = n;
  a.D = D;
  a.inv_D = 1.f / (float)D;
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? fwd_any<float>(a, st) : fwd_any<__nv_bfloat16>(a, st));
}

size_t oomb_layer_norm_workspace(int n, int D) {
  if (n <= 0 || D <= 0 || D > kMaxWidth) return 0;
  return align_up((size_t)bwd_blocks(n, D) * 2 * D * 4, 256);
}

oomb_status oomb_layer_norm_bwd(const void* x, const float* w, const float* mean, const float* rstd, const void* dy,
                                const void* dx_out, int n, int D, int dtype, void* dx, float* dw, float* db,
                                int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  const oomb_status s = check_ln(x, w, n, D, dtype);
  if (s != OOMB_OK) return s;
  if (!mean || !rstd || !dy || !dx) return OOMB_ERR_ARG;
  if ((dw || db) && (!workspace || ws_bytes < oomb_layer_norm_workspace(n, D))) return OOMB_ERR_WORKSPACE;
  const uintptr_t es = dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(dy) % es || reinterpret_cast<uintptr_t>(dx_out) % es ||
      reinterpret_cast<uintptr_t>(dx) % es || reinterpret_cast<uintptr_t>(mean) % 4 ||
      reinterpret_cast<uintptr_t>(rstd) % 4 || reinterpret_cast<uintptr_t>(dw) % 4 ||
      reinterpret_cast<uintptr_t>(db) % 4 || reinterpret_cast<uintptr_t>(workspace) % 16)
    return OOMB_ERR_ALIGN;
  LnArgs a = {};
  a.x = x;
  a.w = w;
  a.param_vec = on16(w);
  a.n = n;
  a.D = D;
  a.inv_D = 1.f / (float)D;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dx_in = dx_out;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.accumulate = accumulate != 0;
  a.part = reinterpret_cast<float*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? bwd_any<float>(a, st) : bwd_any<__nv_bfloat16>(a, st));
}

}  // extern "C"
