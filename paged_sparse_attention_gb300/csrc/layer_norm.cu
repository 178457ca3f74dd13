// Layer norm with weight and bias over rows of D elements.
//
//   mean = sum x / D,  r = 1 / sqrt(sum (x - mean)^2 / D + eps),  xn = (x - mean) r
//   out  = xn w + b
// and, with dy the gradient of out and dx' one that reaches x by another way,
//   t  = dy w,   dx = dx' + r (t - mean(t) - xn mean(t xn))
//   dw = sum dy xn,  db = sum dy   over the rows
// The deviations are squared after the mean is known, from registers: a row whose mean is large
// against its spread loses nothing.
//
// A row is held by one thread block in registers from its load to its stores, so every tensor is
// read once and written once; both kernels are bound by HBM.  Forward: a block a row, the rows in
// flight on an SM hide each other's two sums.  Backward: a block walks the rows b, b + grid, ...
// with the next row's loads in flight, keeps the parameter gradients of its columns and leaves
// them in the workspace; they are added there in block order, the same bits on every run.
#include <cmath>

#include "attn_common.cuh"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kMaxWidth = 16384;
constexpr int kCols = 8;  // columns of a thread in the backward

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
// Sum of N values over the block; every thread gets them.  `buf`: 2 x 32 x N floats used in
// turns, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  const int warps = blockDim.x / 32;
  if (warps == 1) return;
  float* b = buf + turn * 32 * N;
  turn ^= 1;
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i * 32 + threadIdx.x / 32] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < warps; w += 4) {  // the entries behind the last warp are 0
      const float4 x = *reinterpret_cast<const float4*>(b + i * 32 + w);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    v[i] = (s.x + s.y) + (s.z + s.w);
  }
}

// NV vectors of E elements a thread: vector v starts at column (v T + threadIdx.x) E.
template <typename T, int E, int NV>
struct Row {
  // the elements as they are stored, so that a row in flight takes few registers
  using Word = typename std::conditional<E == 1, T, uint4>::type;
  Word raw[NV];
  __device__ __forceinline__ void load(const T* row, int D) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + (int)threadIdx.x) * E;
      if (c < D) raw[v] = *reinterpret_cast<const Word*>(row + c);
    }
  }
  __device__ __forceinline__ void get(int D, float (&f)[NV * E]) const {  // absent elements are 0
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool has = (v * (int)blockDim.x + (int)threadIdx.x) * E < D;
      const T* x = reinterpret_cast<const T*>(&raw[v]);
#pragma unroll
      for (int e = 0; e < E; ++e) f[v * E + e] = has ? to_float<T>(x[e]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T* row, int D, const float (&f)[NV * E]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + (int)threadIdx.x) * E;
      if (c >= D) continue;
      Word w;
      T* x = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = from_float<T>(f[v * E + e]);
      *reinterpret_cast<Word*>(row + c) = w;
    }
  }
};
// fp32 parameters at the same columns (vec: on 16 bytes)
template <int E, int NV>
__device__ __forceinline__ void load_param(const float* p, int D, bool vec, float (&f)[NV * E], float absent) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * (int)blockDim.x + (int)threadIdx.x) * E;
    if (E % 4 == 0 && vec && p && c < D) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p + c + e));
        f[v * E + e] = x.x;
        f[v * E + (E > 1 ? e + 1 : 0)] = x.y;
        f[v * E + (E > 1 ? e + 2 : 0)] = x.z;
        f[v * E + (E > 1 ? e + 3 : 0)] = x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[v * E + e] = p && c < D ? __ldg(p + c + e) : absent;
    }
  }
}

template <typename T, int E, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 512 ? 1024 / THREADS : 1) ln_fwd(const __grid_constant__ LnArgs a) {
  __shared__ __align__(16) float buf[64];
  if (threadIdx.x < 64) buf[threadIdx.x] = 0.f;
  for (int i = threadIdx.x + blockDim.x; i < 64; i += blockDim.x) buf[i] = 0.f;
  if (blockDim.x > 32) __syncthreads();
  int turn = 0;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    Row<T, E, NV> row;
    row.load(reinterpret_cast<const T*>(a.x) + (size_t)i * a.D, a.D);
    float x[NV * E], s[1] = {0.f};
    row.get(a.D, x);
#pragma unroll
    for (int k = 0; k < NV * E; ++k) s[0] += x[k];
    block_sums<1>(s, buf, turn);
    const float mean = s[0] * a.inv_D;
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool has = (v * (int)blockDim.x + (int)threadIdx.x) * E < a.D;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = has ? x[v * E + e] - mean : 0.f;
        x[v * E + e] = c;
        s[0] = fmaf(c, c, s[0]);
      }
    }
    block_sums<1>(s, buf, turn);
    const float r = rsqrtf(fmaf(s[0], a.inv_D, a.eps));
    float w[NV * E], b[NV * E];
    load_param<E, NV>(a.w, a.D, a.param_vec, w, 1.f);
    load_param<E, NV>(a.b, a.D, a.param_vec, b, 0.f);
#pragma unroll
    for (int k = 0; k < NV * E; ++k) x[k] = fmaf(x[k] * r, w[k], b[k]);
    Row<T, E, NV>::store(reinterpret_cast<T*>(a.out) + (size_t)i * a.D, a.D, x);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[i] = mean;
      if (a.rstd) a.rstd[i] = r;
    }
  }
}

// WIDE: 16 columns a thread, whose sums are in shared memory; else 8, in registers.  AHEAD rows are
// in flight beside the one in hand.
template <typename T, int E, int NV, bool WIDE, int AHEAD, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) ln_bwd(const __grid_constant__ LnArgs a) {
  constexpr int C = NV * E;
  extern __shared__ __align__(16) float acc[];  // WIDE: [2 C, T]
  __shared__ __align__(16) float buf[128];
  let_next_launch();
  for (int i = threadIdx.x; i < 128; i += blockDim.x) buf[i] = 0.f;
  float w[C], dw[C], db[C];
  load_param<E, NV>(a.w, a.D, a.param_vec, w, 1.f);
#pragma unroll
  for (int k = 0; k < C; ++k) {
    dw[k] = db[k] = 0.f;
    if constexpr (WIDE) acc[k * blockDim.x + threadIdx.x] = acc[(C + k) * blockDim.x + threadIdx.x] = 0.f;
  }
  __syncthreads();
  int turn = 0;
  Row<T, E, NV> nx[AHEAD], ny[AHEAD], nz[AHEAD];
  float n_mean[AHEAD], n_rstd[AHEAD];
  auto fetch = [&](int64_t i, int u) {
    if (i >= a.n) return;
    const size_t at = (size_t)i * a.D;
    nx[u].load(reinterpret_cast<const T*>(a.x) + at, a.D);
    ny[u].load(reinterpret_cast<const T*>(a.dy) + at, a.D);
    if (a.dx_in) nz[u].load(reinterpret_cast<const T*>(a.dx_in) + at, a.D);
    n_mean[u] = a.mean[i];
    n_rstd[u] = a.rstd[i];
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) fetch(blockIdx.x + (int64_t)u * gridDim.x, u);
  for (int64_t i0 = blockIdx.x; i0 < a.n; i0 += (int64_t)AHEAD * gridDim.x) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t i = i0 + (int64_t)u * gridDim.x;
      if (i >= a.n) break;
      float xn[C], t[C], s[2] = {0.f, 0.f};
      Row<T, E, NV> rz = nz[u];
      nx[u].get(a.D, xn);
      ny[u].get(a.D, t);
      const float mean = n_mean[u], r = n_rstd[u];
      fetch(i + (int64_t)AHEAD * gridDim.x, u);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xn[k] = (xn[k] - mean) * r;  // absent columns: t is 0 there
        if constexpr (WIDE) {
          acc[k * blockDim.x + threadIdx.x] += t[k] * xn[k];
          acc[(C + k) * blockDim.x + threadIdx.x] += t[k];
        } else {
          dw[k] = fmaf(t[k], xn[k], dw[k]);
          db[k] += t[k];
        }
        t[k] *= w[k];
        s[0] += t[k];
        s[1] = fmaf(t[k], xn[k], s[1]);
      }
      block_sums<2>(s, buf, turn);
      const float m0 = s[0] * a.inv_D, m1 = s[1] * a.inv_D;
#pragma unroll
      for (int k = 0; k < C; ++k) t[k] = r * (t[k] - m0 - xn[k] * m1);
      if (a.dx_in) {
        rz.get(a.D, xn);
#pragma unroll
        for (int k = 0; k < C; ++k) t[k] += xn[k];
      }
      Row<T, E, NV>::store(reinterpret_cast<T*>(a.dx) + (size_t)i * a.D, a.D, t);
    }
  }
  float* pw = a.part + (size_t)blockIdx.x * a.D;
  float* pb = a.part + ((size_t)gridDim.x + blockIdx.x) * a.D;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * (int)blockDim.x + (int)threadIdx.x) * E;
    if (c >= a.D) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = v * E + e;
      if (a.dw) pw[c + e] = WIDE ? acc[k * blockDim.x + threadIdx.x] : dw[k];
      if (a.db) pb[c + e] = WIDE ? acc[(C + k) * blockDim.x + threadIdx.x] : db[k];
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

int bwd_cols(int D) { return D <= 512 * kCols ? kCols : 2 * kCols; }
// Blocks of the backward, each with its own parts of the parameter gradients: 512 threads an SM.
int bwd_blocks(int64_t n, int D) {
  const int per_sm = std::max(1, std::min(8, 512 / threads_for(D, bwd_cols(D))));
  return (int)std::min<int64_t>(n, (int64_t)per_sm * device_sm_count());
}

template <typename T, int E, int NV>
cudaError_t fwd(const LnArgs& a, cudaStream_t st) {
  count_launches(1);
  const int threads = threads_for(a.D, E * NV);
  const unsigned grid = (unsigned)std::min<int64_t>(a.n, 1 << 20);
  if (threads <= 128)
    ln_fwd<T, E, NV, 128><<<grid, threads, 0, st>>>(a);
  else if (threads <= 512)
    ln_fwd<T, E, NV, 512><<<grid, threads, 0, st>>>(a);
  else
    ln_fwd<T, E, NV, 1024><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t fwd_any(const LnArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  if (a.D % E == 0 && on16(a.x) && on16(a.out)) return fwd<T, E, 4>(a, st);
  return fwd<T, 1, 16>(a, st);
}

template <typename T, int E, int NV, bool WIDE, int AHEAD, int THREADS>
cudaError_t bwd(const LnArgs& a, int blocks, cudaStream_t st) {
  const int threads = threads_for(a.D, E * NV);
  size_t smem = 0;
  if constexpr (WIDE) {
    static size_t set[kMaxDevices] = {};
    const cudaError_t e =
        set_smem_limit((const void*)ln_bwd<T, E, NV, WIDE, AHEAD, THREADS>, (size_t)2 * E * NV * THREADS * 4, set);
    if (e != cudaSuccess) return e;
    smem = (size_t)2 * E * NV * threads * 4;
  }
  count_launches(1);
  ln_bwd<T, E, NV, WIDE, AHEAD, THREADS><<<(unsigned)blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int E>
cudaError_t bwd_width(const LnArgs& a, int blocks, cudaStream_t st) {
  if (bwd_cols(a.D) == kCols) return bwd<T, E, kCols / E, false, sizeof(T) == 2 ? 3 : 2, 512>(a, blocks, st);
  if (a.D <= 512 * 2 * kCols) return bwd<T, E, 2 * kCols / E, true, 1, 512>(a, blocks, st);
  return bwd<T, E, 2 * kCols / E, true, 1, 1024>(a, blocks, st);
}
template <typename T>
cudaError_t bwd_any(const LnArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const int blocks = bwd_blocks(a.n, a.D);
  const bool vec = a.D % E == 0 && on16(a.x) && on16(a.dy) && on16(a.dx_in) && on16(a.dx);
  const cudaError_t e = vec ? bwd_width<T, E>(a, blocks, st) : bwd_width<T, 1>(a, blocks, st);
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.D + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kStrips);
  cfg.stream = st;
  cudaLaunchAttribute attr;  // a dependent launch: its set-up overlaps the end of the row kernel
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, ln_join, a, blocks);
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
  if (!workspace || ws_bytes < oomb_layer_norm_workspace(n, D)) return OOMB_ERR_WORKSPACE;
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
