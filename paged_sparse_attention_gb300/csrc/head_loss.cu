// Softmax cross entropy of the output projection over a large vocabulary, without the logits.
//
//   z = x W^T, z' = c tanh(z / c) with a cap c;  lse_i = log sum_v exp z'_iv;  loss_i = lse_i - z'_i,t
//   dz = g_i (exp(z' - lse) - [v = t]) (1 - (z'/c)^2);  dx = s dz W;  dW (+)= s dz^T x
//
// The simplest form: tiles of the products on the CUDA cores in fp32.
#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kTM = 64, kTN = 64, kTK = 16;
constexpr int kPieceCols = 2048;

struct HeadArgs {
  const void* x;
  const void* w;
  const int64_t* targets;
  int n, D, V;
  float cap, scale;
  float* loss;
  const float* lse_in;
  float* lse;
  const float* d_loss;
  void* dx;
  void* dw;
  int accumulate;
  uint32_t* err;
  float2* part;  // [tiles of V, n] row maximum and sum of a tile
  float* at;     // [n] logit of the target
  float* dz;     // [n, piece]
  float* dxa;    // [n, D] sum over the pieces
  int v0, cols;  // the piece
};

__device__ __forceinline__ int target_of(const HeadArgs& a, int i) {
  const int64_t t = a.targets[i];
  if (t >= a.V) atomicOr(a.err, OOMB_DEVERR_TOKEN);
  return t < 0 || t >= a.V ? -1 : (int)t;
}

// acc[i][j] = sum_k fa(row, k) fb(col, k) of a 64 x 64 tile, 4 x 4 a thread
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(FA fa, FB fb, int K, float (&acc)[4][4]) {
  __shared__ float sa[kTK][kTM + 1], sb[kTK][kTN + 1];
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kTK) {
    for (int e = threadIdx.x; e < kTK * kTM; e += 256) {
      sa[e % kTK][e / kTK] = k0 + e % kTK < K ? fa(e / kTK, k0 + e % kTK) : 0.f;
      sb[e % kTK][e / kTK] = k0 + e % kTK < K ? fb(e / kTK, k0 + e % kTK) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
}

template <typename T>
__device__ __forceinline__ void logits(const HeadArgs& a, int m0, int v0, float (&z)[4][4]) {
  const T* x = (const T*)a.x;
  const T* w = (const T*)a.w;
  tile_product(
      [&](int r, int k) { return m0 + r < a.n && a.targets[m0 + r] >= 0 ? to_float<T>(x[(size_t)(m0 + r) * a.D + k]) : 0.f; },
      [&](int r, int k) { return v0 + r < a.V ? to_float<T>(w[(size_t)(v0 + r) * a.D + k]) : 0.f; }, a.D, z);
  if (a.cap > 0.f)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[i][j] = a.cap * tanhf(z[i][j] / a.cap);
}

template <typename T>
__global__ void __launch_bounds__(256) head_fwd_tile(const HeadArgs a) {
  const int m0 = blockIdx.x * kTM, v0 = blockIdx.y * kTN;
  float z[4][4];
  logits<T>(a, m0, v0, z);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i) {
    const int r = m0 + ty * 4 + i;
    const int t = r < a.n ? target_of(a, r) : -1;
    float m = -INFINITY, s = 0.f;
    for (int j = 0; j < 4; ++j)
      if (v0 + tx * 4 + j < a.V) m = fmaxf(m, z[i][j]);
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + tx * 4 + j;
      if (v < a.V) s += __expf(z[i][j] - m);
      if (v == t && r < a.n) a.at[r] = z[i][j];
    }
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tx == 0 && r < a.n) a.part[(size_t)blockIdx.y * a.n + r] = make_float2(m, s);
  }
}

__global__ void __launch_bounds__(128) head_fwd_join(const HeadArgs a, int tiles) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= a.n) return;
  float m = -INFINITY, s = 0.f;
  for (int t = 0; t < tiles; ++t) m = fmaxf(m, a.part[(size_t)t * a.n + r].x);
  for (int t = 0; t < tiles; ++t) {
    const float2 p = a.part[(size_t)t * a.n + r];
    s += p.y * __expf(p.x - m);
  }
  const bool has = target_of(a, r) >= 0;
  const float lse = m + logf(s);
  a.lse[r] = has ? lse : 0.f;
  a.loss[r] = has ? lse - a.at[r] : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(256) head_dz_tile(const HeadArgs a) {
  const int m0 = blockIdx.x * kTM, c0 = blockIdx.y * kTN;
  float z[4][4];
  logits<T>(a, m0, a.v0 + c0, z);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i) {
    const int r = m0 + ty * 4 + i;
    if (r >= a.n) continue;
    const int t = target_of(a, r);
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tx * 4 + j;
      if (c >= a.cols) continue;
      float d = 0.f;
      if (t >= 0) {
        d = __expf(z[i][j] - a.lse_in[r]) - (a.v0 + c == t ? 1.f : 0.f);
        if (a.cap > 0.f) d *= 1.f - (z[i][j] / a.cap) * (z[i][j] / a.cap);
        if (a.d_loss) d *= a.d_loss[r];
      }
      a.dz[(size_t)r * kPieceCols + c] = d;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) head_dx_tile(const HeadArgs a) {
  const int m0 = blockIdx.x * kTM, c0 = blockIdx.y * kTN;
  const T* w = (const T*)a.w;
  float acc[4][4];
  tile_product([&](int r, int k) { return m0 + r < a.n ? a.dz[(size_t)(m0 + r) * kPieceCols + k] : 0.f; },
               [&](int c, int k) { return c0 + c < a.D ? to_float<T>(w[(size_t)(a.v0 + k) * a.D + c0 + c]) : 0.f; }, a.cols,
               acc);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (r >= a.n || c >= a.D) continue;
      const float v = (a.v0 ? a.dxa[(size_t)r * a.D + c] : 0.f) + acc[i][j];
      a.dxa[(size_t)r * a.D + c] = v;
      if (a.v0 + a.cols == a.V) ((T*)a.dx)[(size_t)r * a.D + c] = from_float<T>(a.scale * v);
    }
}

template <typename T, typename TW>
__global__ void __launch_bounds__(256) head_dw_tile(const HeadArgs a) {
  const int m0 = blockIdx.x * kTM, c0 = blockIdx.y * kTN;
  const T* x = (const T*)a.x;
  float acc[4][4];
  tile_product([&](int r, int k) { return m0 + r < a.cols ? a.dz[(size_t)k * kPieceCols + m0 + r] : 0.f; },
               [&](int c, int k) {
                 return c0 + c < a.D && a.targets[k] >= 0 ? to_float<T>(x[(size_t)k * a.D + c0 + c]) : 0.f;
               },
               a.n, acc);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (r >= a.cols || c >= a.D) continue;
      TW* to = (TW*)a.dw + (size_t)(a.v0 + r) * a.D + c;
      *to = from_float<TW>(a.accumulate ? to_float<TW>(*to) + a.scale * acc[i][j] : a.scale * acc[i][j]);
    }
}

int tiles(int64_t x, int t) { return (int)((x + t - 1) / t); }

template <typename T>
cudaError_t forward(const HeadArgs& a, cudaStream_t st) {
  count_launches(2);
  head_fwd_tile<T><<<dim3(tiles(a.n, kTM), tiles(a.V, kTN)), 256, 0, st>>>(a);
  head_fwd_join<<<tiles(a.n, 128), 128, 0, st>>>(a, tiles(a.V, kTN));
  return cudaGetLastError();
}
template <typename T>
cudaError_t backward(HeadArgs a, int dw_dtype, cudaStream_t st) {
  for (a.v0 = 0; a.v0 < a.V; a.v0 += kPieceCols) {
    a.cols = std::min(kPieceCols, a.V - a.v0);
    head_dz_tile<T><<<dim3(tiles(a.n, kTM), tiles(a.cols, kTN)), 256, 0, st>>>(a);
    count_launches(1);
    if (a.dx) head_dx_tile<T><<<dim3(tiles(a.n, kTM), tiles(a.D, kTN)), 256, 0, st>>>(a), count_launches(1);
    if (!a.dw) continue;
    count_launches(1);
    const dim3 grid(tiles(a.cols, kTM), tiles(a.D, kTN));
    if (dw_dtype == OOMB_FP32)
      head_dw_tile<T, float><<<grid, 256, 0, st>>>(a);
    else
      head_dw_tile<T, __nv_bfloat16><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

struct Space {
  size_t part, at, dz, dxa, bytes;
};
Space space(int64_t n, int D, int V, bool bwd) {
  Space s = {};
  s.part = 0;
  s.at = align_up((size_t)tiles(V, kTN) * n * 8, 256);
  s.bytes = s.at + align_up((size_t)n * 4, 256);
  if (bwd) {
    s.dz = 0;
    s.dxa = align_up((size_t)n * kPieceCols * 4, 256);
    s.bytes = std::max(s.bytes, s.dxa + align_up((size_t)n * D * 4, 256));
  }
  return s;
}

oomb_status check(const void* x, const void* w, const int64_t* targets, int n, int D, int V, int dtype, float cap,
                  const void* lse, const void* ws, const uint32_t* word) {
  if (!x || !w || !targets || !lse || !word || n <= 0 || D <= 0 || V <= 0 || V > INT_MAX - 1024) return OOMB_ERR_ARG;
  if (!(cap >= 0.f) || cap > 1e30f || (cap > 0.f && cap < 1e-30f)) return OOMB_ERR_ARG;
  if (dtype != OOMB_BF16 && dtype != OOMB_FP32) return OOMB_ERR_DTYPE;
  if (D > 65536) return OOMB_ERR_UNSUPPORTED;
  const uintptr_t es = dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(w) % es ||
      reinterpret_cast<uintptr_t>(targets) % 8 || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(ws) % 256 || reinterpret_cast<uintptr_t>(word) % 4)
    return OOMB_ERR_ALIGN;
  return OOMB_OK;
}

}  // namespace
}  // namespace oomb

using namespace oomb;

extern "C" {

size_t oomb_head_loss_workspace(int n, int D, int V, int dtype, int backward) {
  if (n <= 0 || D <= 0 || D > 65536 || V <= 0 || V > INT_MAX - 1024 || (dtype != OOMB_BF16 && dtype != OOMB_FP32)) return 0;
  return space(n, D, V, backward != 0).bytes;
}

oomb_status oomb_head_loss_fwd(const void* x, const void* w, const int64_t* targets, int n, int D, int V, int dtype,
                               float softcap, float* loss, float* lse, void* workspace, size_t ws_bytes,
                               uint32_t* error_word, void* stream) {
  const oomb_status s = check(x, w, targets, n, D, V, dtype, softcap, lse, workspace, error_word);
  if (s != OOMB_OK) return s;
  if (!loss) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(loss) % 4) return OOMB_ERR_ALIGN;
  const Space p = space(n, D, V, false);
  if (!workspace || ws_bytes < p.bytes) return OOMB_ERR_WORKSPACE;
  HeadArgs a = {};
  a.x = x;
  a.w = w;
  a.targets = targets;
  a.n = n;
  a.D = D;
  a.V = V;
  a.cap = softcap;
  a.loss = loss;
  a.lse = lse;
  a.err = error_word;
  a.part = reinterpret_cast<float2*>((char*)workspace + p.part);
  a.at = reinterpret_cast<float*>((char*)workspace + p.at);
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? forward<float>(a, st) : forward<__nv_bfloat16>(a, st));
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
  const Space p = space(n, D, V, true);
  if (!workspace || ws_bytes < p.bytes) return OOMB_ERR_WORKSPACE;
  HeadArgs a = {};
  a.x = x;
  a.w = w;
  a.targets = targets;
  a.n = n;
  a.D = D;
  a.V = V;
  a.cap = softcap;
  a.scale = scale;
  a.lse_in = lse;
  a.d_loss = d_loss;
  a.dx = dx;
  a.dw = dw;
  a.accumulate = accumulate != 0;
  a.err = error_word;
  a.dz = reinterpret_cast<float*>((char*)workspace + p.dz);
  a.dxa = reinterpret_cast<float*>((char*)workspace + p.dxa);
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == OOMB_FP32 ? backward<float>(a, dw_dtype, st)
                                        : backward<__nv_bfloat16>(a, dw_dtype, st));
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
