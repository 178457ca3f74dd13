// The norms before and after a block, fused with the block's gate and residual scale.
//
//   z  = y * r_post * w_post,  r_post = 1 / sqrt(mean(y^2) + eps)     (z = y without w_post)
//   x' = x + res_scale * g * z                                        (x' = x without y)
//   u  = x' * r_pre * w_pre,   r_pre  = 1 / sqrt(mean(x'^2) + eps)
// and, with dx' the gradient that arrives at x' beside the one through u,
//   t  = du * w_pre,           dx = dx' + r_pre (t - xn mean(t xn)),  xn = x' r_pre
//   dz = res_scale * g * dx,   dy = r_post (q - yn mean(q yn)),       q = dz w_post, yn = y r_post
//   dw_pre = sum du xn,  dw_post = sum dz yn,  dg = res_scale * dx * z  (summed over the rows
//   for a gate per channel).
// x' is never rounded on the way to u, and the backward forms it again from x and y in fp32
// instead of reading the rounded one: the same bytes, and no rounding but the outputs'.
//
// A row is held by one thread block, E consecutive elements a thread (16-byte accesses), in
// registers from its load to its stores: every tensor is read once and written once.  The
// rows' sums over the weight gradients stay with the block (rows b, b + grid, ...), go to the
// workspace once a block and are summed there in block order, so they are the same bits on
// every run.  Widths that are no multiple of the vector, or rows off 16 bytes, take the
// element-wise variant, which reads a row again (from L1/L2) for each pass over it.
#include <cmath>

#include "attn_common.cuh"
#include "block_norm.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kMaxWidth = 16384;
constexpr int kSlowThreads = 512;

// Sum over the block; every thread gets it.  `buf` holds 2 x 32 floats, used in turns so that
// one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float* buf, int& turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
  if (warps == 1) return v;
  float* b = buf + 32 * turn;
  turn ^= 1;
  if (lane == 0) b[threadIdx.x / 32] = v;
  __syncthreads();
  v = lane < warps ? b[lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// E consecutive elements as fp32, and back with one rounding.
template <typename T, int E>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[E]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    const uint4 w = *reinterpret_cast<const uint4*>(p + i);
    const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int e = 0; e < V; ++e) f[i + e] = to_float<T>(x[e]);
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[E]) {
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
template <int E>
__device__ __forceinline__ void load_param(const float* p, int c, float (&f)[E], float otherwise) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    float4 w = make_float4(otherwise, otherwise, otherwise, otherwise);
    if (p) w = *reinterpret_cast<const float4*>(p + c + i);
    f[i] = w.x;
    f[i + 1] = w.y;
    f[i + 2] = w.z;
    f[i + 3] = w.w;
  }
}

// ------------------------------------------------------------------ forward
template <typename T, int E>
__global__ void __launch_bounds__(1024, 1) norm_fwd(const NormArgs a) {
  __shared__ float buf[64];
  int turn = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  const T* y = reinterpret_cast<const T*>(a.y);
  const T* x = reinterpret_cast<const T*>(a.x);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t at = (size_t)row * a.D + c;
    float f[E], r[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = r[e] = 0.f;
    if (in) load_vec<T, E>(x + at, f);
    if (a.y) {
      if (in) load_vec<T, E>(y + at, r);
      if (a.w_post) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += r[e] * r[e];
        const float rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rstd;
        if (in) {
          float w[E];
          load_param<E>(a.w_post, c, w, 1.f);
#pragma unroll
          for (int e = 0; e < E; ++e) r[e] *= rstd * w[e];
        }
      }
      if (in) {
        float g[E];
        if (a.gate && a.gate_rows)
          load_vec<T, E>(reinterpret_cast<const T*>(a.gate) + at, g);
        else
          load_param<E>(reinterpret_cast<const float*>(a.gate), c, g, 1.f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += a.res_scale * g[e] * r[e];
      }
    }
    if (a.w_pre) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += f[e] * f[e];
      const float rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rstd;
      if (in) {
        float w[E];
        load_param<E>(a.w_pre, c, w, 1.f);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] *= f[e] * rstd;
        store_vec<T, E>(reinterpret_cast<T*>(a.u) + at, w);
      }
    }
    if (a.x_out && in) store_vec<T, E>(reinterpret_cast<T*>(a.x_out) + at, f);
  }
}

template <typename T>
__device__ __forceinline__ float gate_at(const NormArgs& a, size_t at, int c) {
  if (!a.gate) return 1.f;
  return a.gate_rows ? to_float<T>(reinterpret_cast<const T*>(a.gate)[at]) : reinterpret_cast<const float*>(a.gate)[c];
}

template <typename T>
__global__ void __launch_bounds__(kSlowThreads) norm_fwd_any(const NormArgs a) {
  __shared__ float buf[64];
  int turn = 0;
  const T* y = reinterpret_cast<const T*>(a.y);
  const T* x = reinterpret_cast<const T*>(a.x);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t at0 = (size_t)row * a.D;
    float r_post = 1.f, r_pre = 1.f;
    if (a.y && a.w_post) {
      float s = 0.f;
      for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        const float v = to_float<T>(y[at0 + c]);
        s += v * v;
      }
      r_post = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = r_post;
    }
    auto value = [&](int c) {
      float v = to_float<T>(x[at0 + c]);
      if (a.y) {
        float z = to_float<T>(y[at0 + c]);
        if (a.w_post) z *= r_post * a.w_post[c];
        v += a.res_scale * gate_at<T>(a, at0 + c, c) * z;
      }
      return v;
    };
    if (a.w_pre) {
      float s = 0.f;
      for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        const float v = value(c);
        s += v * v;
      }
      r_pre = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = r_pre;
    }
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      const float v = value(c);
      if (a.w_pre) reinterpret_cast<T*>(a.u)[at0 + c] = from_float<T>(v * r_pre * a.w_pre[c]);
      if (a.x_out) reinterpret_cast<T*>(a.x_out)[at0 + c] = from_float<T>(v);
    }
  }
}

// ----------------------------------------------------------------- backward
// A block's three sums of a column, in shared memory: [dw_pre | dw_post | dgate] x D.  Each
// column belongs to one thread.
template <typename T, int E>
__global__ void __launch_bounds__(1024, 1) norm_bwd(const NormArgs a) {
  extern __shared__ __align__(16) float acc[];
  __shared__ float buf[64];
  int turn = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  const bool sum_gate = a.gate && !a.gate_rows && a.dgate;
  if (in)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[c + e] = acc[a.D + c + e] = acc[2 * a.D + c + e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t at = (size_t)row * a.D + c;
    float g[E], z[E], dx[E];
    const float r_post = a.w_post ? a.rstd_post[row] : 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dx[e] = z[e] = 0.f;
    if (in && a.y) {
      load_vec<T, E>(reinterpret_cast<const T*>(a.y) + at, z);  // y
      if (a.gate && a.gate_rows)
        load_vec<T, E>(reinterpret_cast<const T*>(a.gate) + at, g);
      else
        load_param<E>(reinterpret_cast<const float*>(a.gate), c, g, 1.f);
    }
    if (in && a.dx_in) load_vec<T, E>(reinterpret_cast<const T*>(a.dx_in) + at, dx);
    if (a.w_pre) {
      const float r_pre = a.rstd_pre[row];
      float t[E], xn[E], s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = xn[e] = 0.f;
      if (in) {
        load_vec<T, E>(reinterpret_cast<const T*>(a.x) + at, xn);
        if (a.y) {
          float w[E];
          load_param<E>(a.w_post, c, w, 1.f);
#pragma unroll
          for (int e = 0; e < E; ++e) xn[e] += a.res_scale * g[e] * (z[e] * (a.w_post ? r_post * w[e] : 1.f));
        }
        float du[E], w[E];
        load_vec<T, E>(reinterpret_cast<const T*>(a.du) + at, du);
        load_param<E>(a.w_pre, c, w, 1.f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          xn[e] *= r_pre;
          t[e] = du[e] * w[e];
          s += t[e] * xn[e];
          acc[c + e] += du[e] * xn[e];
        }
      }
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] += r_pre * (t[e] - xn[e] * mean);
    }
    if (in && a.dx) store_vec<T, E>(reinterpret_cast<T*>(a.dx) + at, dx);
    if (!a.y) continue;
    float q[E], s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = 0.f;
    if (in) {
      float w[E], dg[E];
      load_param<E>(a.w_post, c, w, 1.f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float yn = z[e] * r_post, dgz = a.res_scale * dx[e], dz = dgz * g[e];
        dg[e] = dgz * (yn * w[e]);
        if (a.w_post) acc[a.D + c + e] += dz * yn;
        if (sum_gate) acc[2 * a.D + c + e] += dg[e];
        q[e] = dz * w[e];
        z[e] = yn;
        s += q[e] * yn;
      }
      if (a.gate && a.gate_rows && a.dgate) store_vec<T, E>(reinterpret_cast<T*>(a.dgate) + at, dg);
    }
    if (a.w_post) {
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] = r_post * (q[e] - z[e] * mean);
    }
    if (in && a.dy) store_vec<T, E>(reinterpret_cast<T*>(a.dy) + at, q);
  }
  if (in) {
    float* dst = a.part + (size_t)blockIdx.x * 3 * a.D + c;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(dst + (size_t)k * a.D + e) =
            *reinterpret_cast<const float4*>(acc + (size_t)k * a.D + c + e);
  }
}

template <typename T>
__global__ void __launch_bounds__(kSlowThreads) norm_bwd_any(const NormArgs a) {
  extern __shared__ __align__(16) float acc[];
  __shared__ float buf[64];
  int turn = 0;
  const bool sum_gate = a.gate && !a.gate_rows && a.dgate;
  const T* y = reinterpret_cast<const T*>(a.y);
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* du = reinterpret_cast<const T*>(a.du);
  for (int c = threadIdx.x; c < 3 * a.D; c += blockDim.x) acc[c] = 0.f;
  __syncthreads();
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t at0 = (size_t)row * a.D;
    const float r_post = a.w_post ? a.rstd_post[row] : 1.f, r_pre = a.w_pre ? a.rstd_pre[row] : 1.f;
    auto normed = [&](int c) {  // x' r_pre
      float v = to_float<T>(x[at0 + c]);
      if (a.y) {
        const float z = to_float<T>(y[at0 + c]) * (a.w_post ? r_post * a.w_post[c] : 1.f);
        v += a.res_scale * gate_at<T>(a, at0 + c, c) * z;
      }
      return v * r_pre;
    };
    float mean_pre = 0.f, mean_post = 0.f;
    if (a.w_pre) {
      float s = 0.f;
      for (int c = threadIdx.x; c < a.D; c += blockDim.x) s += to_float<T>(du[at0 + c]) * a.w_pre[c] * normed(c);
      mean_pre = block_sum(s, buf, turn) * a.inv_D;
    }
    auto grad_x = [&](int c, float xn) {
      float v = a.dx_in ? to_float<T>(reinterpret_cast<const T*>(a.dx_in)[at0 + c]) : 0.f;
      if (a.w_pre) v += r_pre * (to_float<T>(du[at0 + c]) * a.w_pre[c] - xn * mean_pre);
      return v;
    };
    if (a.y && a.w_post) {
      float s = 0.f;
      for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        const float dx = grad_x(c, a.w_pre ? normed(c) : 0.f);
        s += a.res_scale * dx * gate_at<T>(a, at0 + c, c) * a.w_post[c] * (to_float<T>(y[at0 + c]) * r_post);
      }
      mean_post = block_sum(s, buf, turn) * a.inv_D;
    }
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      const float xn = a.w_pre ? normed(c) : 0.f;
      const float dx = grad_x(c, xn);
      if (a.w_pre) acc[c] += to_float<T>(du[at0 + c]) * xn;
      if (a.y) {
        const float yn = to_float<T>(y[at0 + c]) * r_post, w = a.w_post ? a.w_post[c] : 1.f;
        const float g = gate_at<T>(a, at0 + c, c), dgz = a.res_scale * dx, dz = dgz * g, dg = dgz * (yn * w);
        if (a.w_post) acc[a.D + c] += dz * yn;
        if (sum_gate) acc[2 * a.D + c] += dg;
        if (a.gate && a.gate_rows && a.dgate) reinterpret_cast<T*>(a.dgate)[at0 + c] = from_float<T>(dg);
        if (a.dy)
          reinterpret_cast<T*>(a.dy)[at0 + c] = from_float<T>(a.w_post ? r_post * (dz * w - yn * mean_post) : dz * w);
      }
      if (a.dx) reinterpret_cast<T*>(a.dx)[at0 + c] = from_float<T>(dx);  // last: dx may be dx_in
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 3 * a.D; c += blockDim.x) a.part[(size_t)blockIdx.x * 3 * a.D + c] = acc[c];
}

// Column sums over the blocks' parts, in block order: 32 columns a block, 8 strips of the
// parts each, the strips joined in order.  out[k] is dw_pre, dw_post or dgate (or nullptr).
__global__ void __launch_bounds__(256) norm_join(const float* __restrict__ part, int n_parts, int D, float* dw_pre,
                                                 float* dw_post, float* dgate, int accumulate) {
  __shared__ float strip[8][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, k = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float* out = k == 0 ? dw_pre : k == 1 ? dw_post : dgate;
  if (!out) return;
  const int p0 = n_parts * w / 8, p1 = n_parts * (w + 1) / 8;
  float s = 0.f;
  if (c < D)
    for (int p = p0; p < p1; ++p) s += part[((size_t)p * 3 + k) * D + c];
  strip[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += strip[i][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

// ------------------------------------------------------------ rows through a ring
// Many rows: a block walks its rows with the next ones in flight.  One thread copies whole
// rows of every tensor that is read (cp.async.bulk) into a ring of kept stages in shared
// memory; the threads wait for a stage, take their elements into registers and hand the stage
// back.  So a block keeps stages x tensors x row bytes of loads in flight whatever its barriers
// wait for, and two blocks of an SM hide each other's sums.
constexpr int kMaxStages = 4;
constexpr int kMaxRowTensors = 5;

struct RowRing {
  const char* src[kMaxRowTensors];  // tensors read, in the order they stand in a stage
  int n_src;
  uint32_t row_bytes;
  int stages;
};

struct __align__(16) RingBars {
  uint64_t full[kMaxStages];
};

__device__ __forceinline__ void ring_issue(const RowRing& r, uint8_t* base, RingBars* bars, int64_t row, int k) {
  mbar_arrive_expect_tx(&bars->full[k], r.row_bytes * (uint32_t)r.n_src);
  uint8_t* dst = base + (size_t)k * r.n_src * r.row_bytes;
  for (int i = 0; i < r.n_src; ++i)
    bulk_load(dst + (size_t)i * r.row_bytes, r.src[i] + (size_t)row * r.row_bytes, r.row_bytes, &bars->full[k]);
}

// Sets the ring up and starts the first rows' copies.
__device__ __forceinline__ void ring_start(const RowRing& r, uint8_t* base, RingBars* bars, int64_t n) {
  if (threadIdx.x == 0) {
    for (int k = 0; k < r.stages; ++k) mbar_init(&bars->full[k], 1);
    fence_mbar_init();
    for (int k = 0; k < r.stages; ++k) {
      const int64_t row = blockIdx.x + (int64_t)k * gridDim.x;
      if (row < n) ring_issue(r, base, bars, row, k);
    }
  }
  __syncthreads();
}

template <typename T, int E>
__global__ void __launch_bounds__(512, E == 8 ? 2 : 1)
    norm_fwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ float buf[64];
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  const bool row_gate = a.gate && a.gate_rows;
  ring_start(ring, stage_mem, &bars, a.n);
  float wp[E], g[E], w[E];
#pragma unroll
  for (int e = 0; e < E; ++e) wp[e] = g[e] = w[e] = 0.f;
  if (in) {
    load_param<E>(a.w_post, c, wp, 1.f);
    load_param<E>(row_gate ? nullptr : reinterpret_cast<const float*>(a.gate), c, g, 1.f);
    load_param<E>(a.w_pre, c, w, 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) wp[e] *= a.res_scale * g[e];  // one factor for z on its way to x'
  }
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    float f[E], r[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = r[e] = 0.f;
    if (!mbar_wait(&bars.full[k], phase, nullptr)) return;  // the copy cannot fail to end
    const T* st = reinterpret_cast<const T*>(stage_mem + (size_t)k * ring.n_src * ring.row_bytes) + c;
    if (in) {
      load_vec<T, E>(st, f);
      if (a.y) load_vec<T, E>(st + a.D, r);
      if (row_gate) load_vec<T, E>(st + 2 * a.D, g);
    }
    __syncthreads();
    const int64_t later = row + (int64_t)ring.stages * gridDim.x;
    if (threadIdx.x == 0 && later < a.n) ring_issue(ring, stage_mem, &bars, later, k);
    if (++k == ring.stages) {
      k = 0;
      phase ^= 1;
    }
    const size_t at = (size_t)row * a.D + c;
    if (a.y) {
      float rstd = 1.f;
      if (a.w_post) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += r[e] * r[e];
        rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rstd;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf(r[e] * rstd, row_gate ? wp[e] * g[e] : wp[e], f[e]);
    }
    if (a.x_out && in) store_vec<T, E>(reinterpret_cast<T*>(a.x_out) + at, f);
    if (a.w_pre) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += f[e] * f[e];
      const float rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rstd;
      if (in) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= rstd * w[e];
        store_vec<T, E>(reinterpret_cast<T*>(a.u) + at, f);
      }
    }
  }
}

// The parameters stay in shared memory ([w_pre | res_scale g | w_post] x D fp32, a thread reads
// its own columns), the sums of their gradients in registers.
template <typename T, int E>
__global__ void __launch_bounds__(512, E == 8 ? 2 : 1)
    norm_bwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ float buf[64];
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  const bool row_gate = a.gate && a.gate_rows, pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  float* par = reinterpret_cast<float*>(stage_mem + (size_t)ring.stages * ring.n_src * ring.row_bytes);
  ring_start(ring, stage_mem, &bars, a.n);
  if (in) {
    float f[E];
    load_param<E>(a.w_pre, c, f, 1.f);
    store_vec<float, E>(par + c, f);
    load_param<E>(row_gate ? nullptr : reinterpret_cast<const float*>(a.gate), c, f, 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] *= a.res_scale;
    store_vec<float, E>(par + a.D + c, f);
    load_param<E>(a.w_post, c, f, 1.f);
    store_vec<float, E>(par + 2 * a.D + c, f);
  }
  // stage order: x (with a pre-norm), y, du, dx', gate rows, each where it is read
  const int at_y = pre ? 1 : 0, at_du = at_y + (a.y ? 1 : 0), at_dx = at_du + (pre ? 1 : 0),
            at_g = at_dx + (a.dx_in ? 1 : 0);
  float a_pre[E], a_post[E], a_gate[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a_pre[e] = a_post[e] = a_gate[e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float r_post = post ? a.rstd_post[row] : 1.f, r_pre = pre ? a.rstd_pre[row] : 1.f;
    float xn[E], yn[E], dx[E], t[E], g[E];
#pragma unroll
    for (int e = 0; e < E; ++e) xn[e] = yn[e] = dx[e] = t[e] = g[e] = 0.f;
    if (!mbar_wait(&bars.full[k], phase, nullptr)) return;  // the copy cannot fail to end
    const T* st = reinterpret_cast<const T*>(stage_mem + (size_t)k * ring.n_src * ring.row_bytes) + c;
    if (in) {
      if (pre) {
        load_vec<T, E>(st, xn);
        load_vec<T, E>(st + at_du * a.D, t);
      }
      if (a.y) load_vec<T, E>(st + at_y * a.D, yn);
      if (a.dx_in) load_vec<T, E>(st + at_dx * a.D, dx);
      load_vec<float, E>(par + a.D + c, g);
      if (row_gate) {
        float gr[E];
        load_vec<T, E>(st + at_g * a.D, gr);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] *= gr[e];
      }
    }
    __syncthreads();
    const int64_t later = row + (int64_t)ring.stages * gridDim.x;
    if (threadIdx.x == 0 && later < a.n) ring_issue(ring, stage_mem, &bars, later, k);
    if (++k == ring.stages) {
      k = 0;
      phase ^= 1;
    }
    const size_t at = (size_t)row * a.D + c;
#pragma unroll
    for (int e = 0; e < E; ++e) yn[e] *= r_post;
    if (pre) {
      float s = 0.f;
      if (in) {
        float w[E];
        if (a.y) {
          load_vec<float, E>(par + 2 * a.D + c, w);
#pragma unroll
          for (int e = 0; e < E; ++e) xn[e] = fmaf(g[e], yn[e] * w[e], xn[e]);
        }
        load_vec<float, E>(par + c, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          xn[e] *= r_pre;
          a_pre[e] = fmaf(t[e], xn[e], a_pre[e]);
          t[e] *= w[e];
          s = fmaf(t[e], xn[e], s);
        }
      }
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = fmaf(r_pre, t[e] - xn[e] * mean, dx[e]);
    }
    if (in && a.dx) store_vec<T, E>(reinterpret_cast<T*>(a.dx) + at, dx);
    if (!a.y) continue;
    float s = 0.f;
    if (in) {
      float w[E];
      load_vec<float, E>(par + 2 * a.D + c, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float z = yn[e] * w[e], dgz = a.res_scale * dx[e], dz = g[e] * dx[e];
        t[e] = dgz * z;                                // gradient of the gate
        a_post[e] = fmaf(dz, yn[e], a_post[e]);
        dx[e] = dz * w[e];
        s = fmaf(dx[e], yn[e], s);
      }
      if (row_gate && a.dgate) {
        store_vec<T, E>(reinterpret_cast<T*>(a.dgate) + at, t);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) a_gate[e] += t[e];
      }
    }
    if (post) {
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = r_post * (dx[e] - yn[e] * mean);
    }
    if (in && a.dy) store_vec<T, E>(reinterpret_cast<T*>(a.dy) + at, dx);
  }
  if (in) {
    float* dst = a.part + (size_t)blockIdx.x * 3 * a.D + c;
    store_vec<float, E>(dst, a_pre);
    store_vec<float, E>(dst + a.D, a_post);
    store_vec<float, E>(dst + 2 * a.D, a_gate);
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Elements a thread holds in the 16-byte variant: 1024 threads have to span a row.
int elements(int D) { return D <= 8192 ? 8 : 16; }

// The 16-byte variant: every row is whole threads' shares, and every row and parameter starts
// on 16 bytes.
bool vector_rows(const NormArgs& a) {
  const void* ptrs[] = {a.x, a.y, a.x_out, a.u, a.gate, a.w_pre, a.w_post, a.du, a.dx_in, a.dx, a.dy, a.dgate};
  if (a.D % elements(a.D)) return false;
  for (const void* p : ptrs)
    if (!on16(p)) return false;
  return true;
}

int threads_for(int D, int E) { return (int)align_up((size_t)((D + E - 1) / E), 32); }

// Rows through the ring where every block has at least four of them to walk and a stage
// fits; else a row is read straight into registers.
constexpr size_t kRingBytes = 200 * 1024;  // of an SM's shared memory, for all its blocks' stages
bool ring_setup(const NormArgs& a, size_t es, bool backward, RowRing* r, unsigned* grid, size_t* smem) {
  if (a.D > 8192) return false;
  const int E = a.D <= 4096 ? 8 : 16, T = threads_for(a.D, E);
  auto add = [&](const void* p) {
    if (p) r->src[r->n_src++] = reinterpret_cast<const char*>(p);
  };
  *r = {};
  if (backward) {
    if (a.w_pre) add(a.x);
    add(a.y);
    add(a.du);
    add(a.dx_in);
  } else {
    add(a.x);
    add(a.y);
  }
  if (a.gate_rows) add(a.gate);
  const size_t bytes = es * a.D;
  r->row_bytes = (uint32_t)bytes;
  const int per_sm = norm_blocks_per_sm(T);
  const int64_t blocks = std::min<int64_t>(a.n, (int64_t)per_sm * device_sm_count());
  if (a.n < 4 * blocks) return false;
  const size_t fixed = backward ? (size_t)3 * a.D * 4 : 0, room = kRingBytes / per_sm;
  if (room < fixed + 2 * bytes * r->n_src) return false;
  r->stages = (int)std::min<size_t>(kMaxStages, (room - fixed) / (bytes * r->n_src));
  *grid = (unsigned)blocks;
  *smem = r->stages * bytes * r->n_src + fixed;
  return true;
}

template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  static size_t set8[kMaxDevices] = {}, set16[kMaxDevices] = {};
  const unsigned rows = (unsigned)std::min<int64_t>(a.n, 1 << 20);
  RowRing ring;
  unsigned grid;
  size_t smem;
  if (!vector_rows(a)) {
    norm_fwd_any<T><<<rows, kSlowThreads, 0, st>>>(a);
  } else if (ring_setup(a, sizeof(T), false, &ring, &grid, &smem)) {
    const bool narrow = a.D <= 4096;
    cudaError_t e = narrow ? set_smem_limit((const void*)norm_fwd_ring<T, 8>, kRingBytes, set8)
                           : set_smem_limit((const void*)norm_fwd_ring<T, 16>, kRingBytes, set16);
    if (e != cudaSuccess) return e;
    if (narrow)
      norm_fwd_ring<T, 8><<<grid, threads_for(a.D, 8), smem, st>>>(a, ring);
    else
      norm_fwd_ring<T, 16><<<grid, threads_for(a.D, 16), smem, st>>>(a, ring);
  } else if (elements(a.D) == 8) {
    norm_fwd<T, 8><<<rows, threads_for(a.D, 8), 0, st>>>(a);
  } else {
    norm_fwd<T, 16><<<rows, threads_for(a.D, 16), 0, st>>>(a);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormArgs& a, cudaStream_t st) {
  static size_t set8[kMaxDevices] = {}, set16[kMaxDevices] = {}, set_any[kMaxDevices] = {};
  static size_t ring8[kMaxDevices] = {}, ring16[kMaxDevices] = {};
  size_t smem = (size_t)3 * a.D * 4;
  unsigned grid = (unsigned)norm_parts(a.n, a.D);
  RowRing ring;
  cudaError_t e;
  if (!vector_rows(a)) {
    e = set_smem_limit((const void*)norm_bwd_any<T>, (size_t)3 * kMaxWidth * 4, set_any);
    if (e != cudaSuccess) return e;
    norm_bwd_any<T><<<grid, kSlowThreads, smem, st>>>(a);
  } else if (ring_setup(a, sizeof(T), true, &ring, &grid, &smem)) {
    const bool narrow = a.D <= 4096;
    e = narrow ? set_smem_limit((const void*)norm_bwd_ring<T, 8>, kRingBytes, ring8)
               : set_smem_limit((const void*)norm_bwd_ring<T, 16>, kRingBytes, ring16);
    if (e != cudaSuccess) return e;
    if (narrow)
      norm_bwd_ring<T, 8><<<grid, threads_for(a.D, 8), smem, st>>>(a, ring);
    else
      norm_bwd_ring<T, 16><<<grid, threads_for(a.D, 16), smem, st>>>(a, ring);
  } else if (elements(a.D) == 8) {
    e = set_smem_limit((const void*)norm_bwd<T, 8>, (size_t)3 * 8192 * 4, set8);
    if (e != cudaSuccess) return e;
    norm_bwd<T, 8><<<grid, threads_for(a.D, 8), smem, st>>>(a);
  } else {
    e = set_smem_limit((const void*)norm_bwd<T, 16>, (size_t)3 * kMaxWidth * 4, set16);
    if (e != cudaSuccess) return e;
    norm_bwd<T, 16><<<grid, threads_for(a.D, 16), smem, st>>>(a);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  float* dgate = a.gate && !a.gate_rows ? reinterpret_cast<float*>(a.dgate) : nullptr;
  if (a.dw_pre || a.dw_post || dgate) {
    norm_join<<<dim3((a.D + 31) / 32, 3), 256, 0, st>>>(a.part, (int)grid, a.D, a.dw_pre, a.dw_post, dgate,
                                                        a.accumulate);
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

// Thread blocks of T threads on an SM: about 28 warps, at most 8 blocks.
int norm_blocks_per_sm(int T) { return std::max(1, std::min(8, 1024 / T)); }

int norm_parts(int64_t n, int D) {
  const int E = D <= 4096 ? 8 : 16;
  return (int)std::min<int64_t>(n, (int64_t)norm_blocks_per_sm((int)align_up((size_t)((D + E - 1) / E), 32)) *
                                       device_sm_count());
}

}  // namespace oomb

using namespace oomb;

extern "C" {

size_t oomb_block_norm_workspace(int n, int D) {
  if (n <= 0 || D <= 0 || D > kMaxWidth) return 0;
  return align_up((size_t)norm_parts(n, D) * 3 * D * 4, 256);
}

// Checks common to both directions; the tensors' element size.
static oomb_status check_norm(const void* x, const void* y, const float* w_post, const void* gate, int gate_rows,
                              const float* w_pre, int n, int D, int dtype, uintptr_t* es) {
  if (!x || n <= 0 || D <= 0 || (!y && !w_pre)) return OOMB_ERR_ARG;
  if (!y && (w_post || gate)) return OOMB_ERR_ARG;
  if (gate_rows != 0 && gate_rows != 1) return OOMB_ERR_ARG;
  if (dtype != OOMB_BF16 && dtype != OOMB_FP32) return OOMB_ERR_DTYPE;
  if (D > kMaxWidth) return OOMB_ERR_UNSUPPORTED;
  *es = dtype_size(dtype);
  const uintptr_t gs = gate_rows ? *es : 4;
  if (reinterpret_cast<uintptr_t>(x) % *es || reinterpret_cast<uintptr_t>(y) % *es ||
      reinterpret_cast<uintptr_t>(gate) % gs || reinterpret_cast<uintptr_t>(w_post) % 4 ||
      reinterpret_cast<uintptr_t>(w_pre) % 4)
    return OOMB_ERR_ALIGN;
  return OOMB_OK;
}

oomb_status oomb_block_norm_fwd(const void* x, const void* y, const float* w_post, const void* gate, int gate_rows,
                                const float* w_pre, float res_scale, float eps, int n, int D, int dtype, void* x_out,
                                void* u, float* rstd_post, float* rstd_pre, void* stream) {
  uintptr_t es;
  const oomb_status s = check_norm(x, y, w_post, gate, gate_rows, w_pre, n, D, dtype, &es);
  if (s != OOMB_OK) return s;
  if ((w_pre != nullptr) != (u != nullptr) || (y && !x_out) || !(eps >= 0.f)) return OOMB_ERR_ARG;
  if ((rstd_post && !w_post) || (rstd_pre && !w_pre)) return OOMB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(x_out) % es || reinterpret_cast<uintptr_t>(u) % es ||
      reinterpret_cast<uintptr_t>(rstd_post) % 4 || reinterpret_cast<uintptr_t>(rstd_pre) % 4)
    return OOMB_ERR_ALIGN;
  NormArgs a = {};
  a.x = x;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.gate_rows = gate_rows;
  a.w_pre = w_pre;
  a.res_scale = res_scale;
  a.eps = eps;
  a.n = n;
  a.D = D;
  a.inv_D = 1.f / (float)D;
  a.x_out = x_out;
  a.u = u;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  return cuda_status(dtype == OOMB_FP32 ? fwd<float>(a, (cudaStream_t)stream)
                                        : fwd<__nv_bfloat16>(a, (cudaStream_t)stream));
}

oomb_status oomb_block_norm_bwd(const void* x, const void* y, const float* w_post, const void* gate, int gate_rows,
                                const float* w_pre, float res_scale, int n, int D, int dtype, const float* rstd_post,
                                const float* rstd_pre, const void* du, const void* dx_out, void* dx, void* dy,
                                float* dw_post, void* dgate, float* dw_pre, int accumulate, void* workspace,
                                size_t ws_bytes, void* stream) {
  uintptr_t es;
  const oomb_status s = check_norm(x, y, w_post, gate, gate_rows, w_pre, n, D, dtype, &es);
  if (s != OOMB_OK) return s;
  if ((w_pre != nullptr) != (du != nullptr) || (!du && !dx_out) || !dx) return OOMB_ERR_ARG;
  if ((w_pre && !rstd_pre) || (w_post && !rstd_post) || (dy && !y)) return OOMB_ERR_ARG;
  if ((dw_pre && !w_pre) || (dw_post && !w_post) || (dgate && !gate)) return OOMB_ERR_ARG;
  if (!workspace || ws_bytes < oomb_block_norm_workspace(n, D)) return OOMB_ERR_WORKSPACE;
  const uintptr_t gs = gate_rows ? es : 4;
  if (reinterpret_cast<uintptr_t>(du) % es || reinterpret_cast<uintptr_t>(dx_out) % es ||
      reinterpret_cast<uintptr_t>(dx) % es || reinterpret_cast<uintptr_t>(dy) % es ||
      reinterpret_cast<uintptr_t>(dgate) % gs || reinterpret_cast<uintptr_t>(rstd_post) % 4 ||
      reinterpret_cast<uintptr_t>(rstd_pre) % 4 || reinterpret_cast<uintptr_t>(dw_post) % 4 ||
      reinterpret_cast<uintptr_t>(dw_pre) % 4 || reinterpret_cast<uintptr_t>(workspace) % 16)
    return OOMB_ERR_ALIGN;
  NormArgs a = {};
  a.x = x;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.gate_rows = gate_rows;
  a.w_pre = w_pre;
  a.res_scale = res_scale;
  a.n = n;
  a.D = D;
  a.inv_D = 1.f / (float)D;
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd_pre = const_cast<float*>(rstd_pre);
  a.du = du;
  a.dx_in = dx_out;
  a.dx = dx;
  a.dy = dy;
  a.dw_post = dw_post;
  a.dw_pre = dw_pre;
  a.dgate = dgate;
  a.accumulate = accumulate;
  a.part = reinterpret_cast<float*>(workspace);
  return cuda_status(dtype == OOMB_FP32 ? bwd<float>(a, (cudaStream_t)stream)
                                        : bwd<__nv_bfloat16>(a, (cudaStream_t)stream));
}

}  // extern "C"
