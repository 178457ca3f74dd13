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
// every run.  Widths that are no multiple of the vector, or rows off 16 bytes, are held the same
// way with one-element accesses, neighbouring threads on neighbouring elements.
#include <cmath>

#include "attn_common.cuh"
#include "block_norm.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kMaxWidth = 16384;

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

// How a block's threads share a row.  VEC: E consecutive elements each, 16-byte accesses.  Else
// elements threadIdx.x + e blockDim.x: any width and any alignment, still whole lines a warp.
template <int E, bool VEC>
struct Share {
  int c[VEC ? 1 : E];
  int D;
  __device__ explicit Share(int width) : D(width) {
    if constexpr (VEC) {
      c[0] = threadIdx.x * E;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) c[e] = threadIdx.x + e * blockDim.x;
    }
  }
  __device__ __forceinline__ bool has(int e) const { return (VEC ? c[0] : c[e]) < D; }
  __device__ __forceinline__ int at(int e) const { return VEC ? c[0] + e : c[e]; }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, float (&f)[E]) const {  // absent elements are 0
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 0.f;
    if constexpr (VEC) {
      if (has(0)) load_vec<T, E>(row + c[0], f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (has(e)) f[e] = to_float<T>(row[c[e]]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, const float (&f)[E]) const {
    if constexpr (VEC) {
      if (has(0)) store_vec<T, E>(row + c[0], f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (has(e)) row[c[e]] = from_float<T>(f[e]);
    }
  }
  __device__ __forceinline__ void param(const float* p, float (&f)[E]) const {  // 1 where there is none
    if (p) {
      load<float>(p, f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 1.f;
    }
  }
};

template <typename T, int E, bool VEC>
__device__ __forceinline__ void load_gate(const NormArgs& a, const Share<E, VEC>& sh, size_t row0, float (&g)[E]) {
  if (a.gate && a.gate_rows)
    sh.template load<T>(reinterpret_cast<const T*>(a.gate) + row0, g);
  else
    sh.param(reinterpret_cast<const float*>(a.gate), g);
}

// ------------------------------------------------------------------ forward
template <typename T, int E, bool VEC>
__global__ void __launch_bounds__(1024, 1) norm_fwd(const __grid_constant__ NormArgs a) {
  __shared__ float buf[64];
  int turn = 0;
  const Share<E, VEC> sh(a.D);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t row0 = (size_t)row * a.D;
    float f[E], r[E];
    sh.template load<T>(reinterpret_cast<const T*>(a.x) + row0, f);
    if (a.y) {
      sh.template load<T>(reinterpret_cast<const T*>(a.y) + row0, r);
      float g[E];
      load_gate<T, E, VEC>(a, sh, row0, g);
      if (a.w_post) {
        float w[E], s = 0.f;
        sh.param(a.w_post, w);
#pragma unroll
        for (int e = 0; e < E; ++e) s += r[e] * r[e];
        const float rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rstd;
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] *= rstd * w[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] += a.res_scale * g[e] * r[e];
    }
    if (a.w_pre) {
      float w[E], s = 0.f;
      sh.param(a.w_pre, w);
#pragma unroll
      for (int e = 0; e < E; ++e) s += f[e] * f[e];
      const float rstd = rsqrtf(block_sum(s, buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rstd;
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] *= f[e] * rstd;
      sh.template store<T>(reinterpret_cast<T*>(a.u) + row0, w);
    }
    if (a.x_out) sh.template store<T>(reinterpret_cast<T*>(a.x_out) + row0, f);
  }
}

// ----------------------------------------------------------------- backward
// A block's three sums of a column, in shared memory: [dw_pre | dw_post | dgate] x D.  Each
// column belongs to one thread.
template <typename T, int E, bool VEC>
__global__ void __launch_bounds__(1024, 1) norm_bwd(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float acc[];
  __shared__ float buf[64];
  int turn = 0;
  const Share<E, VEC> sh(a.D);
  const bool row_gate = a.gate && a.gate_rows;
  const bool sum_gate = a.gate && !a.gate_rows && a.dgate;
  {
    float zero[E];
#pragma unroll
    for (int e = 0; e < E; ++e) zero[e] = 0.f;
    for (int k = 0; k < 3; ++k) sh.template store<float>(acc + (size_t)k * a.D, zero);
  }
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const size_t row0 = (size_t)row * a.D;
    float g[E], z[E], dx[E], w[E];
    const float r_post = a.w_post ? a.rstd_post[row] : 1.f;
    if (a.dx_in) {
      sh.template load<T>(reinterpret_cast<const T*>(a.dx_in) + row0, dx);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = 0.f;
    }
    if (a.y) {
      sh.template load<T>(reinterpret_cast<const T*>(a.y) + row0, z);
      load_gate<T, E, VEC>(a, sh, row0, g);
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] *= r_post;  // yn
    }
    if (a.w_pre) {
      const float r_pre = a.rstd_pre[row];
      float t[E], xn[E], s = 0.f;
      sh.template load<T>(reinterpret_cast<const T*>(a.x) + row0, xn);
      sh.template load<T>(reinterpret_cast<const T*>(a.du) + row0, t);
      if (a.y) {
        sh.param(a.w_post, w);
#pragma unroll
        for (int e = 0; e < E; ++e) xn[e] += a.res_scale * g[e] * (z[e] * w[e]);
      }
      sh.param(a.w_pre, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xn[e] *= r_pre;
        if (sh.has(e)) acc[sh.at(e)] += t[e] * xn[e];
        t[e] *= w[e];
        s += t[e] * xn[e];
      }
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] += r_pre * (t[e] - xn[e] * mean);
    }
    if (a.dx) sh.template store<T>(reinterpret_cast<T*>(a.dx) + row0, dx);
    if (!a.y) continue;
    float s = 0.f, dg[E];
    sh.param(a.w_post, w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float dgz = a.res_scale * dx[e], dz = dgz * g[e];
      dg[e] = dgz * (z[e] * w[e]);
      if (a.w_post && sh.has(e)) acc[a.D + sh.at(e)] += dz * z[e];
      if (sum_gate && sh.has(e)) acc[2 * a.D + sh.at(e)] += dg[e];
      dx[e] = dz * w[e];
      s += dx[e] * z[e];
    }
    if (row_gate && a.dgate) sh.template store<T>(reinterpret_cast<T*>(a.dgate) + row0, dg);
    if (a.w_post) {
      const float mean = block_sum(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = r_post * (dx[e] - z[e] * mean);
    }
    if (a.dy) sh.template store<T>(reinterpret_cast<T*>(a.dy) + row0, dx);
  }
  for (int k = 0; k < 3; ++k) {
    float f[E];
    sh.template load<float>(acc + (size_t)k * a.D, f);
    sh.template store<float>(a.part + ((size_t)blockIdx.x * 3 + k) * a.D, f);
  }
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
constexpr int kNarrow = 448;  // threads up to which a thread holds 8 elements: two blocks fit 72 registers
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
__global__ void __launch_bounds__(E == 8 ? kNarrow : 512, E == 8 ? 2 : 1)
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
__global__ void __launch_bounds__(E == 8 ? kNarrow : 512, E == 8 ? 2 : 1)
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

int ring_elements(int D) { return D <= 8 * kNarrow ? 8 : 16; }

// Rows through the ring where every block has at least four of them to walk and a stage
// fits; else a row is read straight into registers.
constexpr size_t kRingBytes = 200 * 1024;  // of an SM's shared memory, for all its blocks' stages
bool ring_setup(const NormArgs& a, size_t es, bool backward, RowRing* r, unsigned* grid, size_t* smem) {
  if (a.D > 8192 || a.D % ring_elements(a.D)) return false;
  const int T = threads_for(a.D, ring_elements(a.D));
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

template <typename T, int E, bool VEC>
cudaError_t fwd_direct(const NormArgs& a, cudaStream_t st) {
  norm_fwd<T, E, VEC><<<(unsigned)std::min<int64_t>(a.n, 1 << 20), threads_for(a.D, E), 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int E>
cudaError_t fwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_fwd_ring<T, E>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_fwd_ring<T, E><<<grid, threads_for(a.D, E), smem, st>>>(a, ring);
  return cudaGetLastError();
}
template <typename T, int E, bool VEC>
cudaError_t bwd_direct(const NormArgs& a, unsigned grid, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd<T, E, VEC>, (size_t)3 * 1024 * E * 4, set);
  if (e != cudaSuccess) return e;
  norm_bwd<T, E, VEC><<<grid, threads_for(a.D, E), (size_t)3 * a.D * 4, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int E>
cudaError_t bwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd_ring<T, E>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_bwd_ring<T, E><<<grid, threads_for(a.D, E), smem, st>>>(a, ring);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  RowRing ring;
  unsigned grid;
  size_t smem;
  count_launches(1);
  const bool small = elements(a.D) == 8;
  if (!vector_rows(a)) return small ? fwd_direct<T, 8, false>(a, st) : fwd_direct<T, 16, false>(a, st);
  if (ring_setup(a, sizeof(T), false, &ring, &grid, &smem))
    return ring_elements(a.D) == 8 ? fwd_ring<T, 8>(a, ring, grid, smem, st) : fwd_ring<T, 16>(a, ring, grid, smem, st);
  return small ? fwd_direct<T, 8, true>(a, st) : fwd_direct<T, 16, true>(a, st);
}

template <typename T>
cudaError_t bwd(const NormArgs& a, cudaStream_t st) {
  size_t smem;
  unsigned grid = (unsigned)norm_parts(a.n, a.D);
  RowRing ring;
  cudaError_t e;
  const bool small = elements(a.D) == 8;
  if (!vector_rows(a))
    e = small ? bwd_direct<T, 8, false>(a, grid, st) : bwd_direct<T, 16, false>(a, grid, st);
  else if (ring_setup(a, sizeof(T), true, &ring, &grid, &smem))
    e = ring_elements(a.D) == 8 ? bwd_ring<T, 8>(a, ring, grid, smem, st) : bwd_ring<T, 16>(a, ring, grid, smem, st);
  else
    e = small ? bwd_direct<T, 8, true>(a, grid, st) : bwd_direct<T, 16, true>(a, grid, st);
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
  const int E = ring_elements(D);
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
