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
// one barrier a sum is enough; the warps' sums are read as vectors by every thread (a second
// round of shuffles would wait five times as long).
// WARPS: the most warps the block may have (a multiple of 4).
template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* buf, int& turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  float* b = buf + 32 * turn;
  turn ^= 1;
  if (threadIdx.x % 32 == 0) b[threadIdx.x / 32] = v;
  __syncthreads();
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < WARPS; w += 4) {  // the entries behind the last warp stay 0
    const float4 x = *reinterpret_cast<const float4*>(b + w);
    t.x += x.x;
    t.y += x.y;
    t.z += x.z;
    t.w += x.w;
  }
  return (t.x + t.y) + (t.z + t.w);
}
// Before the first sum: no barrier of its own, the first sum's writes come before its barrier
// and touch other entries.
__device__ __forceinline__ void clear_sums(float* buf) {
  for (int i = threadIdx.x; i < 64; i += blockDim.x)
    if (i % 32 >= (int)blockDim.x / 32) buf[i] = 0.f;
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
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
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
        const float rstd = rsqrtf(block_sum<32>(s, buf, turn) * a.inv_D + a.eps);
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
      const float rstd = rsqrtf(block_sum<32>(s, buf, turn) * a.inv_D + a.eps);
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
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
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
      const float mean = block_sum<32>(s, buf, turn) * a.inv_D;
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
      const float mean = block_sum<32>(s, buf, turn) * a.inv_D;
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

// Column sums over the blocks' parts, in block order: 32 columns a block, 16 strips of the
// parts, one a warp, the strips joined in order.  out is dw_pre, dw_post or dgate (or nullptr).
constexpr int kStrips = 16;
__global__ void __launch_bounds__(32 * kStrips) norm_join(const float* __restrict__ part, int n_parts, int D,
                                                          float* dw_pre, float* dw_post, float* dgate,
                                                          int accumulate) {
  __shared__ float strip[kStrips][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, k = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float* out = k == 0 ? dw_pre : k == 1 ? dw_post : dgate;
  if (!out) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: the parts are written from here on
  const int p0 = n_parts * w / kStrips, p1 = n_parts * (w + 1) / kStrips;
  float s = 0.f;
  if (c < D)
#pragma unroll 10
    for (int p = p0; p < p1; ++p) s += part[((size_t)p * 3 + k) * D + c];
  strip[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kStrips; ++i) s += strip[i][lane];
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

// Packed pairs of fp32 (two elements an instruction): a row's work is bound by instructions as
// much as by its bytes.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return f32x2(v, v); }
__device__ __forceinline__ float halves(uint64_t v) {
  float a, b;
  f32x2_split(v, a, b);
  return a + b;
}
template <typename T, int E>
__device__ __forceinline__ void load2(const T* p, uint64_t (&f)[E / 2]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    const uint4 w = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) f[i / 2 + k] = f32x2(x[k] << 16, x[k] & 0xffff0000u);
    } else {
      f[i / 2] = f32x2(x[0], x[1]);
      f[i / 2 + 1] = f32x2(x[2], x[3]);
    }
  }
}
template <typename T, int E>
__device__ __forceinline__ void store2(T* p, const uint64_t (&f)[E / 2]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    uint32_t x[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a, b;
        f32x2_split(f[i / 2 + k], a, b);
        x[k] = pack_bf16x2(a, b);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a, b;
        f32x2_split(f[i / 2 + k], a, b);
        x[2 * k] = __float_as_uint(a);
        x[2 * k + 1] = __float_as_uint(b);
      }
    }
    *reinterpret_cast<uint4*>(p + i) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// x' = x + (c g) (y r_post), c = res_scale gate w_post of the channel, g the token's gate.
template <typename T, int E, bool ROWGATE>
__global__ void __launch_bounds__(E == 8 ? kNarrow : 512, E == 8 ? 2 : 1)
    norm_fwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  constexpr int H = E / 2;
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  ring_start(ring, stage_mem, &bars, a.n);
  uint64_t cw[H], w[H];
#pragma unroll
  for (int e = 0; e < H; ++e) cw[e] = w[e] = 0;
  if (in) {
    float f[E], g[E];
    load_param<E>(a.w_post, c, f, 1.f);
    load_param<E>(ROWGATE ? nullptr : reinterpret_cast<const float*>(a.gate), c, g, 1.f);
#pragma unroll
    for (int e = 0; e < H; ++e)
      cw[e] = f32x2(a.res_scale * g[2 * e] * f[2 * e], a.res_scale * g[2 * e + 1] * f[2 * e + 1]);
    load_param<E>(a.w_pre, c, f, 1.f);
#pragma unroll
    for (int e = 0; e < H; ++e) w[e] = f32x2(f[2 * e], f[2 * e + 1]);
  }
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    uint64_t f[H], r[H], g[H];
#pragma unroll
    for (int e = 0; e < H; ++e) f[e] = r[e] = g[e] = 0;
    if (!mbar_wait(&bars.full[k], phase, nullptr)) return;  // the copy cannot fail to end
    const T* st = reinterpret_cast<const T*>(stage_mem + (size_t)k * ring.n_src * ring.row_bytes) + c;
    if (in) {
      load2<T, E>(st, f);
      if (a.y) load2<T, E>(st + a.D, r);
      if (ROWGATE) load2<T, E>(st + 2 * a.D, g);
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
        uint64_t s = 0;
#pragma unroll
        for (int e = 0; e < H; ++e) s = fma2(r[e], r[e], s);
        rstd = rsqrtf(block_sum<16>(halves(s), buf, turn) * a.inv_D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rstd;
      }
      const uint64_t rs = both(rstd);
#pragma unroll
      for (int e = 0; e < H; ++e) f[e] = fma2(mul2(r[e], rs), ROWGATE ? mul2(cw[e], g[e]) : cw[e], f[e]);
    }
    if (a.x_out && in) store2<T, E>(reinterpret_cast<T*>(a.x_out) + at, f);
    if (a.w_pre) {
      uint64_t s = 0;
#pragma unroll
      for (int e = 0; e < H; ++e) s = fma2(f[e], f[e], s);
      const float rstd = rsqrtf(block_sum<16>(halves(s), buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rstd;
      const uint64_t rs = both(rstd);
      if (in) {
#pragma unroll
        for (int e = 0; e < H; ++e) f[e] = mul2(mul2(f[e], rs), w[e]);
        store2<T, E>(reinterpret_cast<T*>(a.u) + at, f);
      }
    }
  }
}

// With c as above and a = dx yn: dz yn = (res_scale gate) a and the gate's gradient is
// (res_scale w_post) a, so for a gate per channel one sum over the rows of a gives both
// parameter gradients.  The parameters stand in shared memory ([w_pre | c] x D fp32, a thread
// reads its own columns), the sums in registers.
template <typename T, int E, bool ROWGATE>
__global__ void __launch_bounds__(E == 8 ? kNarrow : 512, E == 8 ? 2 : 1)
    norm_bwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  constexpr int H = E / 2;
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const int c = threadIdx.x * E;
  const bool in = c < a.D;
  const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  float* par = reinterpret_cast<float*>(stage_mem + (size_t)ring.stages * ring.n_src * ring.row_bytes);
  ring_start(ring, stage_mem, &bars, a.n);
  if (in) {
    float f[E], g[E];
    load_param<E>(a.w_pre, c, f, 1.f);
    store_vec<float, E>(par + c, f);
    load_param<E>(a.w_post, c, f, 1.f);
    load_param<E>(ROWGATE ? nullptr : reinterpret_cast<const float*>(a.gate), c, g, 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] *= a.res_scale * g[e];
    store_vec<float, E>(par + a.D + c, f);
  }
  // stage order: x (with a pre-norm), y, du, dx', gate rows, each where it is read
  const int at_y = pre ? 1 : 0, at_du = at_y + (a.y ? 1 : 0), at_dx = at_du + (pre ? 1 : 0),
            at_g = at_dx + (a.dx_in ? 1 : 0);
  uint64_t a_pre[H], a_post[H];
#pragma unroll
  for (int e = 0; e < H; ++e) a_pre[e] = a_post[e] = 0;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float r_post = post ? a.rstd_post[row] : 1.f, r_pre = pre ? a.rstd_pre[row] : 1.f;
    uint64_t xo[H], yn[H], dx[H], t[H], g[H];
#pragma unroll
    for (int e = 0; e < H; ++e) xo[e] = yn[e] = dx[e] = t[e] = g[e] = 0;
    if (!mbar_wait(&bars.full[k], phase, nullptr)) return;  // the copy cannot fail to end
    const T* st = reinterpret_cast<const T*>(stage_mem + (size_t)k * ring.n_src * ring.row_bytes) + c;
    if (in) {
      if (pre) {
        load2<T, E>(st, xo);
        load2<T, E>(st + at_du * a.D, t);
      }
      if (a.y) load2<T, E>(st + at_y * a.D, yn);
      if (a.dx_in) load2<T, E>(st + at_dx * a.D, dx);
      if (ROWGATE) load2<T, E>(st + at_g * a.D, g);
    }
    __syncthreads();
    const int64_t later = row + (int64_t)ring.stages * gridDim.x;
    if (threadIdx.x == 0 && later < a.n) ring_issue(ring, stage_mem, &bars, later, k);
    if (++k == ring.stages) {
      k = 0;
      phase ^= 1;
    }
    const size_t at = (size_t)row * a.D + c;
    const uint64_t rp2 = both(r_post);
#pragma unroll
    for (int e = 0; e < H; ++e) yn[e] = mul2(yn[e], rp2);
    uint64_t cw[H];
    if (in) {
      load2<float, E>(par + a.D + c, cw);
    } else {
#pragma unroll
      for (int e = 0; e < H; ++e) cw[e] = 0;
    }
    if (pre) {
      uint64_t s = 0;
      const uint64_t r2 = both(r_pre);
      if (in) {
        uint64_t w[H];
        load2<float, E>(par + c, w);
        if (a.y) {
#pragma unroll
          for (int e = 0; e < H; ++e) xo[e] = fma2(ROWGATE ? mul2(cw[e], g[e]) : cw[e], yn[e], xo[e]);
        }
#pragma unroll
        for (int e = 0; e < H; ++e) {
          a_pre[e] = fma2(mul2(t[e], r2), xo[e], a_pre[e]);
          t[e] = mul2(t[e], w[e]);
          s = fma2(t[e], xo[e], s);
        }
      }
      // xn mean(t xn) r_pre = x' r_pre^3 sum(t x') / D
      const float sum = block_sum<16>(halves(s), buf, turn) * a.inv_D;
      const uint64_t m2 = both(-(r_pre * sum * r_pre) * r_pre);
#pragma unroll
      for (int e = 0; e < H; ++e) dx[e] = fma2(xo[e], m2, fma2(t[e], r2, dx[e]));
    }
    if (in && a.dx) store2<T, E>(reinterpret_cast<T*>(a.dx) + at, dx);
    if (!a.y) continue;
    uint64_t s = 0;
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const uint64_t p = mul2(dx[e], yn[e]);
      if (ROWGATE) {
        a_post[e] = fma2(g[e], p, a_post[e]);
        t[e] = mul2(cw[e], p);
        dx[e] = mul2(mul2(cw[e], g[e]), dx[e]);
      } else {
        a_post[e] = fma2(dx[e], yn[e], a_post[e]);
        dx[e] = mul2(cw[e], dx[e]);
      }
      s = fma2(dx[e], yn[e], s);
    }
    if (ROWGATE && a.dgate && in) store2<T, E>(reinterpret_cast<T*>(a.dgate) + at, t);
    if (post) {
      const float mean = block_sum<16>(halves(s), buf, turn) * a.inv_D;
      const uint64_t m2 = both(-r_post * mean);
#pragma unroll
      for (int e = 0; e < H; ++e) dx[e] = fma2(yn[e], m2, mul2(dx[e], rp2));
    }
    if (in && a.dy) store2<T, E>(reinterpret_cast<T*>(a.dy) + at, dx);
  }
  if (in) {
    float* dst = a.part + (size_t)blockIdx.x * 3 * a.D + c;
    float s[E], w[E], g[E];
#pragma unroll
    for (int e = 0; e < H; ++e) f32x2_split(a_pre[e], s[2 * e], s[2 * e + 1]);
    store_vec<float, E>(dst, s);
    load_param<E>(a.w_post, c, w, 1.f);
    load_param<E>(ROWGATE ? nullptr : reinterpret_cast<const float*>(a.gate), c, g, 1.f);
#pragma unroll
    for (int e = 0; e < H; ++e) f32x2_split(a_post[e], s[2 * e], s[2 * e + 1]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = a.res_scale * s[e];
      s[e] = v * g[e];
      w[e] *= v;
    }
    store_vec<float, E>(dst + a.D, s);
    store_vec<float, E>(dst + 2 * a.D, w);  // not used for a gate per token
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
  const size_t fixed = backward ? (size_t)2 * a.D * 4 : 0, room = kRingBytes / per_sm;
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
template <typename T, int E, bool ROWGATE>
cudaError_t fwd_ring_one(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_fwd_ring<T, E, ROWGATE>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_fwd_ring<T, E, ROWGATE><<<grid, threads_for(a.D, E), smem, st>>>(a, ring);
  return cudaGetLastError();
}
template <typename T, int E>
cudaError_t fwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  return a.gate && a.gate_rows ? fwd_ring_one<T, E, true>(a, ring, grid, smem, st)
                               : fwd_ring_one<T, E, false>(a, ring, grid, smem, st);
}
template <typename T, int E, bool VEC>
cudaError_t bwd_direct(const NormArgs& a, unsigned grid, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd<T, E, VEC>, (size_t)3 * 1024 * E * 4, set);
  if (e != cudaSuccess) return e;
  norm_bwd<T, E, VEC><<<grid, threads_for(a.D, E), (size_t)3 * a.D * 4, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int E, bool ROWGATE>
cudaError_t bwd_ring_one(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd_ring<T, E, ROWGATE>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_bwd_ring<T, E, ROWGATE><<<grid, threads_for(a.D, E), smem, st>>>(a, ring);
  return cudaGetLastError();
}
template <typename T, int E>
cudaError_t bwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  return a.gate && a.gate_rows ? bwd_ring_one<T, E, true>(a, ring, grid, smem, st)
                               : bwd_ring_one<T, E, false>(a, ring, grid, smem, st);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.D + 31) / 32, 3);
    cfg.blockDim = dim3(32 * kStrips);
    cfg.stream = st;
    cudaLaunchAttribute attr;  // a dependent launch: its set-up overlaps the end of the row kernel
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, norm_join, (const float*)a.part, (int)grid, a.D, a.dw_pre, a.dw_post, dgate,
                              a.accumulate);
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
