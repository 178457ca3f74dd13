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
//
// Two kinds of kernels: *_ring for many rows (below), which walk them with the next ones in flight,
// and norm_fwd / norm_bwd, a row straight into registers.  8192 rows, forward / backward with its
// join, direct against ring: bf16 of 3584 88 / 130 against 43 / 72 us, of 8192 213 / 285 against
// 106 / 179; fp32 of 3577 117 / 235 against 87 / 147.  512 rows of 3584: 6.5 / 16.4 against 5.7 /
// 15.3; 64 rows 3.1 / 8.0 against 3.7 / 8.3, so the forward takes the ring from one and a half rows a
// block on.  The backward takes it wherever a stage fits: its sums then stay in registers.
//
// Bounds (GB300, 8192 rows of 3584 in bf16): forward 235 MB in 43 us, 5.5 TB/s; backward 352 MB
// in 66 us, 5.3 TB/s, and the join: HBM with 80 % of the measured copy rate; the rest is the two
// sums of a row, whose barriers two blocks an SM hide only in part (issue 61 %).
#include <atomic>
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
  __device__ __forceinline__ void add(float* sums, const float (&f)[E]) const {
    float x[E];
    load<float>(sums, x);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] += f[e];
    store<float>(sums, x);
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
// A column's sums over the rows: du xn, which is dw_pre, and dx yn (times the token's gate), of which
// dw_post and a channel's dgate are multiples.  A block holds its own, here in shared memory
// ([2] x D, each column one thread's), and norm_join adds up those of the blocks.
template <typename T, int E, bool VEC>
__global__ void __launch_bounds__(1024, 1) norm_bwd(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float acc[];
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
  int turn = 0;
  const Share<E, VEC> sh(a.D);
  const bool row_gate = a.gate && a.gate_rows;
  {
    float zero[E];
#pragma unroll
    for (int e = 0; e < E; ++e) zero[e] = 0.f;
    for (int k = 0; k < 2; ++k) sh.template store<float>(acc + (size_t)k * a.D, zero);
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
        w[e] *= t[e];
        s += w[e] * xn[e];
        t[e] *= xn[e];
      }
      sh.add(acc, t);
      const float mean = block_sum<32>(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] += r_pre * (w[e] - xn[e] * mean);
    }
    if (a.dx) sh.template store<T>(reinterpret_cast<T*>(a.dx) + row0, dx);
    if (!a.y) continue;
    float s = 0.f, dg[E];
    sh.param(a.w_post, w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float dgz = a.res_scale * dx[e], dz = dgz * g[e];
      dg[e] = dgz * (z[e] * w[e]);
      g[e] = dx[e] * z[e] * (row_gate ? g[e] : 1.f);
      dx[e] = dz * w[e];
      s += dx[e] * z[e];
    }
    sh.add(acc + a.D, g);
    if (row_gate && a.dgate) sh.template store<T>(reinterpret_cast<T*>(a.dgate) + row0, dg);
    if (a.w_post) {
      const float mean = block_sum<32>(s, buf, turn) * a.inv_D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = r_post * (dx[e] - z[e] * mean);
    }
    if (a.dy) sh.template store<T>(reinterpret_cast<T*>(a.dy) + row0, dx);
  }
  for (int k = 0; k < 2; ++k) {
    float f[E];
    sh.template load<float>(acc + (size_t)k * a.D, f);
    sh.template store<float>(a.part + ((size_t)k * gridDim.x + blockIdx.x) * a.D, f);
  }
}

// The parameter gradients from the blocks' parts ([2][n_parts][D]), in block order: 32 columns a
// block, one of the two sums, 32 strips of the parts, one a warp, joined in order.
constexpr int kStrips = 32;
__global__ void __launch_bounds__(32 * kStrips) norm_join(const __grid_constant__ NormArgs a, int n_parts) {
  __shared__ float strip[kStrips][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, D = a.D;
  const int c = blockIdx.x * 32 + lane;
  const bool pre = blockIdx.y == 0;
  float* dgate = a.gate_rows ? nullptr : reinterpret_cast<float*>(a.dgate);
  if (pre ? !a.dw_pre : !a.dw_post && !dgate) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: the parts are written from here on
  const float* part = a.part + (size_t)blockIdx.y * n_parts * D + c;
  const int p0 = n_parts * w / kStrips, p1 = n_parts * (w + 1) / kStrips;
  float s = 0.f;
  if (c < D)
#pragma unroll 10
    for (int p = p0; p < p1; ++p) s += part[(size_t)p * D];
  strip[w][lane] = s;
  __syncthreads();
  if (w != 0 || c >= D) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kStrips; ++i) s += strip[i][lane];
  auto put = [&](float* out, float v) {
    if (out) out[c] = a.accumulate ? out[c] + v : v;
  };
  if (pre) {
    put(a.dw_pre, s);
  } else {
    s *= a.res_scale;
    put(a.dw_post, a.gate && !a.gate_rows ? s * reinterpret_cast<const float*>(a.gate)[c] : s);
    put(dgate, a.w_post ? s * a.w_post[c] : s);
  }
}

// ------------------------------------------------------------ rows through a ring
// Many rows: a block walks its rows with the next ones in flight.  One thread copies whole
// rows of every tensor that is read (cp.async.bulk) into a ring of stages in shared memory; the
// threads wait for a stage, take their elements into registers and hand the stage back.  So a
// block keeps stages x tensors x row bytes of loads in flight whatever its barriers wait for,
// and two blocks of an SM hide each other's sums.
// Threads of a block up to which two fit an SM (at 64 and 72 registers), and a class between those
// and 1024 that has registers to spare.
constexpr int kNarrowFwd = 512, kNarrowBwd = 448, kMiddle = 704;
constexpr int kMaxStages = 4;
constexpr int kMaxRowTensors = 5;
constexpr int kPairs = 4;  // pairs of elements a thread holds

struct RowRing {
  const char* src[kMaxRowTensors];  // tensors read, in the order they stand in a stage
  int n_src;
  uint32_t row_bytes, pitch;  // of a row in memory, and from row to row in a stage
  int stages;
  uint32_t tail;  // row that the copies leave out (its end is no multiple of 16 bytes), or ~0
  uint32_t first;  // rows below never come: 0, but for oomb_block_norm_test_timeout
};

struct __align__(16) RingBars {
  uint64_t full[kMaxStages];
};

// Error bits of the block norms on this device since the last oomb_block_norm_check.
__device__ uint32_t norm_error;

// A row's copy: the 16-byte units it lies in.
__device__ __forceinline__ void ring_issue(const RowRing& r, uint8_t* base, RingBars* bars, uint32_t row, int k) {
  if (row == r.tail) {
    mbar_arrive(&bars->full[k]);
    return;
  }
  const size_t at = (size_t)row * r.row_bytes, from = at & ~(size_t)15;
  const uint32_t bytes = (uint32_t)(((at + r.row_bytes + 15) & ~(size_t)15) - from);
  mbar_arrive_expect_tx(&bars->full[k], bytes * (uint32_t)r.n_src);
  uint8_t* dst = base + (size_t)k * r.n_src * r.pitch;
  for (int i = 0; i < r.n_src; ++i) bulk_load(dst + (size_t)i * r.pitch, r.src[i] + from, bytes, &bars->full[k]);
}

// Sets the ring up and starts the first rows' copies.
__device__ __forceinline__ void ring_start(const RowRing& r, uint8_t* base, RingBars* bars, uint32_t n) {
  if (threadIdx.x == 0) {
    for (int k = 0; k < r.stages; ++k) mbar_init(&bars->full[k], 1);
    fence_mbar_init();
    for (int k = 0; k < r.stages; ++k) {
      const uint32_t row = blockIdx.x + (uint32_t)k * gridDim.x;
      if (row >= r.first && row < n) ring_issue(r, base, bars, row, k);
    }
  }
  __syncthreads();
}

// A thread whose wait runs out (mbar_wait raises the error) leaves, at `row` in stage k.  Before that
// thread 0, which asks for the rows, waits for the copies in flight (this row's and the following
// ones'), so that none lands in shared memory that is another block's by then.  The others do not
// hang: a barrier counts the threads that have not left, and without thread 0 their waits run out.
__device__ __noinline__ void ring_give_up(const RowRing& r, RingBars* bars, uint32_t row, uint32_t n, int k,
                                          uint32_t phase) {
  if (threadIdx.x != 0) return;
  for (int j = 0; j < r.stages && row < n; ++j, row += gridDim.x) {
    mbar_wait(&bars->full[k], phase, &norm_error);
    if (++k == r.stages) {
      k = 0;
      phase ^= 1;
    }
  }
}
// In the backward its columns' sums become NaN too: the workspace holds whatever was there before.
__device__ __noinline__ void lose_sums(const NormArgs& a, int first, int step) {
  for (int h = 0; h < 2 * kPairs; ++h) {
    const int c = first + h / 2 * step + h % 2;
    if (c >= a.D) continue;
    a.part[(size_t)blockIdx.x * a.D + c] = NAN;
    a.part[((size_t)gridDim.x + blockIdx.x) * a.D + c] = NAN;
  }
}

// Packed pairs of fp32 (two elements an instruction): a row's work is bound by instructions as
// much as by its bytes.
__device__ __forceinline__ uint64_t both(float v) { return f32x2(v, v); }
__device__ __forceinline__ float halves(uint64_t v) {
  float a, b;
  f32x2_split(v, a, b);
  return a + b;
}
__device__ __forceinline__ uint64_t unpack(uint32_t bf16x2) { return f32x2(bf16x2 << 16, bf16x2 & 0xffff0000u); }

// How a block's threads share a row through the ring.  VEC: 8 consecutive elements each, 16-byte
// accesses.  Else pairs of elements, neighbouring threads on neighbouring pairs: rows of any
// width, at any offset.  (8192 rows of 3584 and of 3577, backward: bf16 72 and 117 us, fp32 124 and
// 147.)
template <bool VEC>
struct Pairs {
  int D, first, step;
  __device__ explicit Pairs(int width)
      : D(width), first((VEC ? 2 * kPairs : 2) * (int)threadIdx.x), step(VEC ? 2 : 2 * (int)blockDim.x) {}
  __device__ __forceinline__ int at(int h) const { return first + h * step; }
  __device__ __forceinline__ bool has(int h) const { return (VEC ? first : at(h)) < D; }
  __device__ __forceinline__ bool whole(int h) const { return VEC || at(h) + 1 < D; }
  // A row: `row` where every pair lies on its own size (`even`), else element by element from
  // `plain`.  Absent elements are 0.
  template <typename T>
  __device__ __forceinline__ void load(const T* row, const T* plain, bool even, uint64_t (&f)[kPairs]) const {
#pragma unroll
    for (int h = 0; h < kPairs; ++h) f[h] = 0;
    if constexpr (VEC) {
      if (!has(0)) return;
      constexpr int V = 16 / sizeof(T);
#pragma unroll
      for (int i = 0; i < 2 * kPairs; i += V) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + first + i);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[i / 2 + k] = unpack(x[k]);
        } else {
          f[i / 2] = f32x2(x[0], x[1]);
          f[i / 2 + 1] = f32x2(x[2], x[3]);
        }
      }
    } else if (even) {
#pragma unroll
      for (int h = 0; h < kPairs; ++h) {
        if (whole(h)) {
          if constexpr (sizeof(T) == 2)
            f[h] = unpack(*reinterpret_cast<const uint32_t*>(row + at(h)));
          else
            f[h] = *reinterpret_cast<const uint64_t*>(row + at(h));
        } else if (has(h)) {
          f[h] = f32x2(to_float<T>(row[at(h)]), 0.f);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < kPairs; ++h)
        if (has(h)) f[h] = f32x2(to_float<T>(plain[at(h)]), whole(h) ? to_float<T>(plain[at(h) + 1]) : 0.f);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, bool even, const uint64_t (&f)[kPairs]) const {
    if constexpr (VEC) {
      if (!has(0)) return;
      float x[2 * kPairs];
#pragma unroll
      for (int h = 0; h < kPairs; ++h) f32x2_split(f[h], x[2 * h], x[2 * h + 1]);
      store_vec<T, 2 * kPairs>(row + first, x);
    } else {
#pragma unroll
      for (int h = 0; h < kPairs; ++h) {
        if (!has(h)) continue;
        float a, b;
        f32x2_split(f[h], a, b);
        if (even && whole(h)) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint32_t*>(row + at(h)) = pack_bf16x2(a, b);
          else
            *reinterpret_cast<uint64_t*>(row + at(h)) = f[h];
        } else {
          row[at(h)] = from_float<T>(a);
          if (whole(h)) row[at(h) + 1] = from_float<T>(b);
        }
      }
    }
  }
  // A parameter (1 where there is none; nothing behind the row).
  __device__ __forceinline__ void param(const float* p, uint64_t (&f)[kPairs]) const {
#pragma unroll
    for (int h = 0; h < kPairs; ++h) f[h] = p ? 0 : both(1.f);
    if (p) load<float>(p, p, VEC, f);
  }
};

// A row of a stage.
template <typename T, bool VEC>
struct StageRow {
  const RowRing& r;
  const uint8_t* base;  // the stage, at the row's offset in its first 16-byte unit
  size_t at;            // bytes in front of the row in memory
  bool tail, even;      // even: pairs lie on their own size, in memory and in the stage
  __device__ StageRow(const RowRing& ring, const uint8_t* stage_mem, uint32_t row, int k)
      : r(ring), at((size_t)row * ring.row_bytes) {
    base = stage_mem + (size_t)k * ring.n_src * ring.pitch + (VEC ? 0 : at & 15);
    tail = !VEC && row == ring.tail;
    even = VEC || at % (2 * sizeof(T)) == 0;
  }
  __device__ __forceinline__ void load(const Pairs<VEC>& c, int i, uint64_t (&f)[kPairs]) const {
    const T* row = reinterpret_cast<const T*>(base + (size_t)i * r.pitch);
    const T* plain = tail ? reinterpret_cast<const T*>(r.src[i] + at) : row;
    c.template load<T>(row, plain, even && !tail, f);
  }
};

constexpr int kSumWarps(int threads) { return (threads + 127) / 128 * 4; }

// x' = x + (c g) (y r_post), c = res_scale gate w_post of the channel, g the token's gate.
template <typename T, bool VEC, bool ROWGATE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= kNarrowFwd ? 2 : 1)
    norm_fwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const Pairs<VEC> cols(a.D);
  const uint32_t n = (uint32_t)a.n;  // below 2^31: no sum of rows and blocks wraps
  ring_start(ring, stage_mem, &bars, n);
  uint64_t cw[kPairs], w[kPairs];
  {
    uint64_t g[kPairs];
    cols.param(a.w_post, cw);
    cols.param(ROWGATE ? nullptr : reinterpret_cast<const float*>(a.gate), g);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) cw[e] = mul2(both(a.res_scale), mul2(g[e], cw[e]));
    cols.param(a.w_pre, w);
  }
  for (uint32_t row = blockIdx.x; row < n; row += gridDim.x) {
    uint64_t f[kPairs], r[kPairs], g[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) r[e] = g[e] = 0;
    if (!mbar_wait(&bars.full[k], phase, &norm_error)) {
      ring_give_up(ring, &bars, row, n, k, phase);
      return;
    }
    const StageRow<T, VEC> st(ring, stage_mem, row, k);
    st.load(cols, 0, f);
    if (a.y) st.load(cols, 1, r);
    if (ROWGATE) st.load(cols, 2, g);
    __syncthreads();
    const uint32_t later = row + (uint32_t)ring.stages * gridDim.x;
    if (threadIdx.x == 0 && later < n) ring_issue(ring, stage_mem, &bars, later, k);
    if (++k == ring.stages) {
      k = 0;
      phase ^= 1;
    }
    const size_t at = (size_t)row * a.D;
    if (a.y) {
      float rstd = 1.f;
      if (a.w_post) {
        uint64_t s = 0;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) s = fma2(r[e], r[e], s);
        rstd = rsqrtf(block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rstd;
      }
      const uint64_t rs = both(rstd);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) f[e] = fma2(mul2(r[e], rs), ROWGATE ? mul2(cw[e], g[e]) : cw[e], f[e]);
    }
    if (a.x_out) cols.template store<T>(reinterpret_cast<T*>(a.x_out) + at, st.even, f);
    if (a.w_pre) {
      uint64_t s = 0;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) s = fma2(f[e], f[e], s);
      const float rstd = rsqrtf(block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rstd;
      const uint64_t rs = both(rstd);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) f[e] = mul2(mul2(f[e], rs), w[e]);
      cols.template store<T>(reinterpret_cast<T*>(a.u) + at, st.even, f);
    }
  }
}

// c as above.  The parameters stand in shared memory ([w_pre | c], fp32, a thread reads
// its own columns), the sums in registers.
template <typename T, bool VEC, bool ROWGATE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= kNarrowBwd ? 2 : 1)
    norm_bwd_ring(const __grid_constant__ NormArgs a, const __grid_constant__ RowRing ring) {
  // EARLY: a row is taken into registers at once and its stage handed back.  Where registers are
  // short (64, or the gate's row too), dx', the gate and c are read where they are used, twice if
  // need be, and the stage goes back at the row's last barrier.  8192 rows, early against late: bf16
  // of 3584 72 and 78 us, of 5120 114 and 129, of 8192 206 and 180; with a gate row 3584 107 and 87.
  constexpr bool EARLY = !ROWGATE && THREADS <= kMiddle;
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ RingBars bars;
  __shared__ __align__(16) float buf[64];
  clear_sums(buf);
  int turn = 0, k = 0;
  uint32_t phase = 0;
  const Pairs<VEC> cols(a.D);
  const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  const int pitch = (a.D + 3) & ~3;  // room for the absent half of the last pair
  float* par = reinterpret_cast<float*>(stage_mem + (size_t)ring.stages * ring.n_src * ring.pitch);
  auto own_param = [&](const float* p, uint64_t (&f)[kPairs]) {
    if constexpr (VEC) {
      cols.template load<float>(p, p, true, f);
    } else {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) f[e] = cols.has(e) ? *reinterpret_cast<const uint64_t*>(p + cols.at(e)) : 0;
    }
  };
  const uint32_t n = (uint32_t)a.n;  // below 2^31: no sum of rows and blocks wraps
  ring_start(ring, stage_mem, &bars, n);
  {
    uint64_t f[kPairs], g[kPairs];
    cols.param(a.w_pre, f);
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
      if (cols.has(e)) *reinterpret_cast<uint64_t*>(par + cols.at(e)) = f[e];
    cols.param(a.w_post, f);
    cols.param(ROWGATE ? nullptr : reinterpret_cast<const float*>(a.gate), g);
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
      if (cols.has(e))
        *reinterpret_cast<uint64_t*>(par + pitch + cols.at(e)) = mul2(both(a.res_scale), mul2(g[e], f[e]));
  }
  // stage order: x (with a pre-norm), y, du, dx', gate rows, each where it is read
  const int at_y = pre ? 1 : 0, at_du = at_y + (a.y ? 1 : 0), at_dx = at_du + (pre ? 1 : 0),
            at_g = at_dx + (a.dx_in ? 1 : 0);
  uint64_t a_pre[kPairs], a_post[kPairs];
#pragma unroll
  for (int e = 0; e < kPairs; ++e) a_pre[e] = a_post[e] = 0;
  if constexpr (EARLY) {
    for (uint32_t row = blockIdx.x; row < n; row += gridDim.x) {
      const float r_post = post ? a.rstd_post[row] : 1.f, r_pre = pre ? a.rstd_pre[row] : 1.f;
      uint64_t xo[kPairs], yn[kPairs], dx[kPairs], t[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) xo[e] = yn[e] = dx[e] = t[e] = 0;
      if (!mbar_wait(&bars.full[k], phase, &norm_error)) {
        ring_give_up(ring, &bars, row, n, k, phase);
        lose_sums(a, cols.first, cols.step);
        return;
      }
      const StageRow<T, VEC> st(ring, stage_mem, row, k);
      if (pre) {
        st.load(cols, 0, xo);
        st.load(cols, at_du, t);
      }
      if (a.y) st.load(cols, at_y, yn);
      if (a.dx_in) st.load(cols, at_dx, dx);
      __syncthreads();
      const uint32_t later = row + (uint32_t)ring.stages * gridDim.x;
      if (threadIdx.x == 0 && later < n) ring_issue(ring, stage_mem, &bars, later, k);
      if (++k == ring.stages) {
        k = 0;
        phase ^= 1;
      }
      const size_t at = (size_t)row * a.D;
      const uint64_t rp2 = both(r_post);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) yn[e] = mul2(yn[e], rp2);
      uint64_t cw[kPairs];
      own_param(par + pitch, cw);
      if (pre) {
        uint64_t s = 0, w[kPairs];
        const uint64_t r2 = both(r_pre);
        own_param(par, w);
        if (a.y) {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) xo[e] = fma2(cw[e], yn[e], xo[e]);
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          t[e] = mul2(t[e], r2);
          a_pre[e] = fma2(t[e], xo[e], a_pre[e]);
          t[e] = mul2(t[e], w[e]);
          s = fma2(t[e], xo[e], s);
        }
        // with t = r_pre du w: xn mean(du w xn) r_pre = x' r_pre^2 sum(t x') / D
        const float sum = block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D;
        const uint64_t m2 = both(-(sum * r_pre) * r_pre);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dx[e] = fma2(xo[e], m2, add2(t[e], dx[e]));
      }
      if (a.dx) cols.template store<T>(reinterpret_cast<T*>(a.dx) + at, st.even, dx);
      if (!a.y) continue;
      uint64_t s = 0;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        a_post[e] = fma2(dx[e], yn[e], a_post[e]);
        dx[e] = mul2(cw[e], dx[e]);
        s = fma2(dx[e], yn[e], s);
      }
      if (post) {
        const float mean = block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D;
        const uint64_t m2 = both(-r_post * mean);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dx[e] = fma2(yn[e], m2, mul2(dx[e], rp2));
      }
      if (a.dy) cols.template store<T>(reinterpret_cast<T*>(a.dy) + at, st.even, dx);
    }
  } else {
    for (uint32_t row = blockIdx.x; row < n; row += gridDim.x) {
      const float r_post = post ? a.rstd_post[row] : 1.f, r_pre = pre ? a.rstd_pre[row] : 1.f;
      uint64_t xo[kPairs], yn[kPairs], dx[kPairs], t[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) yn[e] = dx[e] = 0;
      if (!mbar_wait(&bars.full[k], phase, &norm_error)) {
        ring_give_up(ring, &bars, row, n, k, phase);
        lose_sums(a, cols.first, cols.step);
        return;
      }
      const StageRow<T, VEC> st(ring, stage_mem, row, k);
      auto hand_back = [&]() {
        const uint32_t later = row + (uint32_t)ring.stages * gridDim.x;
        if (threadIdx.x == 0 && later < n) ring_issue(ring, stage_mem, &bars, later, k);
        if (++k == ring.stages) {
          k = 0;
          phase ^= 1;
        }
      };
      const size_t at = (size_t)row * a.D;
      const uint64_t rp2 = both(r_post);
      if (a.y) st.load(cols, at_y, yn);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) yn[e] = mul2(yn[e], rp2);
      uint64_t c[kPairs];
      if (pre) {
        uint64_t s = 0;
        const uint64_t r2 = both(r_pre);
        st.load(cols, 0, xo);
        if (a.y) {
          own_param(par + pitch, c);
          if (ROWGATE) {
            uint64_t g[kPairs];
            st.load(cols, at_g, g);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) c[e] = mul2(c[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < kPairs; ++e) xo[e] = fma2(c[e], yn[e], xo[e]);
        }
        st.load(cols, at_du, t);
        {
          uint64_t w[kPairs];
          own_param(par, w);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            t[e] = mul2(t[e], r2);
            a_pre[e] = fma2(t[e], xo[e], a_pre[e]);
            t[e] = mul2(t[e], w[e]);
            s = fma2(t[e], xo[e], s);
          }
        }
        // with t = r_pre du w: xn mean(du w xn) r_pre = x' r_pre^2 sum(t x') / D
        const float sum = block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D;
        const uint64_t m2 = both(-(sum * r_pre) * r_pre);
        if (a.dx_in) st.load(cols, at_dx, dx);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dx[e] = fma2(xo[e], m2, add2(t[e], dx[e]));
      } else {
        st.load(cols, at_dx, dx);
      }
      if (a.dx) cols.template store<T>(reinterpret_cast<T*>(a.dx) + at, st.even, dx);
      if (!a.y) {
        __syncthreads();
        hand_back();
        continue;
      }
      uint64_t s = 0;
      {
        own_param(par + pitch, c);
        if (ROWGATE) {
          uint64_t g[kPairs];
          st.load(cols, at_g, g);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const uint64_t p = mul2(dx[e], yn[e]);
            a_post[e] = fma2(g[e], p, a_post[e]);
            t[e] = mul2(c[e], p);
            dx[e] = mul2(mul2(c[e], g[e]), dx[e]);
          }
          if (a.dgate) cols.template store<T>(reinterpret_cast<T*>(a.dgate) + at, st.even, t);
        } else {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            a_post[e] = fma2(dx[e], yn[e], a_post[e]);
            dx[e] = mul2(c[e], dx[e]);
          }
        }
      }
      if (post) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) s = fma2(dx[e], yn[e], s);
        const float mean = block_sum<kSumWarps(THREADS)>(halves(s), buf, turn) * a.inv_D;
        const uint64_t m2 = both(-r_post * mean);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dx[e] = fma2(yn[e], m2, mul2(dx[e], rp2));
      } else {
        __syncthreads();
      }
      hand_back();
      if (a.dy) cols.template store<T>(reinterpret_cast<T*>(a.dy) + at, st.even, dx);
    }
  }
  const size_t out = (size_t)blockIdx.x * a.D, half = (size_t)gridDim.x * a.D;
  cols.template store<float>(a.part + out, VEC || out % 2 == 0, a_pre);
  cols.template store<float>(a.part + half + out, VEC || (half + out) % 2 == 0, a_post);
}

std::atomic<bool> g_hold_first_row{false};  // oomb_block_norm_test_timeout

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Elements a thread holds in the 16-byte variant: 1024 threads have to span a row.
int elements(int D) { return D <= 8192 ? 8 : 16; }

int threads_for(int D, int E) { return (int)align_up((size_t)((D + E - 1) / E), 32); }

// Shared memory of an SM, and of a block what it takes beside the ring.
constexpr size_t kSmBytes = 228 * 1024, kBesides = 2 * 1024;
constexpr size_t kRingBytes = kSmBytes - kBesides;  // the most of one block

// Every row and parameter may start on 16 bytes (rows do if their width is right).
bool on16_all(const NormArgs& a) {
  const void* ptrs[] = {a.x, a.y, a.x_out, a.u, a.gate, a.w_pre, a.w_post, a.du, a.dx_in, a.dx, a.dy, a.dgate};
  for (const void* p : ptrs)
    if (!on16(p)) return false;
  return true;
}

// Rows through the ring, where a stage fits and (forward) every block walks at least one and a
// half rows; else a row is read straight into registers.
bool ring_setup(const NormArgs& a, size_t es, bool backward, bool vec, RowRing* r, unsigned* grid, size_t* smem) {
  const size_t bytes = es * a.D;
  if (a.D > 8192 || bytes < 64) return false;
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
  r->row_bytes = (uint32_t)bytes;
  r->pitch = (uint32_t)(vec ? bytes : align_up(bytes, 16) + 16);
  r->tail = (size_t)a.n * bytes % 16 ? (uint32_t)(a.n - 1) : ~0u;
  r->first = g_hold_first_row.load(std::memory_order_relaxed) ? 1 : 0;
  const size_t stage = (size_t)r->pitch * r->n_src, fixed = backward ? 2 * align_up((size_t)a.D, 4) * 4 : 0;
  // as many blocks on an SM as leave each two stages; one block has to do with what there is
  const int T = threads_for(a.D, 2 * kPairs);
  int per_sm = T <= (backward ? kNarrowBwd : kNarrowFwd) ? norm_blocks_per_sm(T) : 1;
  while (per_sm > 1 && kSmBytes / per_sm < kBesides + fixed + 2 * stage) --per_sm;
  const size_t room = kSmBytes / per_sm - kBesides;
  if (room < fixed + stage) return false;
  const int64_t blocks = std::min<int64_t>(a.n, (int64_t)per_sm * device_sm_count());
  if (!backward && a.n < blocks + blocks / 2) return false;
  r->stages = (int)std::min<size_t>(kMaxStages, (room - fixed) / stage);
  *grid = (unsigned)blocks;
  *smem = r->stages * stage + fixed;
  return true;
}

template <typename T, int E, bool VEC>
cudaError_t fwd_direct(const NormArgs& a, cudaStream_t st) {
  norm_fwd<T, E, VEC><<<(unsigned)std::min<int64_t>(a.n, 1 << 20), threads_for(a.D, E), 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, bool VEC, bool ROWGATE, int THREADS>
cudaError_t fwd_ring_one(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_fwd_ring<T, VEC, ROWGATE, THREADS>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_fwd_ring<T, VEC, ROWGATE, THREADS><<<grid, threads_for(a.D, 2 * kPairs), smem, st>>>(a, ring);
  return cudaGetLastError();
}
template <typename T, bool VEC, bool ROWGATE>
cudaError_t fwd_ring_width(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  const int threads = threads_for(a.D, 2 * kPairs);
  if (threads <= kNarrowFwd) return fwd_ring_one<T, VEC, ROWGATE, kNarrowFwd>(a, ring, grid, smem, st);
  if (threads <= kMiddle) return fwd_ring_one<T, VEC, ROWGATE, kMiddle>(a, ring, grid, smem, st);
  return fwd_ring_one<T, VEC, ROWGATE, 1024>(a, ring, grid, smem, st);
}
template <typename T, bool VEC>
cudaError_t fwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  return a.gate && a.gate_rows ? fwd_ring_width<T, VEC, true>(a, ring, grid, smem, st)
                               : fwd_ring_width<T, VEC, false>(a, ring, grid, smem, st);
}
template <typename T, int E, bool VEC>
cudaError_t bwd_direct(const NormArgs& a, unsigned grid, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd<T, E, VEC>, (size_t)2 * 1024 * E * 4, set);
  if (e != cudaSuccess) return e;
  norm_bwd<T, E, VEC><<<grid, threads_for(a.D, E), (size_t)2 * a.D * 4, st>>>(a);
  return cudaGetLastError();
}
template <typename T, bool VEC, bool ROWGATE, int THREADS>
cudaError_t bwd_ring_one(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)norm_bwd_ring<T, VEC, ROWGATE, THREADS>, kRingBytes, set);
  if (e != cudaSuccess) return e;
  norm_bwd_ring<T, VEC, ROWGATE, THREADS><<<grid, threads_for(a.D, 2 * kPairs), smem, st>>>(a, ring);
  return cudaGetLastError();
}
template <typename T, bool VEC, bool ROWGATE>
cudaError_t bwd_ring_width(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  const int threads = threads_for(a.D, 2 * kPairs);
  if (threads <= kNarrowBwd) return bwd_ring_one<T, VEC, ROWGATE, kNarrowBwd>(a, ring, grid, smem, st);
  if (threads <= kMiddle) return bwd_ring_one<T, VEC, ROWGATE, kMiddle>(a, ring, grid, smem, st);
  return bwd_ring_one<T, VEC, ROWGATE, 1024>(a, ring, grid, smem, st);
}
template <typename T, bool VEC>
cudaError_t bwd_ring(const NormArgs& a, const RowRing& ring, unsigned grid, size_t smem, cudaStream_t st) {
  return a.gate && a.gate_rows ? bwd_ring_width<T, VEC, true>(a, ring, grid, smem, st)
                               : bwd_ring_width<T, VEC, false>(a, ring, grid, smem, st);
}
template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  RowRing ring;
  unsigned grid;
  size_t smem;
  count_launches(1);
  const bool small = elements(a.D) == 8, aligned = on16_all(a), vec = aligned && a.D % elements(a.D) == 0;
  if (aligned && ring_setup(a, sizeof(T), false, a.D % 8 == 0, &ring, &grid, &smem))
    return a.D % 8 == 0 ? fwd_ring<T, true>(a, ring, grid, smem, st) : fwd_ring<T, false>(a, ring, grid, smem, st);
  if (!vec) return small ? fwd_direct<T, 8, false>(a, st) : fwd_direct<T, 16, false>(a, st);
  return small ? fwd_direct<T, 8, true>(a, st) : fwd_direct<T, 16, true>(a, st);
}

template <typename T>
cudaError_t bwd(const NormArgs& a, cudaStream_t st) {
  size_t smem;
  unsigned grid = (unsigned)norm_parts(a.n, a.D);
  RowRing ring;
  cudaError_t e;
  const bool small = elements(a.D) == 8, aligned = on16_all(a), vec = aligned && a.D % elements(a.D) == 0;
  if (aligned && ring_setup(a, sizeof(T), true, a.D % 8 == 0, &ring, &grid, &smem))
    e = a.D % 8 == 0 ? bwd_ring<T, true>(a, ring, grid, smem, st) : bwd_ring<T, false>(a, ring, grid, smem, st);
  else if (vec)
    e = small ? bwd_direct<T, 8, true>(a, grid, st) : bwd_direct<T, 16, true>(a, grid, st);
  else
    e = small ? bwd_direct<T, 8, false>(a, grid, st) : bwd_direct<T, 16, false>(a, grid, st);
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (a.dw_pre || a.dw_post || (a.dgate && !a.gate_rows)) {
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
    return cudaLaunchKernelEx(&cfg, norm_join, a, (int)grid);
  }
  return cudaGetLastError();
}

}  // namespace

// Thread blocks of T threads on an SM: about 28 warps, at most 8 blocks.
int norm_blocks_per_sm(int T) { return std::max(1, std::min(8, 1024 / T)); }

int norm_parts(int64_t n, int D) {
  const int T = std::min(1024, threads_for(D, 2 * kPairs));
  return (int)std::min<int64_t>(n, (int64_t)norm_blocks_per_sm(T) * device_sm_count());
}

}  // namespace oomb

using namespace oomb;

extern "C" {

size_t oomb_block_norm_workspace(int n, int D) {
  if (n <= 0 || D <= 0 || D > kMaxWidth) return 0;
  return align_up((size_t)norm_parts(n, D) * 2 * D * 4, 256);
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

oomb_status oomb_block_norm_check(void* stream, uint32_t* bits_out) {
  uint32_t bits = 0;
  const uint32_t none = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&bits, norm_error, sizeof(bits));
  if (e == cudaSuccess && bits) e = cudaMemcpyToSymbol(norm_error, &none, sizeof(none));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (bits_out) *bits_out = bits;
  if (e != cudaSuccess) return cuda_status(e);
  return bits & OOMB_DEVERR_TIMEOUT ? OOMB_ERR_TIMEOUT : bits ? OOMB_ERR_KERNEL : OOMB_OK;
}

void oomb_block_norm_test_timeout(int on) { g_hold_first_row.store(on != 0); }

}  // extern "C"
