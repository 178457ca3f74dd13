// The loss over a vocabulary (head_loss.cu) for few rows, and for small problems, on the CUDA cores.
//
// A few rows leave nearly all of a tensor-core tile empty and W is what has to be read: a warp
// takes four of W's rows at a time, whole rows in order, and the vectors x of up to eight tokens stand
// in shared memory in fp32.  A warp's 4 x 8 sums are joined over its lanes by a transposing
// reduction (31 shuffles for 32 sums), after which each lane has one logit.  fp32 arithmetic throughout,
// with fp32 operands read as they are.  Backward: the logits again, dz kept in fp32, then dx and dw by
// blocks of their own, side by side: one reads W, the other writes dw.
//
//   dot_rows    forward: maximum and sum of exponentials of a warp's logits, the targets' logits;
//               backward: dz
//   grad_rows   dx in parts of the vocabulary, dw
//   join_rows   dx from its parts, in order
// No row is gathered: rows without a target are not read and cost no more than a test.
//
// Small problems (kSmallWork) take it for their latency: two launches forward and three backward against
// three to ten, and none that sets up tensor memory.
#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "head_loss.h"
#include "sm103_ptx.cuh"

namespace oomb {
namespace head {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 4;                       // of W a warp (dot) or a thread (grad) has in hand
constexpr int kCols = 8;                       // columns of a thread
constexpr size_t kMaxVectors = 200 * 1024;     // shared memory for x
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ bool has_target(const SmallArgs& a, int i) {
  const int64_t t = a.targets[i];
  return t >= 0 && t < a.V;
}

// Eight columns of a row, as they are stored: VEC eight that follow one another from c, 16 bytes an access; else
// c, c + step, ... element by element, so that neighbouring threads read neighbouring columns.  Columns behind the
// last are 0.  (One row on 131072 x 3583: 230 us forward in bf16 and 287 in
// fp32, with eight that follow one another here too 279 and 462.)
template <typename T, bool VEC>
struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* row, int c, int step, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        raw[i] = c < D ? *reinterpret_cast<const uint4*>(row + c + i * (16 / sizeof(T))) : make_uint4(0, 0, 0, 0);
    } else {
      T* x = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int e = 0; e < kCols; ++e) x[e] = c + e * step < D ? row[c + e * step] : from_float<T>(0.f);
    }
  }
  __device__ __forceinline__ void pairs(uint64_t (&f)[kCols / 2]) const {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
    for (int k = 0; k < kCols / 2; ++k) {
      if constexpr (sizeof(T) == 2)
        f[k] = f32x2(x[k] << 16, x[k] & 0xffff0000u);
      else
        f[k] = f32x2(x[2 * k], x[2 * k + 1]);
    }
  }
};

// z' = cap tanh(z / cap), and tanh
__device__ __forceinline__ float cap_logit(float z, float cap, float& th) {
  th = 0.f;
  if (cap > 0.f) {
    th = tanhf(z / cap);
    z = cap * th;
  }
  return z;
}

// ------------------------------------------------------------------ logits
// NT: tokens at a time.  grid.y: groups of NT tokens.  DZ: dz is stored, else parts of the row sums.
template <typename T, bool VEC, int NT, bool DZ>
__global__ void __launch_bounds__(kThreads, 2) dot_rows(const __grid_constant__ SmallArgs a) {
  constexpr int kStride = VEC ? kCols : 1;  // between the first columns of two lanes
  constexpr int K = kRows * NT, LOG = K == 32 ? 5 : K == 16 ? 4 : K == 8 ? 3 : 2, DEPTH = sizeof(T) == 4 ? (NT <= 2 ? 2 : 1) : NT == 8 ? 1 : NT == 4 ? 2 : 3;
  // [NT, steps of 256 columns], zeros behind a row; of a step first every lane's first four columns, then the
  // others, so that a warp's 16-byte reads lie side by side
  extern __shared__ __align__(16) float xs[];
  wait_for_launch_before();
  let_next_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t0 = blockIdx.y * NT, steps = (a.D + 255) / 256, pitch = steps * 256;
  if (blockIdx.x == 0)
    for (int t = threadIdx.x; t < NT && t0 + t < a.n; t += kThreads)
      if (a.targets[t0 + t] >= a.V) atomicOr(a.err, OOMB_DEVERR_TOKEN);
  for (int t = 0; t < NT; ++t) {
    const bool has = t0 + t < a.n && has_target(a, t0 + t);
    const T* x = reinterpret_cast<const T*>(a.x) + (size_t)(t0 + t) * a.D;
#pragma unroll 2
    for (int c = threadIdx.x * kCols; c < pitch; c += kThreads * kCols) {
      Eight<T, VEC> raw;
      raw.load(x, VEC ? c : (c & ~255) + (c & 255) / kCols, 32, has ? a.D : 0);
      uint64_t f[kCols / 2];
      raw.pairs(f);
      float* to = xs + t * pitch + (c & ~255) + (c & 255) / 2;
      *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(f[0], f[1]);
      *reinterpret_cast<ulonglong2*>(to + 128) = make_ulonglong2(f[2], f[3]);
    }
  }
  __syncthreads();
  // after the reduction lane l has sum l >> (5 - LOG): row and token
  const int mine = lane >> (5 - LOG), row = mine / NT, tok = mine % NT;
  const bool writes = (lane & ((32 >> LOG) - 1)) == 0 && t0 + tok < a.n && has_target(a, min(t0 + tok, a.n - 1));
  const int64_t target = t0 + tok < a.n ? a.targets[t0 + tok] : -1;
  float lse2 = 0.f, g = 1.f;
  if (DZ && t0 + tok < a.n) {
    lse2 = a.lse_in[t0 + tok] * kLog2e;
    if (a.d_loss) g = a.d_loss[t0 + tok];
  }
  float m = -INFINITY, s = 0.f;  // base 2
  const int groups = (a.V + kRows - 1) / kRows;
  for (int gr = blockIdx.x * kWarps + warp; gr < groups; gr += gridDim.x * kWarps) {
    const int v0 = gr * kRows;
    const T* w[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) w[r] = reinterpret_cast<const T*>(a.w) + (size_t)min(v0 + r, a.V - 1) * a.D;
    Eight<T, VEC> raw[DEPTH][kRows];
    uint64_t acc[kRows][NT];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = 0;
#pragma unroll
    for (int u = 0; u < DEPTH; ++u)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (u < steps) raw[u][r].load(w[r], u * 256 + lane * kStride, 32, a.D);
    for (int s0 = 0; s0 < steps; s0 += DEPTH) {
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) {
        if (s0 + u >= steps) break;
        uint64_t f[kRows][kCols / 2];
#pragma unroll
        for (int r = 0; r < kRows; ++r) raw[u][r].pairs(f[r]);
        if (s0 + u + DEPTH < steps)
#pragma unroll
          for (int r = 0; r < kRows; ++r) raw[u][r].load(w[r], (s0 + u + DEPTH) * 256 + lane * kStride, 32, a.D);
        const float* xp = xs + (s0 + u) * 256 + lane * 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const ulonglong2 x0 = *reinterpret_cast<const ulonglong2*>(xp + t * pitch);
          const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(xp + t * pitch + 128);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            acc[r][t] = fma2(f[r][0], x0.x, acc[r][t]);
            acc[r][t] = fma2(f[r][1], x0.y, acc[r][t]);
            acc[r][t] = fma2(f[r][2], x1.x, acc[r][t]);
            acc[r][t] = fma2(f[r][3], x1.y, acc[r][t]);
          }
        }
      }
    }
    float z[K];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float lo, hi;
        f32x2_split(acc[r][t], lo, hi);
        z[r * NT + t] = lo + hi;
      }
    int cnt = K;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      if (cnt > 1) {
        cnt /= 2;
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < K / 2; ++i) {
          if (i >= cnt) break;
          const float send = up ? z[i] : z[i + cnt], keep = up ? z[i + cnt] : z[i];
          z[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      } else {
        z[0] += __shfl_xor_sync(0xffffffffu, z[0], off);
      }
    }
    const int v = v0 + row;
    float th;
    const float zz = cap_logit(z[0], a.cap, th);
    if (v >= a.V || !writes) continue;
    if constexpr (DZ) {
      float q = ex2_approx(fmaf(zz, kLog2e, -lse2));
      if (v == target) q -= 1.f;
      a.dz[(size_t)(t0 + tok) * a.pitch + v] = q * (g * fmaf(-th, th, 1.f));
    } else if (v == target) {  // kept out of the sum, which it joins at the end
      a.at[t0 + tok] = zz;
    } else {
      const float z2 = zz * kLog2e, to = fmaxf(m, z2), ref = to == -INFINITY ? 0.f : to;
      s = s * ex2_approx(m - ref) + ex2_approx(z2 - ref);
      m = to;
    }
  }
  if constexpr (!DZ) {
    // the lanes of a token: row slots
#pragma unroll
    for (int off = 16; off >= (32 >> LOG) * NT; off >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off), s2 = __shfl_xor_sync(0xffffffffu, s, off);
      const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.f : to;
      s = s * ex2_approx(m - ref) + s2 * ex2_approx(m2 - ref);
      m = to;
    }
    if (row == 0 && writes)
      a.part[(size_t)(t0 + tok) * a.parts + blockIdx.x * kWarps + warp] = make_float2(m, s);
  }
}

// Loss and log-sum-exp, a block a token.
__global__ void __launch_bounds__(kThreads) join_loss(const __grid_constant__ SmallArgs a) {
  __shared__ float2 share[kWarps];
  wait_for_launch_before();
  let_next_launch();
  const int i = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (!has_target(a, i)) {
    if (threadIdx.x == 0) a.loss[i] = a.lse[i] = 0.f;
    return;
  }
  float m = -INFINITY, s = 0.f;
  auto add = [&](float m2, float s2) {
    const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.f : to;
    s = s * ex2_approx(m - ref) + s2 * ex2_approx(m2 - ref);
    m = to;
  };
#pragma unroll 4
  for (int k = threadIdx.x; k < a.parts; k += kThreads) {
    const float2 p = a.part[(size_t)i * a.parts + k];
    add(p.x, p.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    add(m2, s2);
  }
  if (lane == 0) share[warp] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) add(share[w].x, share[w].y);
  loss_of(a.at[i], m, s, a.loss[i], a.lse[i]);
}

// ------------------------------------------------------------------ gradients
// grid.z: dx of eight tokens each, then dw.  grid.y: slabs of columns; threadIdx.x % ct: eight columns,
// / ct: row group.
template <typename T, typename TW, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) grad_rows(const __grid_constant__ SmallArgs a) {
  constexpr int NT = 8;
  __shared__ unsigned char has[kMaxRows];
  wait_for_launch_before();
  let_next_launch();
  for (int t = threadIdx.x; t < a.n; t += blockDim.x) has[t] = has_target(a, t);
  __syncthreads();
  const int group = threadIdx.x / a.ct, step = VEC ? 1 : a.ct;  // step: between a thread's columns
  const int c = blockIdx.y * a.ct * kCols + threadIdx.x % a.ct * (VEC ? kCols : 1);
  const int units = gridDim.x * a.row_groups, unit = blockIdx.x * a.row_groups + group;
  if (group >= a.row_groups || c >= a.D) return;
  const int chunks = (a.V + kRows - 1) / kRows;
  const int first = (int)((int64_t)chunks * unit / units), end = (int)((int64_t)chunks * (unit + 1) / units);
  if (a.dw && blockIdx.z == gridDim.z - 1) {
    for (int ch = first; ch < end; ++ch) {
      const int v0 = ch * kRows;
      uint64_t acc[kRows][kCols / 2];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) acc[r][k] = 0;
      constexpr int B = 4;  // tokens asked for together
      for (int t0 = 0; t0 < a.n; t0 += B) {
        Eight<T, VEC> raw[B];
        float4 d[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const bool live = t0 + u < a.n && has[t0 + u];  // (a token without a target is not read)
          raw[u].load(reinterpret_cast<const T*>(a.x) + (size_t)(live ? t0 + u : 0) * a.D, c, step, live ? a.D : 0);
          // (rows of W behind the last: not used)
          d[u] = live ? *reinterpret_cast<const float4*>(a.dz + (size_t)(t0 + u) * a.pitch + v0)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
          if (t0 + u >= a.n) break;
          uint64_t x[kCols / 2];
          raw[u].pairs(x);
          const float dd[kRows] = {d[u].x, d[u].y, d[u].z, d[u].w};
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const uint64_t dr = f32x2(dd[r], dd[r]);
#pragma unroll
            for (int k = 0; k < kCols / 2; ++k) acc[r][k] = fma2(dr, x[k], acc[r][k]);
          }
        }
      }
      // rows whose old values (fp32 only) are asked for together (a row of 131072 x 3584 in bf16, backward with dw
      // added: 951 us, a vector at a time 1089)
      constexpr int R = 2;
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += R) {
        float old[R][kCols];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < kCols; ++e) old[r][e] = 0.f;
        if (sizeof(TW) == 4 && a.accumulate) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float* from = reinterpret_cast<const float*>(a.dw) + (size_t)min(v0 + r0 + r, a.V - 1) * a.D + c;
            if (a.dw_vec) {
#pragma unroll
              for (int e = 0; e < kCols; e += 4) {
                const float4 o = *reinterpret_cast<const float4*>(from + e);
                old[r][e] = o.x;
                old[r][e + 1] = o.y;
                old[r][e + 2] = o.z;
                old[r][e + 3] = o.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < kCols; ++e)
                if (c + e * step < a.D) old[r][e] = from[e * step];
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (v0 + r0 + r >= a.V) break;
          TW* to = reinterpret_cast<TW*>(a.dw) + (size_t)(v0 + r0 + r) * a.D + c;
          float f[kCols];
#pragma unroll
          for (int k = 0; k < kCols / 2; ++k) f32x2_split(acc[r0 + r][k], f[2 * k], f[2 * k + 1]);
#pragma unroll
          for (int e = 0; e < kCols; ++e) f[e] = fmaf(a.scale, f[e], old[r][e]);
          if (a.dw_vec) {
            if constexpr (sizeof(TW) == 2) {
              *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                         pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            } else {
#pragma unroll
              for (int e = 0; e < kCols; e += 4)
                *reinterpret_cast<float4*>(to + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < kCols; ++e)
              if (c + e * step < a.D) to[e * step] = from_float<TW>(f[e]);
          }
        }
      }
    }
    return;
  }
  {
    const int t0 = blockIdx.z * NT;
    uint64_t acc[NT][kCols / 2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < kCols / 2; ++k) acc[t][k] = 0;
    for (int ch = first; ch < end; ++ch) {
      const int v0 = ch * kRows;
      Eight<T, VEC> raw[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        raw[r].load(reinterpret_cast<const T*>(a.w) + (size_t)min(v0 + r, a.V - 1) * a.D, c, step, a.D);
      float dd[NT][kRows];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bool live = t0 + t < a.n && has[t0 + t];
        const float4 d = live ? *reinterpret_cast<const float4*>(a.dz + (size_t)(t0 + t) * a.pitch + v0)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        dd[t][0] = d.x;
        dd[t][1] = v0 + 1 < a.V ? d.y : 0.f;
        dd[t][2] = v0 + 2 < a.V ? d.z : 0.f;
        dd[t][3] = v0 + 3 < a.V ? d.w : 0.f;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        uint64_t w[kCols / 2];
        raw[r].pairs(w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t0 + t >= a.n) break;
          const uint64_t dr = f32x2(dd[t][r], dd[t][r]);
#pragma unroll
          for (int k = 0; k < kCols / 2; ++k) acc[t][k] = fma2(dr, w[k], acc[t][k]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t0 + t >= a.n || !has[t0 + t]) continue;
      float* to = a.acc + ((size_t)unit * a.n + t0 + t) * a.acc_pitch + c;
      float f[kCols];
#pragma unroll
      for (int k = 0; k < kCols / 2; ++k) f32x2_split(acc[t][k], f[2 * k], f[2 * k + 1]);
      if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < kCols; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < kCols; ++e)
          if (c + e * step < a.D) to[e * step] = f[e];
      }
    }
  }
}

// dx of 32 columns of a token from its parts, a strip of the parts a warp, the strips in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_rows(const __grid_constant__ SmallArgs a, int units) {
  __shared__ float strip[kWarps][33];
  wait_for_launch_before();
  let_next_launch();
  const int i = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  const bool has = has_target(a, i);
  const int per = (units + kWarps - 1) / kWarps, end = min(units, (warp + 1) * per);
  float sum = 0.f;
  if (has && c < a.D) {
#pragma unroll 8
    for (int u = warp * per; u < end; ++u) sum += a.acc[((size_t)u * a.n + i) * a.acc_pitch + c];
  }
  strip[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= a.D) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) sum += strip[w][lane];
  reinterpret_cast<T*>(a.dx)[(size_t)i * a.D + c] = from_float<T>(has ? a.scale * sum : 0.f);
}

// ------------------------------------------------------------------ host side
template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
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

size_t vector_bytes(int D) { return align_up((size_t)D, 256) * 4; }

// Blocks of dot_rows for a vocabulary: two an SM, warps that have four rows at least.
int dot_blocks(int V) { return std::max(1, std::min(2 * device_sm_count(), (V + kRows * kWarps - 1) / (kRows * kWarps))); }

template <typename T, bool VEC, int NT, bool DZ>
cudaError_t dot(const SmallArgs& a, cudaStream_t st) {
  static size_t set[kMaxDevices] = {};
  const cudaError_t e = set_smem_limit((const void*)dot_rows<T, VEC, NT, DZ>, kMaxVectors, set);
  if (e != cudaSuccess) return e;
  return launch(dot_rows<T, VEC, NT, DZ>, dim3((unsigned)dot_blocks(a.V), (unsigned)((a.n + NT - 1) / NT)),
                kThreads, NT * vector_bytes(a.D), st, a);
}
template <typename T, bool VEC, bool DZ>
cudaError_t dot_tokens(const SmallArgs& a, cudaStream_t st) {
  // as many tokens at a time as there are and shared memory holds, but no more than leave every SM a
  // block: a short vocabulary's rows are in L2 for the next tokens
  auto takes = [&](int nt) {
    return a.n > nt / 2 && nt * vector_bytes(a.D) <= kMaxVectors &&
           (int64_t)dot_blocks(a.V) * ((a.n + nt - 1) / nt) >= device_sm_count();
  };
  if constexpr (sizeof(T) == 2)  // (fp32: the registers hold four tokens' sums)
    if (takes(8)) return dot<T, VEC, 8, DZ>(a, st);
  if (takes(4)) return dot<T, VEC, 4, DZ>(a, st);
  if (takes(2)) return dot<T, VEC, 2, DZ>(a, st);
  return dot<T, VEC, 1, DZ>(a, st);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Columns' threads, row groups of a block, slabs and blocks of grad_rows: up to 512 parts of the
// vocabulary, over two blocks an SM before more go into one block.
struct GradGrid {
  int ct, row_groups, slabs, blocks;
};
GradGrid grad_grid(int D, int V) {
  GradGrid g;
  const int threads = (D + kCols - 1) / kCols;
  g.slabs = (threads + kThreads - 1) / kThreads;
  g.ct = (threads + g.slabs - 1) / g.slabs;
  const int units = std::min(512, (V + kRows - 1) / kRows), most = std::max(1, 2 * device_sm_count() / g.slabs);
  g.blocks = std::min(units, most);
  g.row_groups = std::max(1, std::min(kThreads / g.ct, (units + g.blocks - 1) / g.blocks));
  return g;
}

template <typename T>
cudaError_t backward(SmallArgs a, int dw_dtype, cudaStream_t st) {
  const bool vec = a.D % 8 == 0 && on16(a.x) && on16(a.w);
  cudaError_t e = vec ? dot_tokens<T, true, true>(a, st) : dot_tokens<T, false, true>(a, st);
  if (e != cudaSuccess) return e;
  const GradGrid g = grad_grid(a.D, a.V);
  a.ct = g.ct;
  a.row_groups = g.row_groups;
  a.dw_vec = vec && on16(a.dw);
  const int threads = (int)align_up((size_t)g.ct * g.row_groups, 32);
  const dim3 grid((unsigned)g.blocks, (unsigned)g.slabs, (unsigned)((a.dx ? (a.n + 7) / 8 : 0) + (a.dw ? 1 : 0)));
  if (dw_dtype == OOMB_FP32)
    e = vec ? launch(grad_rows<T, float, true>, grid, threads, 0, st, a) : launch(grad_rows<T, float, false>, grid, threads, 0, st, a);
  else
    e = vec ? launch(grad_rows<T, __nv_bfloat16, true>, grid, threads, 0, st, a)
            : launch(grad_rows<T, __nv_bfloat16, false>, grid, threads, 0, st, a);
  if (e != cudaSuccess || !a.dx) return e;
  return launch(join_rows<T>, dim3((unsigned)((a.D + 31) / 32), (unsigned)a.n), kThreads, 0, st, a, g.blocks * g.row_groups);
}

}  // namespace

int small_rows(int D, int V, int dtype) {
  if (vector_bytes(D) > kMaxVectors) return 0;
  const bool fp32 = dtype == OOMB_FP32;
  const int64_t rows = (fp32 ? kSmallWork32 : kSmallWork) / ((int64_t)std::max(D, kSmallWidth) * V);
  return (int)std::min<int64_t>(kMaxRows, std::max<int64_t>(fp32 ? kFewRows32 : kFewRows, rows));
}

size_t small_space(int n, int D, int V, bool backward, SmallSpace* s) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  s->parts = dot_blocks(V) * kWarps;
  s->at = take((size_t)n * 4);
  s->part = take((size_t)n * s->parts * 8);
  if (backward) {
    const GradGrid g = grad_grid(D, V);
    s->pitch = (int)align_up((size_t)V, kRows);
    s->acc_pitch = (int)align_up((size_t)D, kCols);
    s->dz = take((size_t)n * s->pitch * 4);
    s->acc = take((size_t)g.blocks * g.row_groups * n * s->acc_pitch * 4);
  }
  return at;
}

cudaError_t launch_small_fwd(const SmallArgs& a, int dtype, cudaStream_t st) {
  const bool vec = a.D % 8 == 0 && on16(a.x) && on16(a.w);
  cudaError_t e;
  if (dtype == OOMB_FP32)
    e = vec ? dot_tokens<float, true, false>(a, st) : dot_tokens<float, false, false>(a, st);
  else
    e = vec ? dot_tokens<__nv_bfloat16, true, false>(a, st) : dot_tokens<__nv_bfloat16, false, false>(a, st);
  if (e != cudaSuccess) return e;
  return launch(join_loss, dim3((unsigned)a.n), kThreads, 0, st, a);
}

cudaError_t launch_small_bwd(const SmallArgs& a, int dtype, int dw_dtype, cudaStream_t st) {
  return dtype == OOMB_FP32 ? backward<float>(a, dw_dtype, st) : backward<__nv_bfloat16>(a, dw_dtype, st);
}

}  // namespace head
}  // namespace oomb
