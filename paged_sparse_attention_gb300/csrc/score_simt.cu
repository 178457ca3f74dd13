// Chunk attention with capped scores, a distance bias and per-row key ranges on the CUDA
// cores in fp32, for fp32 pools and for the bf16 shapes the tensor-core kernels do not
// take; also the join of split forwards and the document ranges.
//
// Tiles of 64 query rows x 64 keys, 256 threads, a 4 x 4 block of scores per thread: each
// 16-byte read of shared memory feeds 8 multiply-adds.  The keys of a tile are 64 consecutive tokens of the
// selected pages written one after another, so a page may be of any size: a tile can hold
// several small pages or a part of a large one.  Rows whose range is empty, or meets no
// selected page, get O = 0 and LSE = -inf and send no gradient.
//
//   score_fwd_simt   a block per (64 rows, query head, share of the keys); running maximum
//                    and sum, O in registers
//   score_join       the shares of a split forward joined by their log-sum-exps
//   score_dot        D_i = dO_i . O_i
//   score_dq_simt    a block per (64 rows, query head, share of the keys): dQ
//   score_dkdv_simt  a block per (64 keys of the selection, KV head, share of the rows and
//                    query heads of the group): dK and dV of those keys, added once into the
//                    pool rows, which no other block touches (same bits on every run)
//   score_dq_join, score_dkdv_join   the shares of both added up in order, where tiles alone do
//                    not fill the SMs
//
// Shares against none, fp32, 1024 rows of 2 heads on 4096 tokens in documents of 1000, forward and
// backward with its joins: 150 us call after call (130 of them on the device) against 539.  One by
// one from a cold cache the forward takes 29, dQ 36, dK/dV 48, each with a block or two an SM, the
// joins 27, D and the ranges 7.  With more rows, 900 of 6 heads on 3000 keys: 172 us (20 of
// the FMA pipe's 74 TFLOP/s) and 483 (25 with the scores that both passes form).  Bound by shared
// memory, its reads and their latency at two blocks of 8 warps an SM (d <= 64; 128 registers); 8 x 4
// scores a thread (194 / 513) and, for d > 64, 2 x 4 (1515 against 1175 backward) are slower.
#include <climits>
#include <cmath>

#include "score_common.cuh"
#include "sm103_ptx.cuh"

namespace oomb {
namespace {

constexpr int kRows = 64;   // query rows of a tile
constexpr int kKeys = 64;   // keys of a tile
constexpr int kThreads = 256;
constexpr int kMaxD = 128;
constexpr int kLdP = kKeys + 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxParts = 1024;  // of a split forward; 32 on this path, 2 an SM at most on the tensor cores

// fp32 tiles in shared memory: row length d padded to a multiple of 4 plus 4, so that rows
// start on 16 bytes and 8 rows one apart fall into different banks.
__host__ __device__ constexpr int tile_ld(int d) { return d + 4; }

// Positions are 32-bit here (the launchers refuse more tokens).
struct KeyList {
  int32_t pos[kKeys];  // token position, -1: no key
  int64_t off[kKeys];  // element offset of the row in the pools, -1: no key
};

// Keys v0 .. v0 + 63 of the selection's token sequence (entry v / P, token v % P); a key
// outside positions [lo, hi) is left out, so whatever stands there (a NaN, say) stays there.
__device__ __forceinline__ void list_keys(const ScoreArgs& s, int h, int64_t v0, int64_t v1, int lo, int hi,
                                          KeyList* kl) {
  const int P = s.a.g.P;
  if (threadIdx.x < kKeys) {
    const int64_t v = v0 + threadIdx.x;
    int32_t pos = -1;
    int64_t off = -1;
    if (v < v1) {
      const int j = (int)(v / P), t = (int)(v % P);
      const int p = s.a.sel[(size_t)h * s.a.max_sel + j];
      const int64_t blk = score_block(s, h, j, p), at = (int64_t)p * P + t;
      if (blk >= 0 && at >= lo && at < hi) {
        pos = (int32_t)at;
        off = (blk * P + t) * s.a.g.d;
      }
    }
    kl->pos[threadIdx.x] = pos;
    kl->off[threadIdx.x] = off;
  }
}

// Four elements as fp32 (d is a multiple of 4, rows start on 16 bytes or, bf16, on 8).
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// K and V rows of the listed keys as fp32; absent keys are zero.
template <typename T>
__device__ __forceinline__ void load_keys(const ScoreArgs& s, const KeyList* kl, float* sk, float* sv) {
  const int d4 = s.a.g.d / 4, ld = tile_ld(s.a.g.d);
  const T* k = reinterpret_cast<const T*>(s.a.kv.k);
  const T* v = reinterpret_cast<const T*>(s.a.kv.v);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int idx = threadIdx.x; idx < kKeys * d4; idx += kThreads) {
    const int r = idx / d4, e = 4 * (idx % d4);
    const int64_t off = kl->off[r];
    *reinterpret_cast<float4*>(sk + r * ld + e) = off >= 0 ? load4(k + off + e) : zero;
    *reinterpret_cast<float4*>(sv + r * ld + e) = off >= 0 ? load4(v + off + e) : zero;
  }
}

// Rows i0 .. i0 + 63 of head hq of a token-major tensor as fp32; rows past n_q are zero.
template <typename T>
__device__ __forceinline__ void load_rows(const ScoreArgs& s, const void* src, int i0, int hq, float* dst) {
  const int d = s.a.g.d, d4 = d / 4, ld = tile_ld(d);
  const T* x = reinterpret_cast<const T*>(src);
#pragma unroll 4
  for (int idx = threadIdx.x; idx < kRows * d4; idx += kThreads) {
    const int r = idx / d4, e = 4 * (idx % d4), i = i0 + r;
    *reinterpret_cast<float4*>(dst + r * ld + e) =
        i < s.a.n_q ? load4(x + ((size_t)i * s.a.g.Hq + hq) * d + e) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// acc[r][c] = A[ty + 16 r] . B[tx + 16 c] over d columns (d is a multiple of 4).  Even and odd
// columns are summed apart, two products an instruction: half the instructions to issue.
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int d, int ty, int tx, float (&acc)[4][4]) {
  const int ld = tile_ld(d);
  uint64_t sum[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[r][c] = 0;
  for (int e = 0; e < d; e += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const ulonglong2*>(A + (ty + 16 * r) * ld + e);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * c) * ld + e);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[r][c] = fma2(x[r].y, y[c].y, fma2(x[r].x, y[c].x, sum[r][c]));
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float even, odd;
      f32x2_split(sum[r][c], even, odd);
      acc[r][c] = even + odd;
    }
}

// acc[r][c] (columns 4 tx + 64 c) += sum_j W[ty + 16 r][j] X[j], j over 64 rows of X; two columns an
// instruction.  C: groups of 64 columns a row has (1 for d <= 64, else 2).
template <int C>
__device__ __forceinline__ void weigh_rows(const float* W, const float* X, int d, int ty, int tx,
                                           ulonglong2 (&acc)[4][C]) {
  const int ld = tile_ld(d);
  for (int j = 0; j < 64; j += 4) {
    float4 w[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const float4*>(W + (ty + 16 * r) * kLdP + j);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * tx + 64 * c;
      if (col >= d) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(X + (j + u) * ld + col);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = u == 0 ? w[r].x : u == 1 ? w[r].y : u == 2 ? w[r].z : w[r].w;
          const uint64_t pp = f32x2(p, p);
          acc[r][c].x = fma2(pp, x.x, acc[r][c].x);
          acc[r][c].y = fma2(pp, x.y, acc[r][c].y);
        }
      }
    }
  }
}
__device__ __forceinline__ float4 unpaired(const ulonglong2& v) {
  float4 f;
  f32x2_split(v.x, f.x, f.y);
  f32x2_split(v.y, f.z, f.w);
  return f;
}

// Scores in units of log2 (s2 = s log2 e), formed from the raw dot product.
struct ScoreForm {
  float k;       // capped: scale / cap, else scale log2 e
  float cap2;    // cap log2 e; 0: not capped
  float slope2;  // slope log2 e
};
__device__ __forceinline__ ScoreForm score_form(const ScoreArgs& s, int hq) {
  return {s.cap > 0.f ? s.a.scale / s.cap : s.a.scale * kLog2e, s.cap * kLog2e, s.slopes ? s.slopes[hq] * kLog2e : 0.f};
}
// tanh: to |x| = 0.6 a polynomial in x^2 fitted for the least largest relative error of tanh(x) / x
// on [0, 0.6] (a linear program over points of the interval forms it again); with its coefficients
// rounded to fp32 it is off by 4.9e-9, evaluated in fp32 by 7.2e-8.  From there 1 - 2 / (1 + e^2x).
// Both are formed: the lanes of a warp differ.
__device__ __forceinline__ float score_tanh(float x) {
  const float z = x * x;
  float p = fmaf(-0.00585216861f, z, 0.0207536292f);
  p = fmaf(p, z, -0.0537687049f);
  p = fmaf(p, z, 0.13331689f);
  p = fmaf(p, z, -0.333332833f);
  const float far = fmaf(-2.f, rcp_approx(1.f + ex2_approx(2.f * kLog2e * x)), 1.f);
  return fabsf(x) <= 0.6f ? fmaf(x * z, p, x) : far;
}
// The modified score, and in *t the tanh (0 uncapped).
__device__ __forceinline__ float modify(float dot, const ScoreForm& f, int dist, float* t) {
  float x = dot * f.k;
  *t = 0.f;
  if (f.cap2 > 0.f) {
    *t = score_tanh(x);
    x = f.cap2 * *t;
  }
  if (f.slope2 != 0.f) x = fmaf(-f.slope2, (float)abs(dist), x);
  return x;
}

// Ranges of the tile's rows in shared memory and the union [lo, hi) of the non-empty ones.
struct RowSpans {
  int32_t b[kRows], e[kRows];
  int32_t lo, hi;
};
__device__ __forceinline__ void load_spans(const ScoreArgs& s, int i0, RowSpans* rs) {
  if (threadIdx.x < kRows) {
    int64_t b = 0, e = 0;
    if (i0 + (int)threadIdx.x < s.a.n_q) row_span(s, i0 + threadIdx.x, b, e);
    rs->b[threadIdx.x] = (int32_t)b;
    rs->e[threadIdx.x] = (int32_t)e;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int32_t lo = INT_MAX, hi = 0;
    for (int r = threadIdx.x; r < kRows; r += 32)
      if (rs->e[r] > rs->b[r]) {
        lo = min(lo, rs->b[r]);
        hi = max(hi, rs->e[r]);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (threadIdx.x == 0) {
      rs->lo = hi > 0 ? lo : 0;
      rs->hi = hi;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ forward
size_t fwd_smem(int d) { return (size_t)(3 * kKeys * tile_ld(d) + kRows * kLdP) * 4; }

template <typename T, int C>
__global__ void __launch_bounds__(kThreads, 2) score_fwd_simt(const __grid_constant__ ScoreArgs s) {
  const int d = s.a.g.d, P = s.a.g.P, ld = tile_ld(d);
  const int hq = blockIdx.y, h = hq / s.a.g.G, i0 = blockIdx.x * kRows;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  extern __shared__ __align__(16) float dyn[];
  float* sq = dyn;
  float* sk = sq + kRows * ld;
  float* sv = sk + kKeys * ld;
  float* sp = sv + kKeys * ld;
  __shared__ KeyList kl;
  __shared__ RowSpans rs;
  if (blockIdx.x == 0 && blockIdx.z == 0 && hq % s.a.g.G == 0) check_selection(s, h, threadIdx.x, kThreads);
  const int count = sel_count_checked(s.a, h);
  load_spans(s, i0, &rs);
  load_rows<T>(s, s.a.q, i0, hq, sq);
  // entries the tile can see, and this block's share of their tokens (whole key tiles)
  const int j0 = first_entry(s.a, h, count, rs.lo / P);
  const int j1 = rs.hi > rs.lo ? first_entry(s.a, h, count, (rs.hi + P - 1) / P) : j0;
  const int64_t n_tiles = ((int64_t)(j1 - j0) * P + kKeys - 1) / kKeys;
  const int64_t t0 = n_tiles * blockIdx.z / s.n_split, t1 = n_tiles * (blockIdx.z + 1) / s.n_split;
  const int64_t v_end = (int64_t)j1 * P;
  const ScoreForm form = score_form(s, hq);

  float m[4], l[4];  // m in units of log2
  ulonglong2 o[4][C];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[r][c] = make_ulonglong2(0, 0);
  }
  for (int64_t t = t0; t < t1; ++t) {
    __syncthreads();
    list_keys(s, h, (int64_t)j0 * P + t * kKeys, v_end, rs.lo, rs.hi, &kl);
    __syncthreads();
    load_keys<T>(s, &kl, sk, sv);
    __syncthreads();
    float x[4][4];
    dot_tile(sq, sk, d, ty, tx, x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = ty + 16 * r;
      const int b = rs.b[row], e = rs.e[row], qpos = (int)s.a.q_start + i0 + row;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int kpos = kl.pos[tx + 16 * c];
        float th;
        const bool see = kpos >= b && kpos < e;  // an absent key has position -1
        const float v = modify(x[r][c], form, qpos - kpos, &th);
        x[r][c] = see ? v : -INFINITY;
        mx = fmaxf(mx, x[r][c]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m[r], mx);
      const float shift = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2_approx(m[r] - shift);  // 0 while the row has seen nothing
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = ex2_approx(x[r][c] - shift);
        sp[row * kLdP + tx + 16 * c] = p;
        sum += p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[r] = l[r] * alpha + sum;
      m[r] = m_new;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        o[r][c].x = mul2(o[r][c].x, f32x2(alpha, alpha));
        o[r][c].y = mul2(o[r][c].y, f32x2(alpha, alpha));
      }
    }
    __syncthreads();
    weigh_rows(sp, sv, d, ty, tx, o);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + ty + 16 * r;
    if (i >= s.a.n_q) continue;
    const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
    const float lse = l[r] > 0.f ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
    const size_t rh = (size_t)i * s.a.g.Hq + hq;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * tx + 64 * c;
      if (col >= d) continue;
      const float4 w = unpaired(o[r][c]);
      const float v[4] = {w.x * inv, w.y * inv, w.z * inv, w.w * inv};
      if (s.n_split > 1) {
        float* dst = s.part_o + ((size_t)blockIdx.z * s.a.n_q * s.a.g.Hq + rh) * d + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = v[e];
      } else {
        T* dst = reinterpret_cast<T*>(s.a.o_out) + rh * d + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = from_float<T>(v[e]);
      }
    }
    if (tx == 0) {
      if (s.n_split > 1)
        s.part_lse[(size_t)blockIdx.z * s.a.n_q * s.a.g.Hq + rh] = lse;
      else
        s.a.lse_out[(size_t)hq * s.a.n_q + i] = lse;
    }
  }
}

// A block per (row, head): O = sum_z w_z O_z / sum_z w_z with w_z = exp(LSE_z - max LSE).  The
// weights are formed first, so that the reads of all parts are in flight at once; 8 warps take
// the parts z = w, w + 8, ... and are joined in order.
template <typename T>
__global__ void __launch_bounds__(256) score_join(const __grid_constant__ ScoreArgs s) {
  __shared__ float weight[kMaxParts], acc_s[8][kMaxD], max_s[8];
  const int64_t rh = blockIdx.x, rows = (int64_t)s.a.n_q * s.a.g.Hq;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, Hq = s.a.g.Hq, d = s.a.g.d;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: the parts are written from here on
  float m = -INFINITY;
  for (int z = threadIdx.x; z < s.n_split; z += 256) {
    weight[z] = s.part_lse[z * rows + rh];
    m = fmaxf(m, weight[z]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) max_s[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, max_s[w]);
  const float shift = m == -INFINITY ? 0.f : m;
  float acc[kMaxD / 32] = {};
#pragma unroll 8
  for (int z = warp; z < s.n_split; z += 8) {
    const float lz = weight[z], wz = expf(lz - shift);
    const float* src = s.part_o + (z * rows + rh) * d;
#pragma unroll
    for (int c = 0; c < kMaxD / 32; ++c) {
      const float x = lane + 32 * c < d ? src[lane + 32 * c] : 0.f;
      acc[c] += lz > -INFINITY ? wz * x : 0.f;  // a part without keys has written no O
    }
  }
#pragma unroll
  for (int c = 0; c < kMaxD / 32; ++c) acc_s[warp][lane + 32 * c] = acc[c];
  __syncthreads();
  if (threadIdx.x >= d) return;
  float o = 0.f, den = 0.f;
  for (int z = 0; z < s.n_split; ++z) den += expf(weight[z] - shift);
#pragma unroll
  for (int w = 0; w < 8; ++w) o += acc_s[w][threadIdx.x];
  reinterpret_cast<T*>(s.a.o_out)[rh * d + threadIdx.x] = from_float<T>(den > 0.f ? o / den : 0.f);
  if (threadIdx.x == 0) s.a.lse_out[(size_t)(rh % Hq) * s.a.n_q + rh / Hq] = den > 0.f ? m + logf(den) : m;
}

// The same for few parts and, usually, many rows: a warp per (row, head), lane z holding part z's
// log-sum-exp, four columns a lane (512 rows of 28 heads in 2 parts: the whole forward 35.6 us
// against 50.7 with a block a row; of 16 heads in 3 32.4 against 40.1, of 8 in 4 26.1 against 30.1).
constexpr int kFewParts = 16;
template <typename T>
__global__ void __launch_bounds__(256) score_join_few(const __grid_constant__ ScoreArgs s) {
  const int64_t rows = (int64_t)s.a.n_q * s.a.g.Hq, rh = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, Hq = s.a.g.Hq, d = s.a.g.d;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: the parts are written from here on
  if (rh >= rows) return;
  const float lz = lane < s.n_split ? s.part_lse[lane * rows + rh] : -INFINITY;
  float m = lz;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float weight = lz > -INFINITY ? expf(lz - m) : 0.f;
  float den = weight;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int z = 0; z < kFewParts; ++z) {
    const float wz = __shfl_sync(0xffffffffu, weight, z);
    const bool any = __shfl_sync(0xffffffffu, lz, z) > -INFINITY;  // a part without keys has written no O
    if (any && 4 * lane < d) {
      const float4 x = *reinterpret_cast<const float4*>(s.part_o + (z * rows + rh) * d + 4 * lane);
      acc.x += wz * x.x;
      acc.y += wz * x.y;
      acc.z += wz * x.z;
      acc.w += wz * x.w;
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  if (4 * lane < d) {
    T* dst = reinterpret_cast<T*>(s.a.o_out) + rh * d + 4 * lane;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    } else {
      *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
  }
  if (lane == 0) s.a.lse_out[(size_t)(rh % Hq) * s.a.n_q + rh / Hq] = den > 0.f ? m + logf(den) : m;
}

// ----------------------------------------------------------------- backward
template <typename T>
__global__ void __launch_bounds__(256) score_dot(const ScoreArgs s, float* __restrict__ Dbuf) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x % 32, Hq = s.a.g.Hq, d = s.a.g.d;
  if (w >= (int64_t)s.a.n_q * Hq) return;
  const T* o = reinterpret_cast<const T*>(s.a.o) + w * d;
  const T* dout = reinterpret_cast<const T*>(s.a.dout) + w * d;
  float acc = 0.f;
  for (int e = lane; e < d; e += 32) acc += to_float<T>(o[e]) * to_float<T>(dout[e]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (lane == 0) Dbuf[(size_t)(w % Hq) * s.a.n_q + w / Hq] = acc;
}

// P and dA of a thread's 4 x 4 block into shared memory, laid out [row][key] or, for the
// dK/dV kernel, [key][row].
template <bool KEY_MAJOR>
__device__ __forceinline__ void probs_tile(const ScoreArgs& s, const float (&x)[4][4], const float (&dp)[4][4],
                                           const RowSpans* rs, const KeyList* kl, const float* slse2, const float* sD,
                                           const ScoreForm& form, int i0, int ty, int tx, float* sp, float* sda) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = ty + 16 * r;
    const int b = rs->b[row], e = rs->e[row], qpos = (int)s.a.q_start + i0 + row;
    const float lse2 = slse2[row], D = sD[row];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int key = tx + 16 * c, kpos = kl->pos[key];
      const bool see = kpos >= b && kpos < e;
      float t, p = ex2_approx(modify(x[r][c], form, qpos - kpos, &t) - lse2);
      float da = p * (dp[r][c] - D) * fmaf(-t, t, 1.f);
      p = see ? p : 0.f;
      da = see ? da : 0.f;
      const int at = KEY_MAJOR ? key * kLdP + row : row * kLdP + key;
      if (sp) sp[at] = p;
      sda[at] = da;
    }
  }
}

// LSE in units of log2, infinite for rows without keys.
__device__ __forceinline__ void load_stats(const ScoreArgs& s, const float* Dbuf, int i0, int hq, float* slse2,
                                           float* sD) {
  if (threadIdx.x < kRows) {
    const int i = i0 + threadIdx.x;
    const float lse = i < s.a.n_q ? s.a.lse_in[(size_t)hq * s.a.n_q + i] : -INFINITY;
    slse2[threadIdx.x] = lse > -INFINITY ? lse * kLog2e : INFINITY;
    sD[threadIdx.x] = i < s.a.n_q ? Dbuf[(size_t)hq * s.a.n_q + i] : 0.f;
  }
}

size_t dq_smem(int d) { return (size_t)(4 * kKeys * tile_ld(d) + kRows * kLdP) * 4; }
size_t dkdv_smem(int d) { return (size_t)(4 * kKeys * tile_ld(d) + 2 * kRows * kLdP) * 4; }

// list_keys for the keys that a block writes: an entry out of order may name a page that another
// block owns and is left out.
__device__ __forceinline__ void list_owned_keys(const ScoreArgs& s, int h, int64_t v0, int64_t v1, int count,
                                                KeyList* kl) {
  list_keys(s, h, v0, v1, 0, (int)s.total, kl);
  if (threadIdx.x < kKeys && kl->pos[threadIdx.x] >= 0) {
    const int j = (int)((v0 + threadIdx.x) / s.a.g.P);
    const int32_t* row = s.a.sel + (size_t)h * s.a.max_sel;
    if ((j > 0 && row[j - 1] >= row[j]) || (j + 1 < count && row[j + 1] <= row[j]))
      kl->pos[threadIdx.x] = kl->off[threadIdx.x] = -1;
  }
}

// n_split > 1: dQ (unscaled) of the block's share of the keys goes to part[share], [n_q Hq, d].
template <typename T, int C>
__global__ void __launch_bounds__(kThreads, C == 1 ? 2 : 1)
    score_dq_simt(const __grid_constant__ ScoreArgs s, const float* __restrict__ Dbuf, float* __restrict__ part,
                  int n_split) {
  const int d = s.a.g.d, P = s.a.g.P, ld = tile_ld(d);
  const int hq = blockIdx.y, h = hq / s.a.g.G, i0 = blockIdx.x * kRows;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  extern __shared__ __align__(16) float dyn[];
  float* sq = dyn;
  float* sdo = sq + kRows * ld;
  float* sk = sdo + kRows * ld;
  float* sv = sk + kKeys * ld;
  float* sda = sv + kKeys * ld;
  __shared__ KeyList kl;
  __shared__ RowSpans rs;
  __shared__ float slse[kRows], sD[kRows];
  if (blockIdx.x == 0 && hq % s.a.g.G == 0) check_selection(s, h, threadIdx.x, kThreads);
  const int count = sel_count_checked(s.a, h);
  load_spans(s, i0, &rs);
  load_rows<T>(s, s.a.q, i0, hq, sq);
  load_rows<T>(s, s.a.dout, i0, hq, sdo);
  load_stats(s, Dbuf, i0, hq, slse, sD);
  const int j0 = first_entry(s.a, h, count, rs.lo / P);
  const int j1 = rs.hi > rs.lo ? first_entry(s.a, h, count, (rs.hi + P - 1) / P) : j0;
  const int64_t n_tiles = ((int64_t)(j1 - j0) * P + kKeys - 1) / kKeys;
  const int64_t t0 = n_tiles * blockIdx.z / n_split, t1 = n_tiles * (blockIdx.z + 1) / n_split;
  const ScoreForm form = score_form(s, hq);
  ulonglong2 dq[4][C];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) dq[r][c] = make_ulonglong2(0, 0);
  for (int64_t t = t0; t < t1; ++t) {
    __syncthreads();
    list_keys(s, h, (int64_t)j0 * P + t * kKeys, (int64_t)j1 * P, rs.lo, rs.hi, &kl);
    __syncthreads();
    load_keys<T>(s, &kl, sk, sv);
    __syncthreads();
    float x[4][4], dp[4][4];
    dot_tile(sq, sk, d, ty, tx, x);
    dot_tile(sdo, sv, d, ty, tx, dp);
    probs_tile<false>(s, x, dp, &rs, &kl, slse, sD, form, i0, ty, tx, nullptr, sda);
    __syncthreads();
    weigh_rows(sda, sk, d, ty, tx, dq);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + ty + 16 * r;
    if (i >= s.a.n_q) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * tx + 64 * c;
      if (col >= d) continue;
      const size_t at = ((size_t)i * s.a.g.Hq + hq) * d + col;
      const float4 v = unpaired(dq[r][c]);
      if (n_split > 1) {
        *reinterpret_cast<float4*>(part + (size_t)blockIdx.z * s.a.n_q * s.a.g.Hq * d + at) = v;
        continue;
      }
      T* dst = reinterpret_cast<T*>(s.a.dq) + at;
      dst[0] = from_float<T>(v.x * s.a.scale);
      dst[1] = from_float<T>(v.y * s.a.scale);
      dst[2] = from_float<T>(v.z * s.a.scale);
      dst[3] = from_float<T>(v.w * s.a.scale);
    }
  }
}

// n_split > 1: dK (unscaled) and dV of the block's share of the (row tile, query head) pairs go
// to part[share][KV head][key tile], two [64, d] tiles, where the share has seen any row: the
// flag of the share says so.
template <typename T, int C>
__global__ void __launch_bounds__(kThreads, C == 1 ? 2 : 1)
    score_dkdv_simt(const __grid_constant__ ScoreArgs s, const float* __restrict__ Dbuf, float* __restrict__ part,
                    int32_t* __restrict__ flags, int n_split) {
  const int d = s.a.g.d, P = s.a.g.P, G = s.a.g.G, ld = tile_ld(d);
  const int h = blockIdx.y;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  extern __shared__ __align__(16) float dyn[];
  float* sq = dyn;
  float* sdo = sq + kRows * ld;
  float* sk = sdo + kRows * ld;
  float* sv = sk + kKeys * ld;
  float* sp = sv + kKeys * ld;
  float* sda = sp + kRows * kLdP;
  __shared__ KeyList kl;
  __shared__ RowSpans rs;
  __shared__ float slse[kRows], sD[kRows];
  __shared__ int key_lo, key_hi;
  __shared__ int t_first, t_last;
  const int count = sel_count_checked(s.a, h);
  const int64_t v0 = (int64_t)blockIdx.x * kKeys, v1 = (int64_t)count * P;
  if (v0 >= v1) return;
  list_owned_keys(s, h, v0, v1, count, &kl);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int p = kl.pos[threadIdx.x], q = kl.pos[threadIdx.x + 32];
    int lo = min(p < 0 ? INT_MAX : p, q < 0 ? INT_MAX : q), hi = max(p, q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (threadIdx.x == 0) {
      key_lo = lo;
      key_hi = hi;
      t_first = INT_MAX;
      t_last = -1;
    }
  }
  __syncthreads();
  // the row tiles from the first to the last with a row that sees a key of this tile; the shares
  // cut these, so that a key tile few rows see is still spread over many blocks
  const int n_tiles = (s.a.n_q + kRows - 1) / kRows;
  if (key_hi >= 0) {
    if (!s.begin && !s.end) {
      if (threadIdx.x == 0 && key_lo < s.a.q_start + s.a.n_q) {
        t_first = key_lo > s.a.q_start ? (int)((key_lo - s.a.q_start) / kRows) : 0;
        t_last = n_tiles - 1;
      }
    } else {
      int first = INT_MAX, last = -1;
      for (int i = threadIdx.x; i < s.a.n_q; i += kThreads) {
        int64_t b, e;
        row_span(s, i, b, e);
        if (e > b && b <= key_hi && e > key_lo) {
          first = min(first, i / kRows);
          last = i / kRows;
        }
      }
      if (last >= 0) {
        atomicMin(&t_first, first);
        atomicMax(&t_last, last);
      }
    }
  }
  __syncthreads();
  const int n_items = t_last < 0 ? 0 : (t_last - t_first + 1) * G;  // (row tile, query head)
  const int u0 = (int)((int64_t)n_items * blockIdx.z / n_split);
  const int u1 = (int)((int64_t)n_items * (blockIdx.z + 1) / n_split);
  const size_t slot = ((size_t)blockIdx.z * gridDim.y + h) * gridDim.x + blockIdx.x;
  if (u0 == u1) {
    if (n_split > 1 && threadIdx.x == 0) flags[slot] = 0;
    return;
  }
  load_keys<T>(s, &kl, sk, sv);
  bool seen = false;
  ulonglong2 dk[4][C], dv[4][C];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) dk[r][c] = dv[r][c] = make_ulonglong2(0, 0);
  for (int tile = u0 / G; tile * G < u1; ++tile) {
    const int i0 = (t_first + tile) * kRows;
    __syncthreads();
    load_spans(s, i0, &rs);
    if (rs.hi <= key_lo || rs.lo > key_hi) continue;  // no row of the tile sees these keys
    for (int gq = max(0, u0 - tile * G); gq < min(G, u1 - tile * G); ++gq) {
      const int hq = h * G + gq;
      seen = true;
      __syncthreads();
      load_rows<T>(s, s.a.q, i0, hq, sq);
      load_rows<T>(s, s.a.dout, i0, hq, sdo);
      load_stats(s, Dbuf, i0, hq, slse, sD);
      __syncthreads();
      float x[4][4], dp[4][4];
      dot_tile(sq, sk, d, ty, tx, x);
      dot_tile(sdo, sv, d, ty, tx, dp);
      probs_tile<true>(s, x, dp, &rs, &kl, slse, sD, score_form(s, hq), i0, ty, tx, sp, sda);
      __syncthreads();
      weigh_rows(sp, sdo, d, ty, tx, dv);
      weigh_rows(sda, sq, d, ty, tx, dk);
    }
  }
  if (n_split > 1 && threadIdx.x == 0) flags[slot] = seen;
  if (!seen) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int key = ty + 16 * r;
    if (n_split > 1) {
      float* dst = part + slot * 2 * kKeys * d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = 4 * tx + 64 * c;
        if (col >= d) continue;
        *reinterpret_cast<float4*>(dst + key * d + col) = unpaired(dk[r][c]);
        *reinterpret_cast<float4*>(dst + (kKeys + key) * d + col) = unpaired(dv[r][c]);
      }
      continue;
    }
    if (kl.pos[key] < 0) continue;
    const int j = (int)((v0 + key) / P), t = (int)((v0 + key) % P);
    const int phys = s.a.kv.table[s.a.sel[(size_t)h * s.a.max_sel + j]];  // checked by list_keys
    const size_t base = (grad_block(s.a, h, j, phys) * P + t) * d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * tx + 64 * c;
      if (col >= d) continue;
      float4* gk = reinterpret_cast<float4*>(s.a.dk_pool + base + col);
      float4* gv = reinterpret_cast<float4*>(s.a.dv_pool + base + col);
      float4 a = *gk, b = *gv;
      const float4 k4 = unpaired(dk[r][c]), v4 = unpaired(dv[r][c]);
      a.x += s.a.scale * k4.x;
      a.y += s.a.scale * k4.y;
      a.z += s.a.scale * k4.z;
      a.w += s.a.scale * k4.w;
      b.x += v4.x;
      b.y += v4.y;
      b.z += v4.z;
      b.w += v4.w;
      *gk = a;
      *gv = b;
    }
  }
}

// dq = scale * sum of the shares, in order.
template <typename T>
__global__ void __launch_bounds__(256) score_dq_join(const __grid_constant__ ScoreArgs s, const float* __restrict__ part,
                                                     int n_split) {
  const int64_t total = (int64_t)s.a.n_q * s.a.g.Hq * s.a.g.d;
  const int64_t at = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (at >= total) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int z = 0; z < n_split; ++z) {
    const float4 x = *reinterpret_cast<const float4*>(part + z * total + at);
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  T* dst = reinterpret_cast<T*>(s.a.dq) + at;
  dst[0] = from_float<T>(acc.x * s.a.scale);
  dst[1] = from_float<T>(acc.y * s.a.scale);
  dst[2] = from_float<T>(acc.z * s.a.scale);
  dst[3] = from_float<T>(acc.w * s.a.scale);
}

// Ranges leave an unknown part of the key tiles without rows, so dK/dV are cut into this many blocks
// an SM slot: those without rows leave at once, the others still fill the SMs (1024 fp32 rows in
// documents on 4096 tokens: 1 184 us, 2 134, 4 125, 6 120 with more to join).
constexpr int kDkdvFill = 4;
constexpr int kMaxShares = 2048;

// dK += scale * sum of the shares, dV += sum of the shares, for 64 / gridDim.z of a tile's keys.
__global__ void __launch_bounds__(256) score_dkdv_join(const __grid_constant__ ScoreArgs s,
                                                       const float* __restrict__ part,
                                                       const int32_t* __restrict__ flags, int n_split) {
  const int d = s.a.g.d, d4 = d / 4, P = s.a.g.P, h = blockIdx.y;
  __shared__ KeyList kl;
  const int count = sel_count_checked(s.a, h);
  const int64_t v0 = (int64_t)blockIdx.x * kKeys, v1 = (int64_t)count * P;
  if (v0 >= v1) return;
  const size_t tile = 2 * (size_t)kKeys * d, shares = (size_t)gridDim.y * gridDim.x;
  const size_t slot = (size_t)h * gridDim.x + blockIdx.x;
  // the shares that have seen a row, in order: the reads of several are then in flight at once
  __shared__ uint16_t seen[kMaxShares];
  __shared__ int n_seen;
  if (threadIdx.x < 32) {
    int n = 0;
    for (int z0 = 0; z0 < n_split; z0 += 32) {
      const int z = z0 + threadIdx.x;
      const bool f = z < n_split && flags[z * shares + slot] != 0;
      const unsigned mask = __ballot_sync(0xffffffffu, f);
      if (f) seen[n + __popc(mask & ((1u << threadIdx.x) - 1u))] = (uint16_t)z;
      n += __popc(mask);
    }
    if (threadIdx.x == 0) n_seen = n;
  }
  __syncthreads();
  if (n_seen == 0) return;
  list_owned_keys(s, h, v0, v1, count, &kl);
  __syncthreads();
  const int keys = kKeys / gridDim.z, key0 = keys * blockIdx.z;
  for (int idx = threadIdx.x; idx < 2 * keys * d4; idx += blockDim.x) {
    const int r = idx / d4, key = key0 + r % keys, col = 4 * (idx % d4);
    const bool is_k = r < keys;
    if (kl.pos[key] < 0) continue;
    const float* src = part + slot * tile + (size_t)(is_k ? key : kKeys + key) * d + col;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < n_seen; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(src + seen[i] * shares * tile);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const int j = (int)((v0 + key) / P), t = (int)((v0 + key) % P);
    const int phys = s.a.kv.table[s.a.sel[(size_t)h * s.a.max_sel + j]];  // checked by list_owned_keys
    const size_t at = (grad_block(s.a, h, j, phys) * P + t) * d + col;
    const float f = is_k ? s.a.scale : 1.f;
    float4* g = reinterpret_cast<float4*>((is_k ? s.a.dk_pool : s.a.dv_pool) + at);
    float4 y = *g;
    y.x += f * acc.x;
    y.y += f * acc.y;
    y.z += f * acc.z;
    y.w += f * acc.w;
    *g = y;
  }
}

// Row i at position t = q_start + i in document c (doc_start[c] <= t < doc_start[c + 1]):
// keys [doc_start[c], max(t + 1, min(doc_start[c] + prefix_len[c], doc_start[c + 1]))).
__global__ void doc_spans(const int64_t* __restrict__ doc_start, const int64_t* __restrict__ prefix_len, int n_docs,
                          int64_t q_start, int n_q, int64_t* __restrict__ key_begin, int64_t* __restrict__ key_end) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n_q) return;
  const int64_t t = q_start + i;
  int lo = 0, hi = n_docs + 1;  // boundaries <= t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (doc_start[mid] <= t) lo = mid + 1; else hi = mid;
  }
  int64_t b = t, e = t;  // outside every document: nothing is visible
  if (lo >= 1 && lo <= n_docs) {
    const int c = lo - 1;
    b = doc_start[c];
    e = t + 1;
    if (prefix_len) {
      const int64_t last = doc_start[c + 1];
      const int64_t pe = prefix_len[c] > last - b ? last : b + prefix_len[c];
      e = pe > e ? pe : e;
    }
  }
  key_begin[i] = b;
  key_end[i] = e;
}

// Thread blocks that may share one tile's keys: as many as fill the SMs twice when the rows alone do
// not, at most 32 (the join reads every share).  Two blocks fit an SM up to d = 120; of wider heads
// only one does, and the second half of the blocks waits for the first.
int simt_split_limit(const Geometry& g, int n_q) {
  const int64_t tiles = (int64_t)((n_q + kRows - 1) / kRows) * g.Hq;
  return (int)std::min<int64_t>(32, std::max<int64_t>(1, 2 * (int64_t)device_sm_count() / tiles));
}

// Parts the keys of a row may be cut into, and the most rows x parts that any n_q comes to.
int64_t part_rows_limit(const Geometry& g) { return (int64_t)device_sm_count() * (tc_supported(g) ? 512 : 128); }
int parts_limit(const Geometry& g, int n_q) {
  const int64_t most = std::max<int64_t>(1, part_rows_limit(g) / ((int64_t)n_q * g.Hq));
  return (int)std::min<int64_t>(most, tc_supported(g) ? score_tc_parts_limit(g, n_q) : simt_split_limit(g, n_q));
}

template <typename T, int C>
cudaError_t fwd_simt(ScoreArgs& s, cudaStream_t st) {
  static size_t smem_set[kMaxDevices] = {};
  cudaError_t e = set_smem_limit((const void*)score_fwd_simt<T, C>, fwd_smem(64 * C), smem_set);
  if (e != cudaSuccess) return e;
  const int64_t key_tiles = ((int64_t)s.a.max_sel * s.a.g.P + kKeys - 1) / kKeys;
  s.n_split = (int)std::min<int64_t>(parts_limit(s.a.g, s.a.n_q), std::max<int64_t>(1, key_tiles / 2));
  dim3 grid((s.a.n_q + kRows - 1) / kRows, s.a.g.Hq, s.n_split);
  score_fwd_simt<T, C><<<grid, kThreads, fwd_smem(s.a.g.d), st>>>(s);
  count_launches(1);
  return cudaGetLastError();
}

// Backward: shares of a tile, so that the tiles fill the SMs (two blocks fit one for d <= 64).
struct BwdSplit {
  int dq, dkdv;
  size_t dq_bytes, dkdv_bytes;  // of the shares' sums
};
int64_t simt_slots(const Geometry& g) { return (int64_t)device_sm_count() * (g.d <= 64 ? 2 : 1); }
size_t dkdv_tile_bytes(const Geometry& g) { return (size_t)2 * kKeys * g.d * 4; }
BwdSplit simt_bwd_split(const Geometry& g, int n_q, int max_sel) {
  BwdSplit b;
  const int64_t slots = simt_slots(g), row_tiles = (n_q + kRows - 1) / kRows;
  const int64_t key_tiles = ((int64_t)max_sel * g.P + kKeys - 1) / kKeys;
  b.dq = (int)std::min<int64_t>(std::max<int64_t>(1, slots / (row_tiles * g.Hq)), std::max<int64_t>(1, key_tiles / 2));
  const int64_t fill = std::max<int64_t>(1, kDkdvFill * slots / (key_tiles * g.Hkv));
  b.dkdv = (int)std::min<int64_t>({fill, row_tiles * g.G, kMaxShares});
  b.dq_bytes = b.dq > 1 ? align_up((size_t)b.dq * n_q * g.Hq * g.d * 4, 256) : 0;
  b.dkdv_bytes = b.dkdv > 1 ? (size_t)b.dkdv * key_tiles * g.Hkv * dkdv_tile_bytes(g) : 0;
  return b;
}
size_t dkdv_flag_bytes(const Geometry& g) { return align_up((size_t)kDkdvFill * simt_slots(g) * 4, 256); }

template <typename T, int C>
cudaError_t bwd_simt(const ScoreArgs& s, cudaStream_t st) {
  static size_t set_dq[kMaxDevices] = {}, set_dkdv[kMaxDevices] = {};
  cudaError_t e = set_smem_limit((const void*)score_dq_simt<T, C>, dq_smem(64 * C), set_dq);
  if (e == cudaSuccess) e = set_smem_limit((const void*)score_dkdv_simt<T, C>, dkdv_smem(64 * C), set_dkdv);
  if (e != cudaSuccess) return e;
  const Geometry& g = s.a.g;
  const int d = g.d;
  const BwdSplit b = simt_bwd_split(g, s.a.n_q, s.a.max_sel);
  char* ws = reinterpret_cast<char*>(s.a.ws);
  float* Dbuf = reinterpret_cast<float*>(ws);
  int32_t* flags = reinterpret_cast<int32_t*>(ws + align_up((size_t)g.Hq * s.a.n_q * 4, 256));
  float* part_dq = reinterpret_cast<float*>(reinterpret_cast<char*>(flags) + dkdv_flag_bytes(g));
  float* part_kv = reinterpret_cast<float*>(reinterpret_cast<char*>(part_dq) + b.dq_bytes);
  const int64_t warps = (int64_t)s.a.n_q * g.Hq;
  score_dot<T><<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(s, Dbuf);
  dim3 gq((s.a.n_q + kRows - 1) / kRows, g.Hq, b.dq);
  score_dq_simt<T, C><<<gq, kThreads, dq_smem(d), st>>>(s, Dbuf, part_dq, b.dq);
  if (b.dq > 1) score_dq_join<T><<<(unsigned)((warps * d / 4 + 255) / 256), 256, 0, st>>>(s, part_dq, b.dq);
  dim3 gk((unsigned)(((int64_t)s.a.max_sel * g.P + kKeys - 1) / kKeys), g.Hkv, b.dkdv);
  score_dkdv_simt<T, C><<<gk, kThreads, dkdv_smem(d), st>>>(s, Dbuf, part_kv, flags, b.dkdv);
  if (b.dkdv > 1) score_dkdv_join<<<dim3(gk.x, gk.y, 8), 256, 0, st>>>(s, part_kv, flags, b.dkdv);
  count_launches(3 + (b.dq > 1) + (b.dkdv > 1));
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_width(ScoreArgs& s, cudaStream_t st) {
  return s.a.g.d <= 64 ? fwd_simt<T, 1>(s, st) : fwd_simt<T, 2>(s, st);
}
template <typename T>
cudaError_t bwd_width(const ScoreArgs& s, cudaStream_t st) {
  return s.a.g.d <= 64 ? bwd_simt<T, 1>(s, st) : bwd_simt<T, 2>(s, st);
}

}  // namespace

// Forward workspace: the parts' outputs, their log-sum-exps, and the order of the query tiles.
struct FwdSpace {
  size_t o, lse, order;
};
static size_t order_bytes(const Geometry& g, int n_q) {
  return tc_supported(g) ? align_up((size_t)n_q / 64 * 4 + 4, 256) : 0;
}
static FwdSpace fwd_space(const Geometry& g, int n_q) {
  const int n = parts_limit(g, n_q);
  const size_t rows = n > 1 ? (size_t)n_q * g.Hq * n : 0;
  return {align_up(rows * g.d * 4, 256), align_up(rows * 4, 256), order_bytes(g, n_q)};
}
size_t score_fwd_need(const Geometry& g, int n_q) {
  const FwdSpace f = fwd_space(g, n_q);
  return f.o + f.lse + f.order;
}
// Fewer rows are cut into more parts, so what one n_q needs says little about a smaller one.
// The size that is handed out covers every call of up to n_q rows.
size_t score_fwd_workspace_bytes(const Geometry& g, int n_q) {
  const int64_t parts = tc_supported(g) ? score_tc_parts_limit(g, 0) : simt_split_limit(g, 1);
  const size_t rows = (size_t)std::min(part_rows_limit(g), (int64_t)n_q * g.Hq * parts);
  return align_up(rows * g.d * 4, 256) + align_up(rows * 4, 256) + order_bytes(g, n_q);
}

size_t score_bwd_need(const Geometry& g, int n_q, int max_sel) {
  if (tc_supported(g)) return score_bwd_tc_workspace_bytes(g, n_q);
  const BwdSplit b = simt_bwd_split(g, n_q, max_sel);
  return align_up((size_t)g.Hq * n_q * 4, 256) + dkdv_flag_bytes(g) + b.dq_bytes + b.dkdv_bytes;
}
// Covers every call of up to n_q rows: D, and the most that the shares of dQ and dK/dV take.
size_t score_bwd_workspace_bytes(const Geometry& g, int n_q) {
  if (tc_supported(g)) return score_bwd_tc_workspace_bytes(g, n_q);
  const size_t slots = (size_t)simt_slots(g);
  return align_up((size_t)g.Hq * n_q * 4, 256) + dkdv_flag_bytes(g) +
         align_up((size_t)std::min(n_q, kRows) * slots * g.d * 4, 256) + kDkdvFill * slots * dkdv_tile_bytes(g);
}

cudaError_t launch_score_fwd(ScoreArgs& s, cudaStream_t st) {
  const FwdSpace f = fwd_space(s.a.g, s.a.n_q);
  char* ws = reinterpret_cast<char*>(s.a.ws);
  s.part_o = reinterpret_cast<float*>(ws);
  s.part_lse = reinterpret_cast<float*>(ws + f.o);
  s.order = reinterpret_cast<int32_t*>(ws + f.o + f.lse);
  const bool f32 = s.a.g.dtype == OOMB_FP32;
  s.n_split = parts_limit(s.a.g, s.a.n_q);
  cudaError_t e = tc_supported(s.a.g) ? launch_score_fwd_tc(s, st)
                  : f32               ? fwd_width<float>(s, st)
                                      : fwd_width<__nv_bfloat16>(s, st);
  if (e != cudaSuccess || s.n_split <= 1) return e;
  // a dependent launch: its set-up overlaps the end of the forward, whose parts it waits for
  cudaLaunchConfig_t cfg = {};
  const bool few = s.n_split <= kFewParts;
  const unsigned rows = (unsigned)(s.a.n_q * s.a.g.Hq);
  cfg.gridDim = dim3(few ? (rows + 7) / 8 : rows);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (few)
    e = f32 ? cudaLaunchKernelEx(&cfg, score_join_few<float>, s)
            : cudaLaunchKernelEx(&cfg, score_join_few<__nv_bfloat16>, s);
  else
    e = f32 ? cudaLaunchKernelEx(&cfg, score_join<float>, s) : cudaLaunchKernelEx(&cfg, score_join<__nv_bfloat16>, s);
  count_launches(1);
  return e;
}

cudaError_t launch_score_bwd(const ScoreArgs& s, cudaStream_t st) {
  if (tc_supported(s.a.g)) return launch_score_bwd_tc(s, st);
  return s.a.g.dtype == OOMB_FP32 ? bwd_width<float>(s, st) : bwd_width<__nv_bfloat16>(s, st);
}

cudaError_t launch_doc_spans(const int64_t* doc_start, const int64_t* prefix_len, int n_docs, int64_t q_start, int n_q,
                             int64_t* key_begin, int64_t* key_end, cudaStream_t st) {
  doc_spans<<<(unsigned)(((int64_t)n_q + 127) / 128), 128, 0, st>>>(doc_start, prefix_len, n_docs, q_start, n_q, key_begin, key_end);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace oomb
