// Rotary embedding with positions in several axes (optional bias, rotation, cast), the
// multi-axis sibling of bias_rope.
//
// out[i, h, :] = R(i) (in[i, h, :] + bias[h, :]), R(i) turning each pair (j, j + d/2) by
// positions[axis(j), i] * freq_j.  The angle in turns is position * (freq_j / 2 pi): with the
// factor held as a 96-bit fraction of a turn (turn_ladder.h), the product modulo one turn is the
// angle, whatever the position's size and sign.  Its top 32 bits, known to 2^-31
// turns for every 64-bit position, go to sincospif as a float: 2^-26 turns.  No double-precision
// arithmetic on the device, where it would bound the kernel.
//
// Bytes: the tensor once in and once out.  A block takes a few tokens: their cos/sin (one per
// pair) go to shared memory once and serve every head; a thread moves 16-byte vectors of both
// halves of a head's row.  Shapes or pointers off 16 bytes go element by element (24,576 tokens of
// 28 heads in bf16: 63 us against 154).
//
// Bounds (GB300, 8192 tokens of 28 heads, fp32 in, bf16 out): 176 MB in 32 us, 5.5 TB/s, 81 % of
// the measured copy rate: HBM; the rest is the angles in front of a block's first loads.  Asking
// for the loads before the angles was slower (36.8), and so were streaming stores (35).
#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "turn_ladder.h"

namespace oomb {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;  // head_dim <= 128
constexpr int kMaxAxes = 8;
constexpr int kMaxTokens = 16;  // tokens of a block

struct RopeArgs {
  const void* in;
  const float* bias;
  void* out;
  const int64_t* positions;
  int64_t n;
  int H, half, n_axes, mode, tokens;
  // Of a pair, read as two words: lanes read different pairs, so a word takes as many cycles as
  // there are lanes (8192 tokens of 28 heads: 31.5 us, with three arrays 32.2).
  struct {
    uint64_t turn;        // freq_j / 2 pi as a fraction of 2^64
    uint32_t rest, axis;  // the next 32 bits; its axis
  } pair[kMaxHalf];
};

template <typename T, int E>
__device__ __forceinline__ void load_e(const T* p, float (&f)[E]) {
  if constexpr (E == 1) {
    f[0] = to_float<T>(p[0]);
  } else {
    constexpr int V = E * sizeof(T) >= 16 ? 16 / (int)sizeof(T) : E;  // elements of one access
#pragma unroll
    for (int i = 0; i < E; i += V) {
      __align__(16) T x[V];
      if constexpr (V * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p + i);
      else
        *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(p + i);
#pragma unroll
      for (int e = 0; e < V; ++e) f[i + e] = to_float<T>(x[e]);
    }
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T* p, const float (&f)[E]) {
  if constexpr (E == 1) {
    p[0] = from_float<T>(f[0]);
  } else {
    constexpr int V = E * sizeof(T) >= 16 ? 16 / (int)sizeof(T) : E;
#pragma unroll
    for (int i = 0; i < E; i += V) {
      __align__(16) T x[V];
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = from_float<T>(f[i + e]);
      if constexpr (V * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(p + i) = *reinterpret_cast<const uint4*>(x);
      else
        *reinterpret_cast<uint2*>(p + i) = *reinterpret_cast<const uint2*>(x);
    }
  }
}

// E pairs at a time; half is a multiple of E.
template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(kThreads) rope_axes(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float cs[kMaxTokens * kMaxHalf], sn[kMaxTokens * kMaxHalf];
  const int half = a.half, H = a.H;
  const int64_t i0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)(a.n - i0 < a.tokens ? a.n - i0 : a.tokens);
  if (a.mode != 0) {
    for (int idx = threadIdx.x; idx < nt * half; idx += kThreads) {
      const int t = idx / half, j = idx % half;
      const uint64_t turn = a.pair[j].turn, word = *reinterpret_cast<const uint64_t*>(&a.pair[j].rest);
      const uint64_t rest = (uint32_t)word;
      const int64_t pos = a.positions[(int64_t)(word >> 32) * a.n + i0 + t];
      const uint64_t up = (uint64_t)pos >> 32, down = (uint32_t)pos;
      const uint64_t angle = (uint64_t)pos * turn + up * rest + ((down * rest) >> 32) - (pos < 0 ? rest << 32 : 0);
      const int32_t frac = (int32_t)(angle >> 32);  // the angle in 2^-32 turns, in [-1/2, 1/2)
      float s, c;
      sincospif((float)frac * 0x1p-31f, &s, &c);
      cs[t * half + j] = c;
      sn[t * half + j] = a.mode == 2 ? -s : s;
    }
    __syncthreads();
  }
  const int per_head = half / E, per_token = H * per_head;
  const TI* in = reinterpret_cast<const TI*>(a.in) + (size_t)i0 * H * 2 * half;
  TO* out = reinterpret_cast<TO*>(a.out) + (size_t)i0 * H * 2 * half;
  for (int idx = threadIdx.x; idx < nt * per_token; idx += kThreads) {
    const int t = idx / per_token, r = idx % per_token, h = r / per_head, j = (r % per_head) * E;
    const size_t at = ((size_t)t * H + h) * 2 * half + j;
    float x[E], y[E];
    load_e<TI, E>(in + at, x);
    load_e<TI, E>(in + at + half, y);
    if (a.bias) {
      float b[E], c[E];
      load_e<float, E>(a.bias + (size_t)h * 2 * half + j, b);
      load_e<float, E>(a.bias + (size_t)h * 2 * half + j + half, c);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] += b[e];
        y[e] += c[e];
      }
    }
    if (a.mode != 0) {
      float c[E], s[E];
      load_e<float, E>(cs + t * half + j, c);
      load_e<float, E>(sn + t * half + j, s);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float p = x[e] * c[e] - y[e] * s[e], q = y[e] * c[e] + x[e] * s[e];
        x[e] = p;
        y[e] = q;
      }
    }
    store_e<TO, E>(out + at, x);
    store_e<TO, E>(out + at + half, y);
  }
}

template <typename TI, typename TO>
cudaError_t launch(RopeArgs& a, cudaStream_t st) {
  // 8 pairs a thread where both halves of every row are whole 16-byte vectors of either type
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool wide = a.half % 8 == 0 && on16(a.in) && on16(a.out) && on16(a.bias);
  // tokens a block: enough work for its threads without leaving SMs idle (24,576 tokens of 28 heads:
  // 1 a block 84 us, 2 68, 4 63, 8 63; 1000 tokens 5.0, 4.9, 5.3, 6.2)
  const int64_t per_token = (int64_t)a.H * (wide ? a.half / 8 : a.half);
  int tokens = (int)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, 4 * kThreads / per_token));
  while (tokens > 1 && (a.n + tokens - 1) / tokens < 4 * (int64_t)device_sm_count()) tokens /= 2;
  a.tokens = tokens;
  const unsigned grid = (unsigned)((a.n + tokens - 1) / tokens);
  if (wide)
    rope_axes<TI, TO, 8><<<grid, kThreads, 0, st>>>(a);
  else
    rope_axes<TI, TO, 1><<<grid, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace
}  // namespace oomb

using namespace oomb;

extern "C" oomb_status oomb_bias_rope_axes(const void* in, int in_dtype, const float* bias, void* out, int out_dtype,
                                           int n, int H, int d, const int64_t* positions, int n_axes,
                                           const uint8_t* pair_axis, float theta, int own_ladder, int mode,
                                           void* stream) {
  if (!in || !out || n <= 0 || H <= 0 || d <= 0 || d % 2 || d > 2 * kMaxHalf) return OOMB_ERR_ARG;
  if (mode < 0 || mode > 2 || own_ladder < 0 || own_ladder > 1) return OOMB_ERR_ARG;
  if ((in_dtype != OOMB_BF16 && in_dtype != OOMB_FP32) || (out_dtype != OOMB_BF16 && out_dtype != OOMB_FP32))
    return OOMB_ERR_DTYPE;
  if (in == out && in_dtype != out_dtype) return OOMB_ERR_ARG;
  if ((int64_t)H * d > INT_MAX) return OOMB_ERR_UNSUPPORTED;  // the kernel counts a token's pairs in 32 bits
  RopeArgs a = {};
  const int half = d / 2;
  if (mode != 0) {
    if (!positions || !pair_axis || n_axes <= 0 || n_axes > kMaxAxes) return OOMB_ERR_ARG;
    if (!(theta > 1.0f) || std::isinf(theta)) return OOMB_ERR_ARG;
    int count[kMaxAxes] = {};
    for (int j = 0; j < half; ++j) {
      if (pair_axis[j] >= n_axes) return OOMB_ERR_ARG;
      ++count[pair_axis[j]];
    }
    for (int ax = 0; ax < (own_ladder ? n_axes : 1); ++ax) {  // ladder after ladder
      const int c = own_ladder ? count[ax] : half;
      uint64_t hi[kMaxHalf];
      uint32_t lo[kMaxHalf];
      if (c > 0) turn_ladder((double)theta, c, hi, lo);
      for (int j = 0, r = 0; j < half; ++j) {
        if (own_ladder && pair_axis[j] != ax) continue;
        a.pair[j] = {hi[r], lo[r], pair_axis[j]};
        ++r;
      }
    }
  }
  const uintptr_t ea = dtype_size(in_dtype), eb = dtype_size(out_dtype);
  if (reinterpret_cast<uintptr_t>(in) % ea || reinterpret_cast<uintptr_t>(out) % eb ||
      reinterpret_cast<uintptr_t>(bias) % 4 || reinterpret_cast<uintptr_t>(positions) % 8)
    return OOMB_ERR_ALIGN;
  a.in = in;
  a.bias = bias;
  a.out = out;
  a.positions = positions;
  a.n = n;
  a.H = H;
  a.half = half;
  a.n_axes = n_axes;
  a.mode = mode;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (in_dtype == OOMB_FP32)
    e = out_dtype == OOMB_FP32 ? launch<float, float>(a, st) : launch<float, __nv_bfloat16>(a, st);
  else
    e = out_dtype == OOMB_FP32 ? launch<__nv_bfloat16, float>(a, st) : launch<__nv_bfloat16, __nv_bfloat16>(a, st);
  return cuda_status(e);
}
