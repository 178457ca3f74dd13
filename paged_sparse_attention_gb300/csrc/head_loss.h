// Arguments of the kernels of the loss over a vocabulary (head_loss.cu, head_gemm.cuh).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

namespace oomb {
namespace head {

// Rows with a target are gathered: row r of a product is row rows[r] of the caller's, r < *count.
struct GemmArgs {
  const int* count; // rows with a target; behind it the parts that K of dx is cut into
  const int* rows;
  int n;            // the caller's rows
  int group;        // row tiles whose tiles come one after another
  int tms, tns;     // tiles of rows (kDw) and of columns
  int steps;        // of K (not kDw)
  int passes;       // 1, or 6 products of parts
  int chunk;        // steps of K that are summed on the tensor cores
  int row_b;        // first row of the piece in W's map
  // the piece of the vocabulary: columns [v0, v0 + cols)
  int v0, cols;
  const int64_t* targets;
  float cap;
  // kLse
  float2* part;     // [n, parts] maximum and sum of half a tile's columns, base 2
  int parts, part0;
  const float* at;  // [n] logit of the target, which is not in the sums
  // kDz
  const float* lse;
  const float* d_loss;
  __nv_bfloat16* dz;  // [passes == 1 ? 1 : 3, n, pitch]
  int pitch;
  // kDx, kDw
  float* acc;       // kDx: [splits, n, acc_pitch] sums of the pieces; kDw: [dw_splits, cols, acc_pitch]
  int acc_pitch, add, last, dw_splits;
  void* out;
  int out_cols, out_fp32, out_vec, accumulate;
  float scale;
  uint32_t* err;
};

// ---- few rows and small problems (head_small.cu)
// What goes there, by the operands' type: fp32 costs the tensor cores six products, these cores one.
// Both sides measured, forward and backward, us on CUDA cores / tensor cores, n of V x D:
//   bf16:  12 of 10000 x 1000: 81 / 63   32 of 2000 x 1000: 70 / 48   64 of 1000 x 256: 35 / 41
//          48 of 1000 x 500: 55 / 49     32 of 8000 x 64: 67 / 41
//   fp32:  16 of 30000 x 4096: 1110 / 1572   24 of the same: 1599 / 1592   24 of 10000 x 1000: 179 / 180
//          64 of 1000 x 1000: 76 / 116   128 of 1000 x 500: 150 / 90   32 of 8000 x 64: 78 / 71
constexpr int kFewRows = 8, kFewRows32 = 16;  // rows that always take it (bf16, fp32)
constexpr int64_t kSmallWork = 1 << 24, kSmallWork32 = 1 << 26;  // products n V D up to which more rows do
constexpr int kSmallWidth = 256;              // a logit costs as much as of this many columns at least
constexpr int kMaxRows = 64;                  // and how many more

struct SmallArgs {
  const void* x;
  const void* w;
  const int64_t* targets;
  int n, D, V;
  float cap, scale;
  uint32_t* err;
  float* loss;         // forward
  float* lse;
  float2* part;        // [n, parts]
  int parts;
  float* at;           // [n] logit of the target
  const float* lse_in; // backward
  const float* d_loss;
  float* dz;           // [n, pitch]
  int pitch;
  float* acc;          // [units, n, acc_pitch] parts of dx
  int acc_pitch;
  void* dx;
  void* dw;
  int accumulate, dw_vec;
  int ct, row_groups;
};
struct SmallSpace {
  size_t at, part, dz, acc;
  int parts, pitch, acc_pitch;
};
// Rows up to which a problem goes this way (0: none do).
int small_rows(int D, int V, int dtype);
// Bytes of workspace, and what lies where.
size_t small_space(int n, int D, int V, bool backward, SmallSpace* s);
cudaError_t launch_small_fwd(const SmallArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_small_bwd(const SmallArgs& a, int dtype, int dw_dtype, cudaStream_t st);

#ifdef __CUDACC__
// Loss and log-sum-exp of a row from its target's logit z and the sum s 2^m of the other exponentials.
// A sure row's loss is small and keeps its own precision; a target's logit of +infinity makes it no number (inf - inf).
__device__ __forceinline__ void loss_of(float z, float m, float s, float& loss, float& lse) {
  const float rest = (m + log2f(s)) * 0.6931471805599453f;
  if (z >= rest) {
    loss = z < INFINITY ? log1pf(s * exp2f(m - z * 1.4426950408889634f)) : z - z;
    lse = z + loss;
  } else {
    const float more = log1pf(expf(z - rest));
    loss = (rest - z) + more;
    lse = rest + more;
  }
}
#endif

}  // namespace head
}  // namespace oomb
