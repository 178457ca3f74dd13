// Arguments of the kernels of the loss over a vocabulary (head_loss.cu, head_gemm.cuh).
#pragma once
#include <cuda_bf16.h>

#include <cstddef>
#include <cstdint>

namespace oomb {
namespace head {

// Rows with a target are gathered: row r of a product is row rows[r] of the caller's, r < *count.
struct GemmArgs {
  const int* count;
  const int* rows;
  int n;            // the caller's rows
  int group;        // row tiles whose tiles come one after another
  int tms, tns;     // tiles of rows (kDw) and of columns
  int steps;        // of K (not kDw)
  int splits;       // K is cut in this many parts (kDx)
  int passes;       // 1, or 6 products of parts
  int chunk;        // steps of K that are summed on the tensor cores
  int row_b;        // first row of the piece in W's map
  // the piece of the vocabulary: columns [v0, v0 + cols)
  int v0, cols;
  const int64_t* targets;
  float cap;
  // kLse
  float2* part;     // [n, parts] maximum and sum of 128 columns, base 2
  int parts, part0;
  const float* at;  // [n] logit of the target, which is not in the sums
  // kDz
  const float* lse;
  const float* d_loss;
  __nv_bfloat16* dz;  // [passes == 1 ? 1 : 3, n, pitch]
  int pitch;
  // kDx, kDw
  float* acc;       // kDx: [splits, n, acc_pitch] sums of the pieces
  int acc_pitch, add, last;
  void* out;
  int out_cols, out_fp32, out_vec, accumulate;
  float scale;
  uint32_t* err;
};

}  // namespace head
}  // namespace oomb
