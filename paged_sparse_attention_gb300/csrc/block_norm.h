// Arguments of the block-norm kernels (block_norm.cu).
#pragma once
#include <cstddef>
#include <cstdint>

namespace oomb {

struct NormArgs {
  const void* x;       // [n, D] residual stream
  const void* y;       // [n, D] block output, or nullptr
  const float* w_post; // [D] or nullptr
  const void* gate;    // [D] fp32, or [n, D] of the tensors' type (gate_rows), or nullptr
  int gate_rows;
  const float* w_pre;  // [D] or nullptr
  float res_scale, eps, inv_D;
  int64_t n;
  int D;
  void* x_out;         // forward
  void* u;
  float* rstd_post;    // [n]
  float* rstd_pre;     // [n]
  const void* du;      // backward
  const void* dx_in;   // gradient at x_out, or nullptr (zero)
  void* dx;
  void* dy;
  float* dw_post;
  float* dw_pre;
  void* dgate;
  int accumulate;
  float* part;         // [2, norm_parts, D]
};

int norm_blocks_per_sm(int T);
// Thread blocks of the backward, each with its own partial weight gradients.
int norm_parts(int64_t n, int D);

}  // namespace oomb
