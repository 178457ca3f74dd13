// Arguments of the embedding kernels (embed.cu).
#pragma once
#include <cstddef>
#include <cstdint>

#include <vector_types.h>

namespace oomb {

struct EmbedArgs {
  const int64_t* tokens;  // [n]
  const void* table;      // [V, D]
  void* out;              // [n, D]
  const void* d_out;      // [n, D]
  float* d_table;         // [V, D]
  int64_t n;
  int V, D;
  int rows;               // forward: rows of a block
  int accumulate;
  float scale;
  uint32_t* err;
  int key_bits;           // of V, which stands for no token
  int* order;             // [n] rows, by token and then by row
  int* sorted;            // [n] their tokens
  int* sec_order;         // the same, each section by itself
  int* sec_sorted;
  int64_t windows;        // of sorted rows
  int* n_long;            // [2] tokens whose rows lie in several windows, in a few and in many
  int4* long_runs;        // [windows] each: the token, its first and last window; those in many from the end
  float* part;            // sums of their pieces
  int64_t pitch;
};

}  // namespace oomb
