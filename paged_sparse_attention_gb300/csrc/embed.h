// Arguments of the embedding kernels (embed.cu).
#pragma once
#include <cstddef>
#include <cstdint>

#include <vector_types.h>

namespace oomb {

constexpr int kTileRows = 4;  // sorted rows whose pieces one block sums

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
  int section;            // keys ranked against each other
  int* order;             // [n] rows, by token and then by row
  int* sorted;            // [n] their tokens
  int* sec_order;         // the same, each section by itself
  int* sec_sorted;
  int* n_long;            // tokens whose rows lie in several windows
  int2* long_runs;        // each: the token and its last window
  float* part;            // sums of their pieces
  int64_t pitch;
};

}  // namespace oomb
