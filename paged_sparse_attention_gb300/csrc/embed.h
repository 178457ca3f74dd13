// Arguments of the embedding kernels (embed.cu).
#pragma once
#include <cstddef>
#include <cstdint>

namespace oomb {

constexpr int kTileRows = 16;  // sorted rows whose pieces one block sums

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
  int* order;             // [n] rows, by token and then by row
  int* sorted;            // [n] their tokens
  int* sec_order;         // the same, each section by itself
  int* sec_sorted;
  float* part;            // sums of the pieces of long runs
  int64_t pitch;
};

}  // namespace oomb
