// Pieces, tiles and workspace of the loss over a vocabulary (head_loss.cu): host arithmetic alone, so that what
// the launches write can be held against what the workspace reserves without a GPU.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "../../include/oomb.h"

namespace oomb {
namespace head {

constexpr int kTile = 256, kHalf = 128, kStep = 64;  // tile, a CTA's share of it, columns of K a stage
// Tiles of kNarrow columns instead of kTile where there are few tiles and a cluster's time is its loop over K.
constexpr int kNarrow = 64;

// Workspace given to a piece's dz, and to staged parts of W where it cannot be read in place
// (kStagedOdd: bf16 rows that are on 16 bytes unless the caller's pointer is not).  Both directions with 256, 512
// and 1024 MB for dz: 8192 rows on 131072 x 3584 18882, 18762 and 18773 us, 951 on 32001 x 1000 in fp32 1077, 1081 and
// 1119; 1600 of 4001 on 50001 x 2048 with 256 and 512 MB 932 and 876 us in a run of 20 ms, 992 and 952 in one of a
// second (1024 MB: 6 % above 512).
constexpr size_t kAccBytes = 256u << 20, kDzBytes = 512u << 20, kStagedBytes = 256u << 20, kStagedOdd = 32u << 20;

inline int tiles(int64_t x, int t) { return (int)((x + t - 1) / t); }
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Whether every cluster has one narrow tile of the logits of `rows` and `cols` at most.  (A step of K takes a
// narrow tile 0.30 us and a wide one 0.33, so it does not pay to have more of them.)
inline bool is_narrow(int64_t rows, int64_t cols, int clusters) {
  return (int64_t)tiles(rows, kTile) * tiles(cols, kNarrow) <= clusters;
}
// Most rows that are.
inline int64_t narrow_rows(int64_t cols, int clusters) { return (int64_t)kTile * (clusters / tiles(cols, kNarrow)); }

// Forward: the tiles' width, and how many parts of a row's sum they leave (half a tile's columns each).
struct RowParts {
  bool narrow;
  int parts;
};
inline RowParts row_parts(int64_t rows, int V, int piece, int clusters) {
  const bool narrow = is_narrow(rows, piece, clusters);
  return {narrow, tiles(V, narrow ? kNarrow / 2 : kHalf)};
}

// Parts that K of dx may be cut into: as many as kAccBytes hold, 64 at most.
inline int most_splits(int64_t n, int D) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(64, (int64_t)(kAccBytes / ((size_t)n * up((size_t)D, 4) * 4))));
}
// Parts that the rows of a piece's dw are cut into where it has few tiles: of 8 steps at least.
inline int dw_splits(int64_t n, int D, int cols, int clusters) {
  const int64_t of = (int64_t)tiles(cols, kTile) * tiles(D, kTile);
  return (int)std::max<int64_t>(1, std::min<int64_t>(clusters / of, tiles(n, kStep) / 8));
}

// Where things lie in the workspace, and the pieces of the vocabulary.
struct Plan {
  int parts_of, pitch_d;       // bf16 parts of an operand, elements of a staged row
  bool staged;                 // W is read through the workspace
  int piece;                   // columns of a piece (the last may have fewer)
  int pitch_z;
  size_t count, rows, at, x, w, part, dz, acc, acc_w, bytes;
};
inline Plan make_plan(int64_t n, int D, int V, int dtype, bool backward, bool w_on16, int clusters) {
  Plan p = {};
  p.parts_of = dtype == OOMB_FP32 ? 3 : 1;
  // rows on lines of 128 bytes: a box of 64 columns that straddles two asks for both (951 rows on 32001 x 1000 in
  // fp32: 303 us, 230)
  p.pitch_d = (int)up((size_t)D, 64);
  const bool never_in_place = dtype == OOMB_FP32 || D % 8 != 0;
  p.staged = never_in_place || !w_on16;
  const size_t row_bytes = (size_t)p.parts_of * p.pitch_d * 2;
  const int64_t v256 = (int64_t)up((size_t)V, kTile);
  // the pieces' sizes are multiples of a tile, about equal
  auto piece_of = [&](int64_t most) {
    const int64_t pieces = (V + most - 1) / most;
    return (int)std::min<int64_t>(V, (int64_t)up((size_t)((V + pieces - 1) / pieces), kTile));
  };
  const int64_t staged_rows = std::min<int64_t>(
      v256, std::max<int64_t>(kTile, (int64_t)((never_in_place ? kStagedBytes : kStagedOdd) / row_bytes) / kTile * kTile));
  int64_t most = p.staged ? staged_rows : v256;
  const size_t z_bytes = (size_t)p.parts_of * n * 2;  // of a column of dz
  if (backward) most = std::min<int64_t>(most, std::max<int64_t>(kTile, (int64_t)(kDzBytes / z_bytes) / kTile * kTile));
  p.piece = piece_of(most);
  p.pitch_z = (int)up((size_t)p.piece, 64);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up(bytes, 256);
    return here;
  };
  p.count = take(8);
  p.rows = take((size_t)n * 4);
  p.at = take((size_t)n * 4);
  p.x = take((size_t)n * row_bytes);
  p.w = take((size_t)staged_rows * row_bytes);  // the same for every n
  const size_t common = at;
  // parts of wide tiles, or of narrow ones for as many rows as may have them (most where W is staged: its
  // pieces are the smallest); row_parts counts a single piece by V itself, and so does this
  const int64_t narrow = std::min<int64_t>(n, narrow_rows(piece_of(staged_rows), clusters));
  p.part = take(std::max((size_t)n * tiles(V, kHalf), (size_t)narrow * tiles(V, kNarrow / 2)) * 8);
  const size_t forward_bytes = at;
  at = common;
  // room that grows with n although a piece of more rows has fewer columns
  p.dz = take(std::min<size_t>(z_bytes * up((size_t)V, 64), std::max<size_t>(kDzBytes, z_bytes * kTile)));
  const size_t acc = (size_t)n * up((size_t)D, 4) * 4;
  p.acc = take(std::max(acc, std::min(64 * acc, kAccBytes)));
  p.acc_w = take((size_t)clusters * kTile * kTile * 4);  // a tile a cluster at most
  p.bytes = backward ? std::max(forward_bytes, at) : forward_bytes;
  return p;
}

}  // namespace head
}  // namespace oomb
