// Shared pieces of the chunk attention with modified scores (score_simt.cu,
// score_tc_fwd.cu, score_tc_bwd.cu): the arguments, the visible key range of a query
// row, and the range of selection entries a set of rows can see.
//
//   a_ij = scale q_i . k_j
//   s_ij = cap tanh(a_ij / cap)  (cap = 0: a_ij)  -  slope_h |i - j|
//   visible(i, j): begin_i <= j < end_i, j a token of a selected page
//   P = softmax of s over the visible keys, O = P V
// and, with dP = dO V^T and D_i = dO_i . O_i,
//   dA = P (dP - D) (1 - tanh^2(a / cap)),  dQ = scale dA K,  dK += scale dA^T Q,  dV += P^T dO.
#pragma once
#include "attn_common.cuh"

namespace oomb {

struct ScoreArgs {
  AttnArgs a;
  float cap;              // 0: scores are not capped
  const float* slopes;    // [Hq] or nullptr
  const int64_t* begin;   // [n_q] or nullptr (0)
  const int64_t* end;     // [n_q] or nullptr (causal: q_start + i + 1)
  int64_t total;          // tokens appended: no row sees a key at or after it
  int n_view;             // pages a selection may name
  int n_split;            // forward: thread blocks sharing one tile's keys
  float* part_o;          // n_split > 1: [n_split, n_q * Hq, d] partial outputs (normalised)
  float* part_lse;        // n_split > 1: [n_split, n_q * Hq]
  int32_t* order;         // room for the order of the forward's query tiles
};

// Keys [b, e) that query row i may see; e >= b, both within [0, total].
__device__ __forceinline__ void row_span(const ScoreArgs& s, int i, int64_t& b, int64_t& e) {
  b = s.begin ? s.begin[i] : 0;
  e = s.end ? s.end[i] : s.a.q_start + i + 1;
  b = b < 0 ? 0 : b;
  e = e > s.total ? s.total : e;
  if (e <= b) b = e = 0;  // an empty row
}

// First entry of KV head h's selection (ascending, `count` long) at or above page.  On a
// selection that is not ascending the result is some index in [0, count].
__device__ __forceinline__ int first_entry(const AttnArgs& a, int h, int count, int64_t page) {
  const int32_t* row = a.sel + (size_t)h * a.max_sel;
  int lo = 0, hi = count;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (row[mid] < page) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Flags a selection that is not strictly ascending pages of the view (threads tid of
// nthreads each look at a share of the entries).
__device__ __forceinline__ void check_selection(const ScoreArgs& s, int h, int tid, int nthreads) {
  const int count = sel_count_checked(s.a, h);
  const int32_t* row = s.a.sel + (size_t)h * s.a.max_sel;
  for (int e = tid; e < count; e += nthreads) {
    const int p = row[e];
    if (p < 0 || p >= s.n_view || (e > 0 && row[e - 1] >= p)) atomicOr(s.a.err, OOMB_DEVERR_SEL);
  }
}

// Block of K/V holding entry j of head h's selection (logical page p), or -1 when the page
// is outside the view or unmapped (flagged; such a page is left out).
__device__ __forceinline__ int64_t score_block(const ScoreArgs& s, int h, int j, int p) {
  const AttnArgs& a = s.a;
  if (p < 0 || p >= s.n_view || p >= a.g.max_logical) return -1;  // flagged by check_selection
  const int phys = a.kv.table[p];
  if (phys < 0 || phys >= a.g.num_phys) {
    atomicOr(a.err, OOMB_DEVERR_PAGE);
    return -1;
  }
  if (a.kv.staged) return (int64_t)(a.kv.stage_h0 + h) * a.kv.stage_stride + j;
  return (int64_t)phys * a.g.Hkv + h;
}

// ---- launchers ----
bool score_tc_packs(const Geometry& g, int n_q);       // tensor cores: a group's rows fit one tile
int score_tc_parts_limit(const Geometry& g, int n_q);  // most parts the keys of a tile are cut into
cudaError_t launch_score_fwd_tc(ScoreArgs& s, cudaStream_t st);
cudaError_t launch_score_bwd_tc(const ScoreArgs& s, cudaStream_t st);
size_t score_bwd_tc_workspace_bytes(const Geometry& g, int n_q);
size_t score_fwd_need(const Geometry& g, int n_q);  // bytes that this call uses
size_t score_bwd_need(const Geometry& g, int n_q, int max_sel);
size_t score_fwd_workspace_bytes(const Geometry& g, int n_q);  // enough for every call of up to n_q rows
size_t score_bwd_workspace_bytes(const Geometry& g, int n_q);
cudaError_t launch_score_fwd(ScoreArgs& s, cudaStream_t st);
cudaError_t launch_score_bwd(const ScoreArgs& s, cudaStream_t st);
cudaError_t launch_doc_spans(const int64_t* doc_start, const int64_t* prefix_len, int n_docs, int64_t q_start, int n_q,
                             int64_t* key_begin, int64_t* key_end, cudaStream_t st);

}  // namespace oomb
