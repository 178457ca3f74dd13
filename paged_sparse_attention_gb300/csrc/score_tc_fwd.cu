// tcgen05 forward of the attention with modified scores (bf16, head_dim 128, page 128).
//
// Two layouts of a thread block's two 128-row tiles A and B:
//  rows   tiles A and B are neighbouring 128-row tiles of one query head.  Both read the same
//         pages, each K and V tile loaded once.  Heaviest pairs first: the last ones of a causal
//         chunk; where the rows have ranges, in the order that score_fwd_plan finds.
//  packed where all rows of the G heads of a group fit one tile (n_q G <= 128: single tokens
//         and short tails): row r is token r / G, head r % G, so K and V are read once for
//         the whole group, and A and B hold the same rows and take alternate pages.
// Pages that no row of the block can see are left out: the ranges of the rows give an
// interval of the ascending selection.  Where the tiles do not fill the SMs, n_split thread
// blocks share the interval, their parts joined by score_join (packed: A and B of one block
// are two parts).
//
// Packed against rows, 1 row, 28 query heads on 4: 4 pages 9.5 against 12.1 us, 64 pages 13.2
// against 28.6, 1024 pages 52.7 against 327.  score_fwd_plan, where rows have ranges: documents of
// 12000 tokens with prefixes, 8192 rows 555 us with it, 614 without; of 1500, 4001 rows 155 and 204.
//
// Bounds (GB300).  Packed, one token on 131,072 with 28 query heads on 4: 56 us for 268 MB with the
// join, 4.8 TB/s: 18 us of launch, set-up and join, then HBM (twice and four times the tokens take
// 95 and 172 us: 7.0 TB/s of reads).  Rows,
// 4096 rows on 97 pages: cap 50 in 572 us, 1064 TFLOP/s, 54 % of the measured bf16 peak; without a
// modification 498 us, 1221 (the plain forward 531), with a bias 475, with a cap that most scores
// come near 834: there the exponential unit is the bound, with three operations a score; else the
// chain of one tile, S, its softmax, P V, which two tiles overlap but do not hide (cap 50: tensor
// pipe active 51 %, exponential unit 23 %, issue 53 %).
//
// Warp roles (576 threads): warp 0 TMA producer (K ring of 3, V ring of 2 or 3 tiles), warp 1 MMA
// issuer and TMEM owner, warps 2-9 softmax of tile A, 10-17 of tile B.  A query row belongs to
// two threads, 64 scores each: with one thread a row the score arithmetic of one tile takes
// longer than the products of the other, and two warps of a scheduler can share the units
// that one warp alone leaves idle while it waits for its own results.  The two exchange their
// maxima through shared memory and a barrier of their pair of warps.  The tensor core runs
// PV_A(j), S_A(j+1), PV_B(j), S_B(j+1).  MMAs complete in order, so the softmax warp that has
// seen S_X(j) knows that PV_X(j-1) is done and frees the ring slots.
// TMEM columns: S_A, S_B (P over S, bf16), O_A, O_B, 128 each.
// Scores and row sums are fp32; P is rounded to bf16, the operand type of the second product.
#include "score_tc_common.cuh"

namespace oomb {
namespace {

using namespace tc;

constexpr int kKStages = 3;
constexpr int kVStages = 3;  // two used by the rows layout; the packed one has the third where tile B's Q would be
constexpr int kThreads = 576;
constexpr int kTileWarps = 8;  // softmax warps of a tile
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when the row maximum grows by more
constexpr float kNear = 90.0f;             // log2 units: 2^-90 and what is 2^-36 of it are fp32 numbers
constexpr float kNothing = -127.0f;        // log2 units: 2^x is zero in fp32 with flushed denormals

struct ScoreFwdParams {
  ScoreArgs s;
  CapConst cap;
  float scale_log2;
  int n_tiles, n_pairs;
  const int32_t* order;  // rows: pair of tiles of each grid row, or nullptr (last pair first)
};

struct __align__(8) FwdBarriers {
  uint64_t q_full;
  uint64_t k_full[kKStages];
  uint64_t k_empty[kKStages];
  uint64_t v_full[kVStages];
  uint64_t v_empty[kVStages];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_done[2];
  uint64_t mma_done;
  float half[2][2][kTile];  // per tile, column half and row: maximum of the scores, at the end the sum of P
  int kv_row[64];           // first row in the K/V maps of ring entry e, at e % 64
  int64_t lo[8], hi[8];     // key range seen by each 32 rows of the tiles
  int below[4];          // selected pages below: tile A's first, A's end, B's first, B's end
  uint32_t tmem_base;
  int abort;
  int fail[2][4];  // page (+ 1) at which a warp of the pair that shares these 32 rows gave up waiting
};

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 2 * kTileBytes;
constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
constexpr uint32_t kOffBar = kOffV + 2 * kTileBytes;
// No alignment slack: there is no static shared memory, and the dynamic window starts on a
// 1 KB boundary (checked at entry; the swizzled tiles need it).
template <bool PACK>
constexpr int v_stages() { return PACK ? 3 : 2; }
__device__ __forceinline__ uint32_t v_offset(int stage) {
  return stage < 2 ? kOffV + (uint32_t)stage * kTileBytes : kOffQ + kTileBytes;
}
constexpr size_t kSmemBytes = kOffBar + sizeof(FwdBarriers);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// The pages of the two tiles, as steps of the walk over the selection (step i is entry i, or
// count - 1 - i in the reversed walk).  rows: tile x reads [first[x], first[x] + n[x]), and the
// ring holds the steps [lo, lo + n_ring) in order.  packed: tile x reads its own n[x] steps
// from first[x], and the ring alternates between the tiles.
struct TilePages {
  int first[2], n[2], lo, n_ring;
};

template <bool PACK>
__device__ __forceinline__ int ring_of(const TilePages& t, int x, int j) {  // ring entry of tile x's page j
  return PACK ? 2 * j + x : t.first[x] - t.lo + j;
}

template <bool PACK, bool REVERSED>
__device__ __forceinline__ TilePages tile_pages(const ScoreFwdParams& p, const int (&below)[4], int count) {
  TilePages t;
  int a0 = below[0], a1 = max(below[0], below[1]), b0 = below[2], b1 = max(below[2], below[3]);
  if (REVERSED) {
    const int u = a0, v = b0;
    a0 = count - a1;
    a1 = count - u;
    b0 = count - b1;
    b1 = count - v;
  }
  if (PACK) {
    // the interval's share of this block, half of it for each tile, A the odd page.  A slot of
    // either ring is waited for only when its last user has a later page of its own, whose S
    // tells it that the slot is free (V: entry e waits for e - 3, whose tile also has e - 1)
    const int n = a1 - a0;
    const int c0 = a0 + (int)((int64_t)n * blockIdx.z / p.s.n_split);
    const int c1 = a0 + (int)((int64_t)n * (blockIdx.z + 1) / p.s.n_split);
    t.first[0] = c0;
    t.n[0] = (c1 - c0 + 1) / 2;
    t.first[1] = c0 + t.n[0];
    t.n[1] = c1 - c0 - t.n[0];
    t.lo = 0;
    t.n_ring = c1 - c0;
    return t;
  }
  // this block's share of the union of the two intervals
  const bool ea = a0 == a1, eb = b0 == b1;
  const int lo = ea ? b0 : eb ? a0 : min(a0, b0), hi = ea ? b1 : eb ? a1 : max(a1, b1);
  const int c0 = lo + (int)((int64_t)(hi - lo) * blockIdx.z / p.s.n_split);
  const int c1 = lo + (int)((int64_t)(hi - lo) * (blockIdx.z + 1) / p.s.n_split);
  a0 = min(max(a0, c0), c1);
  a1 = min(max(a1, c0), c1);
  b0 = min(max(b0, c0), c1);
  b1 = min(max(b1, c0), c1);
  // B ends no earlier than A and no page between them is left out (pages a tile cannot see
  // are masked): the ring's slots are then freed by B where B reads the page, else by A
  if (b0 >= b1) {
    b0 = b1 = a1;
  } else if (a0 >= a1) {
    a0 = a1 = b0;
  } else {
    b1 = max(b1, a1);
    b0 = min(b0, a1);
  }
  t.first[0] = a0;
  t.n[0] = a1 - a0;
  t.first[1] = b0;
  t.n[1] = b1 - b0;
  t.lo = a0 < a1 ? min(a0, b0) : b0;
  t.n_ring = max(a1, b1) - t.lo;
  return t;
}

// Reduction of 64 scores by a three-operand function, in eight chains.
template <typename F>
__device__ __forceinline__ float row_reduce(const uint32_t (&s)[64], F f) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = f(__uint_as_float(s[k]), __uint_as_float(s[8 + k]), __uint_as_float(s[16 + k]));
#pragma unroll
  for (int c = 24; c < 56; c += 16)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f(v[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + 8 + k]));
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = f(v[k], __uint_as_float(s[56 + k]), __uint_as_float(s[56 + k]));
  return f(f(v[0], v[1], v[2]), f(v[3], v[4], v[5]), f(v[6], v[7], v[7]));
}

template <bool CAP, bool BIAS, bool PACK>
__global__ void __launch_bounds__(kThreads, 1)
    score_fwd_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ ScoreFwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  const AttnArgs& a = p.s.a;
  if (smem_u32(smem_raw) & 1023u) {  // uniform over the grid: every block leaves here
    if (threadIdx.x == 0) atomicOr(a.err, OOMB_DEVERR_SMEM);
    return;
  }
  uint8_t* sm = smem_raw;
  FwdBarriers* bar = reinterpret_cast<FwdBarriers*>(sm + kOffBar);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = a.g.G, Hq = a.g.Hq;
  const int h = PACK ? (int)blockIdx.x : (int)blockIdx.x / G;
  const int pair = p.order ? p.order[blockIdx.y] : p.n_pairs - 1 - (int)blockIdx.y;
  // With a bias the pages are walked from the nearest to the farthest: the row maximum then
  // comes first and O is hardly ever rescaled (upwards, a head whose bias changes by more than
  // 2^8 over a page would rescale at every page).  The tile that ends the walk last has to be
  // B: the later rows in the upward walk, the earlier ones (which start below) in the reversed.
  constexpr bool REVERSED = BIAS;
  const int tile[2] = {2 * pair + (REVERSED ? 1 : 0), 2 * pair + (REVERSED ? 0 : 1)};
  const int32_t* sel_row = a.sel + (size_t)h * a.max_sel;
  const int raw_count = a.sel_count[h];
  // this thread's first entry and the one before it, asked for early
  const int tid_entry = min((int)threadIdx.x, a.max_sel - 1);
  const int sel_mine = sel_row[tid_entry], sel_before = sel_row[max(tid_entry - 1, 0)];
  const int count = raw_count < 0 ? 0 : min(raw_count, a.max_sel);  // flagged below
  volatile int* abort = &bar->abort;
  constexpr int kV = v_stages<PACK>();

  // softmax thread: its row and query head
  const int x = warp < 2 ? 0 : (warp - 2) >> 3;      // tile
  const int half = warp < 2 ? 0 : (warp - 2) >> 2 & 1;  // key columns [64 half, 64 half + 64)
  const int r = (warp & 3) * 32 + lane;              // row of the tile == TMEM lane
  int row = 0, hq = 0;
  bool valid = false;
  int64_t kb = 0, ke = INT64_MAX;  // range common to the warp's rows (rows that do not exist ask for no masking)
  if (warp >= 2) {
    if (PACK) {
      valid = r < a.n_q * G;
      row = valid ? r / G : 0;
      hq = h * G + (valid ? r % G : 0);
    } else {
      row = tile[x] * kTile + r;
      valid = row < a.n_q;
      hq = (int)blockIdx.x;
    }
    int64_t lo = INT64_MAX, hi = 0;
    if (!p.s.begin && !p.s.end) {  // causal: the warp's first and last row tell
      const int first = (warp & 3) * 32, rows = PACK ? a.n_q * G : min(kTile, a.n_q - tile[x] * kTile);
      if (first < rows) {
        const int last = min(first + 31, rows - 1), t0 = PACK ? 0 : tile[x] * kTile;
        lo = 0;
        hi = a.q_start + t0 + (PACK ? last / G : last) + 1;
        ke = a.q_start + t0 + (PACK ? first / G : first) + 1;
      }
    } else {
      if (valid) row_span(p.s, row, kb, ke);
      if (valid && ke > kb) {
        lo = kb;
        hi = ke;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        kb = max(kb, __shfl_xor_sync(0xffffffffu, kb, o));
        ke = min(ke, __shfl_xor_sync(0xffffffffu, ke, o));
      }
    }
    if (lane == 0 && half == 0) {
      bar->lo[4 * x + (warp & 3)] = lo;
      bar->hi[4 * x + (warp & 3)] = hi;
    }
    if (PACK) {  // rows of Q that no load fills
      const int used = a.n_q * G;
      for (int idx = (int)threadIdx.x - 64; idx < (kTile - used) * 16; idx += kThreads - 64) {
        const int rr = used + idx / 16, c = idx % 16;
        *reinterpret_cast<uint4*>(sm + kOffQ + (c >> 3) * kHalfBytes + rr * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], kTileWarps);
      mbar_init(&bar->o_done[i], 1);
    }
    mbar_init(&bar->mma_done, 1);
    bar->abort = 0;
    for (int i = 0; i < 4; ++i) bar->below[i] = bar->fail[0][i] = bar->fail[1][i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  if (threadIdx.x == 0) {  // Q needs none of what follows
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    if (PACK) {
      const uint32_t bytes = (uint32_t)(a.n_q * G) * 128u;
      mbar_arrive_expect_tx(&bar->q_full, 2 * bytes);
      tma_load_3d(sm + kOffQ, &tq, &bar->q_full, 0, h * G, 0);
      tma_load_3d(sm + kOffQ + kHalfBytes, &tq, &bar->q_full, 64, h * G, 0);
    } else {
      // a tile past the last one has no pages and is not loaded
      mbar_arrive_expect_tx(&bar->q_full, (2 * pair + 1 < p.n_tiles ? 2u : 1u) * kTileBytes);
      for (int i = 0; i < 2; ++i) {
        if (tile[i] >= p.n_tiles) continue;
        uint8_t* dst = sm + kOffQ + i * kTileBytes;
        tma_load_3d(dst, &tq, &bar->q_full, 0, (int)blockIdx.x, tile[i] * kTile);
        tma_load_3d(dst + kHalfBytes, &tq, &bar->q_full, 64, (int)blockIdx.x, tile[i] * kTile);
      }
    }
  }
  {
    // entries below the first page a tile sees and below the end of the last one, counted by
    // all threads (the selection ascends); the selection is checked in the same pass
    int64_t page[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      int64_t lo = INT64_MAX, hi = 0;
      for (int w = 4 * t; w < 4 * t + 4; ++w) {
        lo = min(lo, bar->lo[w]);
        hi = max(hi, bar->hi[w]);
      }
      page[2 * t] = hi > 0 ? lo / kTile : 0;
      page[2 * t + 1] = (hi + kTile - 1) / kTile;
    }
    int n[4] = {0, 0, 0, 0};
    bool bad = false;
    for (int e = threadIdx.x; e < count; e += kThreads) {
      const int pg = e < kThreads ? sel_mine : sel_row[e];
      const int before = e < kThreads ? sel_before : sel_row[e - 1];
      bad |= pg < 0 || pg >= p.s.n_view || (e > 0 && before >= pg);
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] += pg < page[i] ? 1 : 0;
    }
    if (bad || (threadIdx.x == 0 && count != raw_count)) atomicOr(a.err, OOMB_DEVERR_SEL);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int sum = __reduce_add_sync(0xffffffffu, n[i]);
      if (lane == 0 && sum) atomicAdd(&bar->below[i], sum);
    }
  }
  __syncthreads();
  const int below[4] = {bar->below[0], bar->below[1], bar->below[2], bar->below[3]};
  const TilePages t = tile_pages<PACK, REVERSED>(p, below, count);
  auto entry = [&](int step) { return REVERSED ? count - 1 - step : step; };  // of the selection

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // The lanes look up 32 ring entries at a time (page, physical page: two loads that wait for
    // one another); lane 0 waits for free slots and issues the copies.
    int jk = 0, jv = 0;
    bool up = true;
    for (int base = 0; up && base < t.n_ring; base += 32) {
      const int e = base + lane;
      if (e < t.n_ring) {
        const int j = entry(PACK ? t.first[e & 1] + (e >> 1) : t.lo + e);
        const int64_t blk = score_block(p.s, h, j, sel_row[j]);
        // a page left out is masked whole and, read from below the pools' first row, all zero
        bar->kv_row[e % 64] = blk < 0 ? -kTile : (int)(blk * kTile);
      }
      __syncwarp();
      if (lane == 0) {
        const int to = min(base + 32, t.n_ring);  // V is at most a few entries behind K
        long long last = clock64();
        while (jk < to || (to == t.n_ring && jv < to)) {
          bool progressed = false;
          if (jk < to) {
            const int ks = jk % kKStages;
            if (jk < kKStages || mbar_test_wait(&bar->k_empty[ks], ((jk / kKStages) - 1) & 1)) {
              const int rw = bar->kv_row[jk % 64];
              mbar_arrive_expect_tx(&bar->k_full[ks], kTileBytes);
              tma_load_2d(sm + kOffK + ks * kTileBytes, &tk, &bar->k_full[ks], 0, rw);
              tma_load_2d(sm + kOffK + ks * kTileBytes + kHalfBytes, &tk, &bar->k_full[ks], 64, rw);
              ++jk;
              progressed = true;
            }
          }
          if (jv < jk) {
            const int vs = jv % kV;
            if (jv < kV || mbar_test_wait(&bar->v_empty[vs], ((jv / kV) - 1) & 1)) {
              const int rw = bar->kv_row[jv % 64];
              mbar_arrive_expect_tx(&bar->v_full[vs], kTileBytes);
              tma_load_2d(sm + v_offset(vs), &tv, &bar->v_full[vs], 0, rw);
              tma_load_2d(sm + v_offset(vs) + kHalfBytes, &tv, &bar->v_full[vs], 64, rw);
              ++jv;
              progressed = true;
            }
          }
          if (progressed) {
            last = clock64();
          } else if (*abort) {
            up = false;
            break;
          } else if (clock64() - last > (1ll << 31)) {
            atomicOr(a.err, kErrMbarTimeout);
            *abort = 1;
            up = false;
            break;
          }
        }
      }
      up = __shfl_sync(0xffffffffu, up, 0);
    }
    if (lane == 0) {
      // drain: every armed stage must have landed before the block may exit
      for (int jj = (jk > kKStages ? jk - kKStages : 0); jj < jk; ++jj)
        mbar_wait(&bar->k_full[jj % kKStages], (jj / kKStages) & 1, a.err, nullptr);
      for (int jj = (jv > kV ? jv - kV : 0); jj < jv; ++jj)
        mbar_wait(&bar->v_full[jj % kV], (jj / kV) & 1, a.err, nullptr);
      mbar_wait(&bar->q_full, 0, a.err, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && t.n_ring > 0) {
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(128, 128, false, true);
      bool ok = mbar_wait(&bar->q_full, 0, a.err, abort);
      auto issue_s = [&](int xx, int j) -> bool {  // S = Q K_j^T
        const int e = ring_of<PACK>(t, xx, j);
        if (!mbar_wait(&bar->k_full[e % kKStages], (e / kKStages) & 1, a.err, abort)) return false;
        tc_fence_after();
        const uint32_t aQ = smem_u32(sm + kOffQ + (PACK ? 0 : xx * kTileBytes));
        const uint32_t aK = smem_u32(sm + kOffK + (e % kKStages) * kTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem + xx * 128, desc_kmajor(aQ, kk), desc_kmajor(aK, kk), idesc_s, kk > 0);
        mma_commit(&bar->s_full[xx]);
        return true;
      };
      auto issue_pv = [&](int xx, int j) -> bool {  // O += P V_j
        const int e = ring_of<PACK>(t, xx, j);
        if (!mbar_wait(&bar->v_full[e % kV], (e / kV) & 1, a.err, abort)) return false;
        if (!mbar_wait(&bar->p_full[xx], j & 1, a.err, abort)) return false;
        tc_fence_after();
        const uint32_t aV = smem_u32(sm + v_offset(e % kV));
        const uint32_t ap = tmem + xx * 128, o = tmem + 256 + xx * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(o, ap + kk * 8, desc_mnmajor(aV, kk), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        if (j == t.n[xx] - 1) mma_commit(&bar->o_done[xx]);
        return true;
      };
      // step i: rows, ring entry i; packed, page i of each tile
      const int steps = PACK ? max(t.n[0], t.n[1]) : t.n_ring;
      int off[2];  // page of tile x at step i is i - off[x]
#pragma unroll
      for (int xx = 0; xx < 2; ++xx) off[xx] = PACK ? 0 : t.first[xx] - t.lo;
      for (int xx = 0; ok && xx < 2; ++xx)
        if (t.n[xx] > 0 && off[xx] == 0) ok = issue_s(xx, 0);
      for (int i = 0; ok && i < steps; ++i)
        for (int xx = 0; ok && xx < 2; ++xx) {
          const int j = i - off[xx];
          if (j >= 0 && j < t.n[xx]) ok = issue_pv(xx, j);
          if (ok && j + 1 >= 0 && j + 1 < t.n[xx]) ok = issue_s(xx, j + 1);
        }
      // every issued MMA must finish before TMEM is released
      mma_commit(&bar->mma_done);
      mbar_wait(&bar->mma_done, 0, a.err, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int nx = t.n[x];
    const uint32_t lane_off = tmem_lane_base(warp);
    const uint32_t tS = tmem + lane_off + x * 128;
    const uint32_t tO = tmem + lane_off + 256 + x * 128 + half * 64;  // this thread's columns of O
    const int pair_bar = 1 + 4 * x + (warp & 3);  // barrier of the two warps that share the rows
    volatile float* mine = &bar->half[x][half][r];
    volatile float* other = &bar->half[x][half ^ 1][r];
    volatile int* fail = &bar->fail[x][warp & 3];
    const int64_t qpos = a.q_start + row;
    const float slope2 = BIAS ? p.s.slopes[hq] * kLog2e : 0.f;
    const int32_t* sel = sel_row + entry(t.first[x]);
    constexpr int kNext = REVERSED ? -1 : 1;
    const int b_first = t.first[1] - t.lo, b_end = b_first + t.n[1];  // rows: ring entries of tile B
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int pg = nx > 0 ? sel[0] : 0;
    for (int j = 0; j < nx; ++j) {
      const bool known = pg >= 0 && pg < p.s.n_view && pg < a.g.max_logical;
      const int phys = known ? a.kv.table[pg] : -1;
      const int64_t p0 = (int64_t)pg * kTile + half * 64;  // this thread's first key
      const bool mapped = phys >= 0 && phys < a.g.num_phys;  // a page left out has no visible key
      const bool whole = mapped && kb <= p0 && ke >= p0 + 64;  // the same for the whole warp
      const int pg_next = j + 1 < nx ? sel[kNext * (j + 1)] : 0;
      if (ok) ok = mbar_wait(&bar->s_full[x], j & 1, a.err, abort);
      ok = __all_sync(0xffffffffu, ok);  // TMEM loads and stores below are warp-collective
      if (!ok) {  // meet the other warp of the pair at its barrier, so that both leave here
        if (lane == 0) *fail = j + 1;
        named_bar_sync(pair_bar, 64);
        break;
      }
      tc_fence_after();
      if (((warp - 2) & 7) == 0 && lane == 0) {
        const int e = ring_of<PACK>(t, x, j);
        if (PACK) {  // each ring entry has one user
          mbar_arrive(&bar->k_empty[e % kKStages]);
          if (j > 0) mbar_arrive(&bar->v_empty[ring_of<PACK>(t, x, j - 1) % kV]);
        } else if (x == 1 || e < b_first || e >= b_end) {  // the last user of page e
          mbar_arrive(&bar->k_empty[e % kKStages]);
          if (e > 0) mbar_arrive(&bar->v_empty[(e - 1) % kV]);
        }
      }
      uint32_t sr[64];
      tmem_ld32(tS + half * 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tmem_ld32(tS + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tmem_wait_ld();
      // ref: no less than the largest score of this half row, from one pass over the raw dot
      // products.  `direct` (every key visible, a bias linear over the page): the scores are
      // formed inside the exponent, P = 2^(score - m).  That needs an m within about 2^90 of the
      // row's largest score, so that no P that counts is lost: either ref is that near (kNear),
      // or it does not raise the m of the pages before.  `nothing`: every P is zero in fp32.
      // Elsewhere the scores are formed in place, in log2 units, and ref is their maximum.
      const float f0 = BIAS ? (float)(qpos - p0) : 0.f;  // distance of key column c: |f0 - c|
      const float b0 = -slope2 * f0;
      const bool behind = BIAS && __all_sync(0xffffffffu, f0 >= 64.f);  // every key behind its row: linear in c
      TanhForm form = kWide;
      float ref, spread = 0.f;  // spread: how far ref may be above the largest score
      if constexpr (CAP) {
        const float amax = row_reduce(sr, [](float u, float v, float w) { return fmax3_abs(u, v, w); });
        form = __all_sync(0xffffffffu, amax <= p.cap.edge2)   ? kDegree2
               : __all_sync(0xffffffffu, amax <= p.cap.edge3) ? kDegree3
                                                              : kWide;
        ref = fminf(fabsf(p.scale_log2) * amax, p.cap.cap2);  // |cap tanh(x)| <= |cap x|, cap
        spread = 2.f * ref;
      } else {
        const float top = row_reduce(sr, [](float u, float v, float w) { return fmax3(u, v, w); });
        ref = p.scale_log2 >= 0.f ? p.scale_log2 * top : INFINITY;
      }
      if constexpr (BIAS) {
        ref += fmaxf(b0, fmaf(slope2, 63.f, b0));
        spread = fmaf(fabsf(slope2), (float)kTile, spread);
      }
      const bool direct = whole && (!BIAS || behind) && (CAP || p.scale_log2 >= 0.f) &&
                          __all_sync(0xffffffffu, spread <= kNear || ref <= m + kRescaleThreshold);
      const bool nothing = behind && __all_sync(0xffffffffu, ref - m < kNothing);
      if (!direct && !nothing) {
        if constexpr (CAP) {
          if (form != kWide) {  // (the wide form is off by 2^-23 of the cap, too much under a large one)
#pragma unroll
            for (int c = 0; c < 64; ++c)
              sr[c] = __float_as_uint(p.cap.cap2 * tanh_of<kDegree3>(__uint_as_float(sr[c]), p.cap));
          } else {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              sr[c] = __float_as_uint(p.cap.cap2 * tanh_of<kWide>(__uint_as_float(sr[c]), p.cap));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) sr[c] = __float_as_uint(p.scale_log2 * __uint_as_float(sr[c]));
        }
        if constexpr (BIAS) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            sr[c] = __float_as_uint(fmaf(-slope2, fabsf(f0 - (float)c), __uint_as_float(sr[c])));
        }
        if (!whole) {
          int64_t rb = p0, re = p0 + 64;  // the row's own range, read again: few pages are cut by it
          if (valid) row_span(p.s, row, rb, re);
          rb -= p0;
          re -= p0;
          const int cb = mapped ? (int)max((int64_t)0, min(rb, (int64_t)64)) : 64;
          const int ce = mapped ? (int)max((int64_t)0, min(re, (int64_t)64)) : 0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < cb || c >= ce) sr[c] = 0xff800000u;  // -inf
        }
        ref = row_reduce(sr, [](float u, float v, float w) { return fmax3(u, v, w); });
      }
      // the row's maximum over both halves.  One buffer is enough: no warp sees the next S
      // before every warp of the tile has handed in its P of this page
      *mine = ref;
      named_bar_sync(pair_bar, 64);
      if (*fail == j + 1) {  // (a later page's failure is met at that page's barrier)
        ok = false;
        break;
      }
      ref = fmaxf(ref, *other);
      bool rescale_o = false;
      float alpha = 1.f;
      if (ref > m + kRescaleThreshold || (m == -INFINITY && ref > -INFINITY)) {
        const float m_new = fmaxf(m, ref);
        alpha = exp2f(m - m_new);  // 0 when m == -inf
        rescale_o = (j > 0) && (m > -INFINITY);
        l *= alpha;
        m = m_new;
      }
      const float neg_m = (m == -INFINITY) ? 0.f : -m;
      if (!(BIAS && nothing)) {
        // P = 2^(score - m) of column pairs: arg(pair) is the exponent
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        auto exponentials = [&](auto arg) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float t0, t1;
            arg(c, t0, t1);
            const float p0v = ex2_approx(t0), p1v = ex2_approx(t1);
            sum[c & 3] += p0v + p1v;
            sr[c] = pack_bf16x2(p0v, p1v);
          }
        };
        const uint64_t negm2 = f32x2(neg_m, neg_m);
        auto pair_of = [&](int c) { return f32x2(sr[2 * c], sr[2 * c + 1]); };
        // what the exponent adds to a score: -m, and in the direct case the bias
        const float b0m = b0 + neg_m;
        auto shift = [&](int c) {
          return BIAS ? f32x2(fmaf(slope2, (float)(2 * c), b0m), fmaf(slope2, (float)(2 * c + 1), b0m)) : negm2;
        };
        if (!direct) {
          exponentials([&](int c, float& t0, float& t1) { f32x2_split(fadd2(pair_of(c), negm2), t0, t1); });
        } else if constexpr (!CAP) {
          const uint64_t sc2 = f32x2(p.scale_log2, p.scale_log2);
          exponentials([&](int c, float& t0, float& t1) { f32x2_split(ffma2(pair_of(c), sc2, shift(c)), t0, t1); });
        } else if (form == kDegree2) {
          const float* q = p.cap.poly2;
          const float k2 = p.cap.cap2;
          const uint64_t q0 = f32x2(q[0] * k2, q[0] * k2), q1 = f32x2(q[1] * k2, q[1] * k2), q2 = f32x2(q[2] * k2, q[2] * k2);
          exponentials([&](int c, float& t0, float& t1) {
            const uint64_t S = pair_of(c), z = fmul2(S, S);
            f32x2_split(ffma2(S, ffma2(ffma2(q2, z, q1), z, q0), shift(c)), t0, t1);
          });
        } else if (form == kDegree3) {
          const float* q = p.cap.poly3;
          const float k2 = p.cap.cap2;
          const uint64_t q0 = f32x2(q[0] * k2, q[0] * k2), q1 = f32x2(q[1] * k2, q[1] * k2),
                         q2 = f32x2(q[2] * k2, q[2] * k2), q3 = f32x2(q[3] * k2, q[3] * k2);
          exponentials([&](int c, float& t0, float& t1) {
            const uint64_t S = pair_of(c), z = fmul2(S, S);
            f32x2_split(ffma2(S, ffma2(ffma2(ffma2(q3, z, q2), z, q1), z, q0), shift(c)), t0, t1);
          });
        } else {  // cap2 tanh(x) = cap2 - 2 cap2 / (1 + e^2x)
          const uint64_t k2 = f32x2(p.cap.cap2, p.cap.cap2), one = f32x2(1.f, 1.f);
          const uint64_t arg2 = f32x2(p.cap.arg, p.cap.arg), m2k = f32x2(-2.f * p.cap.cap2, -2.f * p.cap.cap2);
          exponentials([&](int c, float& t0, float& t1) {
            float e0, e1;
            f32x2_split(fmul2(pair_of(c), arg2), e0, e1);
            f32x2_split(fadd2(f32x2(ex2_approx(e0), ex2_approx(e1)), one), e0, e1);
            f32x2_split(ffma2(f32x2(rcp_approx(e0), rcp_approx(e1)), m2k, fadd2(shift(c), k2)), t0, t1);
          });
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // The rescale is decided per row but the TMEM accesses are warp-collective: the warp
      // rescales when any of its rows needs it, the other rows scale by alpha = 1 (exact).
      if (__any_sync(0xffffffffu, rescale_o)) {  // PV of the previous page finished before this S
        if (!rescale_o) alpha = 1.f;
#pragma unroll 1
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + cc * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int ee = 0; ee < 32; ++ee) o[ee] = __float_as_uint(__uint_as_float(o[ee]) * alpha);
          tmem_st32(tO + cc * 32, o);
        }
      }
      if (BIAS && nothing) {
        uint32_t zero[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) zero[c] = 0u;
        tmem_st32(tS + half * 32, zero);
      } else {
        // packed key columns 2c, 2c + 1 of this half -> column 32 half + c (both halves of S are
        // in registers since the pair's barrier)
        tmem_st32(tS + half * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->p_full[x]);
      pg = pg_next;
    }
    // epilogue: this thread's half row of O, normalised by the sum over both halves
    const size_t rows = (size_t)a.n_q * Hq, rh = (size_t)row * Hq + hq;
    const int part = PACK ? 2 * (int)blockIdx.z + x : (int)blockIdx.z;
    const bool split = PACK || p.s.n_split > 1;
    bool done = __all_sync(0xffffffffu, ok && nx > 0 && mbar_wait(&bar->o_done[x], 0, a.err, abort));
    if (nx > 0) {  // (done: the last PV has run, so every warp of the tile is past its last exchange)
      if (done)
        *mine = l;
      else if (lane == 0)
        *fail = nx + 1;
      named_bar_sync(pair_bar, 64);
      done = done && !*fail;
      if (done) l += *other;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float lse = done ? (m + log2f(l)) * kLn2 : -INFINITY;
    if (done && split) {
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + cc * 32, o);
        tmem_wait_ld();
        if (!valid) continue;
        float4* dst = reinterpret_cast<float4*>(p.s.part_o + ((size_t)part * rows + rh) * kD + half * 64 + cc * 32);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                               __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
      }
    } else if (done) {
      // through shared memory (the tile's Q, read by the last S, is free), so that a warp writes
      // whole 256-byte rows: 16-byte chunk c of row r stands at c ^ (r & 15)
      tc_fence_after();
      uint8_t* stage = sm + kOffQ + x * kTileBytes;
#pragma unroll 1
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + cc * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint4 w;
          w.x = pack_bf16x2(__uint_as_float(o[8 * v + 0]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
          w.y = pack_bf16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
          w.z = pack_bf16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
          w.w = pack_bf16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
          const int c = half * 8 + cc * 4 + v;
          *reinterpret_cast<uint4*>(stage + r * 256 + ((c ^ (r & 15)) * 16)) = w;
        }
      }
      named_bar_sync(pair_bar, 64);
      const int c = lane & 15, row0 = tile[x] * kTile;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // this warp: 16 of the pair's 32 rows, two at a time
        const int rr = (warp & 3) * 32 + half * 16 + 2 * i + (lane >> 4);
        if (row0 + rr < a.n_q)
          *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o_out) + ((size_t)(row0 + rr) * Hq + hq) * kD +
                                    c * 8) =
              *reinterpret_cast<const uint4*>(stage + rr * 256 + ((c ^ (rr & 15)) * 16));
      }
    } else if (!split && valid) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o_out) + rh * kD + half * 64);
      for (int v = 0; v < 8; ++v) dst[v] = make_uint4(0, 0, 0, 0);
    }
    if (valid && half == 0) {
      if (split)
        p.s.part_lse[(size_t)part * rows + rh] = lse;  // -inf: score_join does not read the part's O
      else
        a.lse_out[(size_t)hq * a.n_q + row] = lse;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Pairs of tiles by the pages that their rows' ranges span, most first (ties: the later pair).
// One block; the pairs are few.
constexpr int kMaxPlan = 256;
__global__ void __launch_bounds__(1024) score_fwd_plan(const __grid_constant__ ScoreArgs s, int n_pairs,
                                                       int32_t* __restrict__ order) {
  __shared__ unsigned long long lo[kMaxPlan], hi[kMaxPlan];
  __shared__ int pages[kMaxPlan];
  const int lane = threadIdx.x % 32;
  for (int i = threadIdx.x; i < n_pairs; i += 1024) {
    lo[i] = ~0ull;
    hi[i] = 0;
  }
  __syncthreads();
  for (int i0 = (int)threadIdx.x - lane; i0 < s.a.n_q; i0 += 1024) {  // 32 rows of one pair a warp
    int64_t b = 0, e = 0;
    if (i0 + lane < s.a.n_q) row_span(s, i0 + lane, b, e);
    if (e <= b) b = INT64_MAX;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b = min(b, __shfl_xor_sync(0xffffffffu, b, o));
      e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
    }
    if (lane == 0 && e > 0) {
      atomicMin(&lo[i0 / (2 * kTile)], (unsigned long long)b);
      atomicMax(&hi[i0 / (2 * kTile)], (unsigned long long)e);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_pairs; i += 1024)
    pages[i] = hi[i] ? (int)((hi[i] + kTile - 1) / kTile - lo[i] / kTile) : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n_pairs; i += 1024) {
    int rank = 0;
    for (int k = 0; k < n_pairs; ++k) rank += pages[k] > pages[i] || (pages[k] == pages[i] && k > i);
    order[rank] = i;
  }
}

// 3-D map over a token-major [n, H, 128] bf16 tensor: box = every token, G heads, 64 columns.
bool make_tmap_group(CUtensorMap* m, const void* base, int n, int H, int G) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)H, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)H * kD * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)n};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool CAP, bool BIAS, bool PACK>
cudaError_t launch_one(const ScoreFwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       cudaStream_t st) {
  static size_t smem_set[kMaxDevices] = {};
  cudaError_t e = set_smem_limit((const void*)score_fwd_tc<CAP, BIAS, PACK>, kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(PACK ? p.s.a.g.Hkv : p.s.a.g.Hq, p.n_pairs, p.s.n_split);
  score_fwd_tc<CAP, BIAS, PACK><<<grid, kThreads, kSmemBytes, st>>>(tq, tk, tv, p);
  count_launches(1);
  return cudaGetLastError();
}

template <bool CAP, bool BIAS>
cudaError_t launch_pack(bool pack, const ScoreFwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t st) {
  return pack ? launch_one<CAP, BIAS, true>(p, tq, tk, tv, st) : launch_one<CAP, BIAS, false>(p, tq, tk, tv, st);
}

}  // namespace

bool score_tc_packs(const Geometry& g, int n_q) { return (int64_t)n_q * g.G <= kTile; }

// Parts the keys of a tile may be cut into (n_q = 0: for any number of rows).
int score_tc_parts_limit(const Geometry& g, int n_q) {
  const int sms = std::min(device_sm_count(), 512);  // score_join takes up to 1024 parts
  const int packed = 2 * std::max(1, sms / g.Hkv);
  const int64_t units = (int64_t)((std::max(n_q, 1) + 2 * kTile - 1) / (2 * kTile)) * g.Hq;
  const int rows = (int)std::min<int64_t>(1024, std::max<int64_t>(1, 4 * (int64_t)sms / units));
  if (n_q == 0) return std::max(packed, rows);
  return score_tc_packs(g, n_q) ? packed : rows;
}

cudaError_t launch_score_fwd_tc(ScoreArgs& s, cudaStream_t st) {
  const Geometry& g = s.a.g;
  const int limit = s.n_split, sms = device_sm_count();  // parts that the workspace has room for
  const bool pack = score_tc_packs(g, s.a.n_q) && limit >= 2;
  ScoreFwdParams p;
  p.n_tiles = (s.a.n_q + kTile - 1) / kTile;
  p.n_pairs = pack ? 1 : (p.n_tiles + 1) / 2;
  if (pack) {
    // one block per SM, as long as each has a page for either tile (two where the parts are of many
    // rows); up to 16 pages a block each: one of its tiles then idles, but the shorter walk counts
    // for more.  28 query heads on 4, 1 row and 18: 4 pages 9.5 and 13.1 us in 4 blocks, 10.1 and 15.7
    // in 2; 16 pages 10.9 and 14.8 in 16, 10.9 and 16.7 in 8; 64 pages 13.2 and 19.8 in 32, 13.9 and
    // 20.1 in 16 (from a cold L2 25.6 and 24.4 for 17 rows).  16 heads on 2 and 8 on 8, 1 row and 8 on
    // 4 to 1024 pages: within 4 % of the best cut
    const int pages = s.a.max_sel, each = (int64_t)s.a.n_q * g.Hq > 256 ? 4 : 2;
    s.n_split = std::min(limit / 2, std::max((pages + each - 1) / each, std::min(pages, 16)));
  } else {
    // Waves of blocks, each as long as its pages and about four more for set-up and epilogue; once
    // the keys are cut, the join takes as long as two pages and one more for every 8000 rows of
    // parts (28 query heads: 200 rows on 16 pages 25.1 us in 4 parts, 39.4 in one; 300 rows on 8
    // pages 27.6 in 2, 25.0 in one).  Made for many heads: of 16 on 2 and 8 on 8 it cuts too little and
    // loses up to a quarter (300 rows on 8 pages, 8 on 8: 23.8 us in 3 parts, 18.9 in 8).
    const int64_t units = (int64_t)p.n_pairs * g.Hq;
    double best = 0.0;
    for (int n = 1; n <= limit && (n == 1 || s.a.max_sel / n >= 2); ++n) {
      const double join = n > 1 ? 2.0 + (double)s.a.n_q * g.Hq * n / 8000.0 : 0.0;
      const double t = (double)((units * n + sms - 1) / sms) * ((double)s.a.max_sel / n + 4.0) + join;
      if (n == 1 || t < 0.95 * best) {
        best = t;
        s.n_split = n;
      }
    }
  }
  CUtensorMap tq, tk, tv;
  const bool ok = pack ? make_tmap_group(&tq, s.a.q, s.a.n_q, g.Hq, g.G) : make_tmap_heads(&tq, s.a.q, s.a.n_q, g.Hq);
  if (!ok || !make_tmap_rows(&tk, s.a.kv.k, kv_rows(s.a)) || !make_tmap_rows(&tv, s.a.kv.v, kv_rows(s.a)))
    return cudaErrorInvalidValue;
  p.s = s;
  p.cap = make_cap(s.cap, s.a.scale);
  p.scale_log2 = s.a.scale * kLog2e;
  p.order = nullptr;
  cudaError_t e;
  // With ranges the pairs' work is not known here; worth a launch where the blocks queue for SMs.
  if (!pack && (s.begin || s.end) && p.n_pairs <= kMaxPlan && (int64_t)p.n_pairs * g.Hq * s.n_split > sms) {
    score_fwd_plan<<<1, 1024, 0, st>>>(s, p.n_pairs, s.order);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.order = s.order;
  }
  if (s.cap > 0.f)
    e = s.slopes ? launch_pack<true, true>(pack, p, tq, tk, tv, st) : launch_pack<true, false>(pack, p, tq, tk, tv, st);
  else
    e = s.slopes ? launch_pack<false, true>(pack, p, tq, tk, tv, st)
                 : launch_pack<false, false>(pack, p, tq, tk, tv, st);
  s.n_split = pack ? 2 * s.n_split : s.n_split;  // parts for the join
  return e;
}

}  // namespace oomb
