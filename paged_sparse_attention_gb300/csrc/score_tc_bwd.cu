// tcgen05 backward of the attention with modified scores (bf16, head_dim 128, page 128).
//
// The layout of the plain backward: one cluster of n_split thread blocks per (selected page,
// KV head), K and V of the page stationary in shared memory, the page's steps (query tile x
// query head of the group) cut into n_split ranges and walked in two 64-row halves,
//   S^T = K Q^T    dP^T = V dO^T    dV += P^T dO    dK += dA^T Q    dQ^T = K^T dA^T,
// dQ added to an fp32 accumulator, dK/dV summed over the cluster in rank order through
// distributed shared memory and added once into the pool rows (no atomics on the pool).
// What differs:
//   score_bwd_prep  also writes every row's key range and, per 128-row tile, the union of its
//                   rows' ranges and the range common to all of them
//   score_bwd_tc    finds the first and the last tile whose rows can see the page and walks
//                   only those; a page that no row sees leaves at once.  The softmax warps
//                   form P = 2^(s2 - LSE log2 e) from the capped and biased score and
//                   dA = P (dP - D) (1 - tanh^2); only a tile whose common range does not
//                   cover the page looks at the rows' ranges.
// P and dA are rounded to bf16, the operand type of the products that read them; sums are fp32.
//
// Bounds (GB300).  8192 rows on 193 pages, 28 query heads on 4, cap 50: 7.13 ms, 849 TFLOP/s, 43 % of
// the measured bf16 peak, by TMEM and shared-memory traffic as the plain backward (915 there, and
// 910 here without the cap); a step of 128 rows costs 3.6 us a thread block, 3.9 with the cap.
// Documents of 1500 tokens, 4001 rows: 320 us of this kernel, 369 of the call (score_bwd_prep 24,
// score_bwd_convert 16), 4.9 us a step: 40 % of the steps are cut by a range, and blocks of 25 steps
// pay for their set-up and for the sum over the cluster (tensor pipe active 46 %).
//
// Warp roles of score_bwd_tc (448 threads): warp 0 TMA producer, warp 1 MMA issuer and TMEM
// owner, warps 2-9 softmax (thread = key row, 32 of a half's 64 query columns) and epilogue,
// warps 10-13 dQ read-out.  TMEM columns: half a [0,128), half b [128,256): S^T, dP^T, then
// packed P^T and dA^T over S^T and dQ^T over dP^T; dV [256,384); dK [384,512).
#include <type_traits>

#include "score_tc_common.cuh"

namespace oomb {

int bwd_split(int max_sel, int n_own, int n_tiles, int G, int Hkv, const int* cluster_slots);  // attn_tc_bwd.cu

namespace {

using namespace tc;

constexpr int kRing = 4;  // Q/dO half tiles in flight
constexpr int kHalf = 64;
constexpr uint32_t kHalfTile = kHalf * kD * 2;  // 16 KB: one 64-row half tile (two 8 KB boxes)
constexpr uint32_t kHalfBox = kHalfTile / 2;
constexpr int kThreads = 448;
constexpr int kSoftmaxThreads = 256;
constexpr int kMaxCluster = 4;
constexpr int kBatch = 4;  // epilogue: pool rows in flight per thread

// A query tile's key ranges: the union of its rows' ranges [lo, hi) (empty: lo = hi = 0) and
// the range [clo, chi) that all of its rows see.
struct TileSpan {
  int64_t lo, hi, clo, chi;
};

struct ScoreBwdParams {
  ScoreArgs s;
  CapConst cap;
  const float* lse2;       // [Hq, n_pad] LSE * log2(e) (kWideCap: - cap2), +inf on rows without keys and padded rows
  const float* Dbuf;       // [Hq, n_pad] rowsum(dO * O), 0 on padded rows
  const longlong2* span;   // [n_pad] key range of each row
  const TileSpan* tiles;   // [n_tiles]
  float* dq_acc;
  int n_pad, n_tiles, n_split;
  float scale_da, scale_log2;  // scale_da: of what dK and dQ are summed from (kWideCap: 4 scale)
};

struct __align__(8) BwdBarriers {
  uint64_t kv_full;
  uint64_t hs_full[kRing];
  uint64_t hs_empty[kRing];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t dq_full[2];
  uint64_t dq_free[2];
  uint64_t acc_full;
  uint64_t staged;   // one arrival per CTA of the cluster: its partial dK/dV is staged
  uint64_t reduced;  // one arrival per CTA of the cluster: it has read every staging
  uint32_t tmem_base;
  int abort;
  int t_first, t_last;  // query tiles that can see the page
};

// shared memory map (offsets from the 1024-aligned base)
constexpr uint32_t kOffK = 0;
constexpr uint32_t kOffV = kOffK + kTileBytes;
constexpr uint32_t kOffRing = kOffV + kTileBytes;                 // kRing x (Q half, dO half)
constexpr uint32_t kOffDS = kOffRing + kRing * 2 * kHalfTile;     // 2 x dS^T half [128 keys][64 q]
constexpr uint32_t kOffVec = kOffDS + 2 * kHalfTile;              // kRing x (lse2[64], D[64])
constexpr uint32_t kOffBar = kOffVec + kRing * 2 * kHalf * 4;
// No alignment slack: the kernel has no static shared memory, and its dynamic window
// starts on a 1 KB boundary (checked at entry; the swizzled tiles need it).
constexpr size_t kSmemBytes = kOffBar + sizeof(BwdBarriers);
static_assert(kSmemBytes <= 232448, "shared memory budget");
// Epilogue staging of a CTA's partial gradients, over the K/V tiles and the ring (all
// MMAs have completed by then): [128 key rows][64 float4] = dV columns (float4 0..31)
// then scale*dK (32..63), float4 c of row j stored at position c ^ (j & 7).
constexpr uint32_t kOffStage = 0;
constexpr uint32_t kStageRow = 2 * kD * 4;  // 1 KB
static_assert(kOffStage + kTile * kStageRow <= kOffDS, "staging must not reach the dS tiles");

__device__ __forceinline__ uint32_t stage_off(int j, int c) {
  return (uint32_t)j * kStageRow + (uint32_t)((c ^ (j & 7)) * 16);
}

// Transpose of the 32 x 32 bit matrix whose row `lane` is x.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1, m ^= m << s) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, s);
    x = lane & s ? (x & ~m) | ((y & ~m) >> s) : (x & m) | ((y & m) << s);
  }
  return x;
}

// How the cap's tanh is formed.  kWideCap: r = 1 / (1 + e^2x) alone; the score cap (1 - 2 r) is
// then off by about 2^-23 cap, whose constant is folded into lse2, and 1 - tanh^2 = 4 (r - r^2),
// whose factor is left to scale_da.  One form for every x: a polynomial for small x beside it
// costs more in instruction cache than it saves (8K chunk: 7.11 against 7.59 ms).  kLargeCap, for
// caps above kCapLimit, where that error would count: the polynomial where all |x| are small.
enum CapForm { kNoCap, kWideCap, kLargeCap };
constexpr float kCapLimit = 256.0f;  // error of a score at most 2^-15, of P then 2^-15 of it

template <CapForm CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    score_bwd_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                 const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ ScoreBwdParams p) {
  // cluster = the n_split blocks of one (page s, KV head h); page-major order.  Every early
  // return below depends on (s, h) alone, so a cluster leaves as a whole.
  const AttnArgs& a = p.s.a;
  const int G = a.g.G, Hkv = a.g.Hkv;
  const int part = (int)(blockIdx.x % (unsigned)p.n_split);
  const int sh = (int)(blockIdx.x / (unsigned)p.n_split);
  const int h = sh % Hkv, s = sh / Hkv;
  const int32_t* row = a.sel + (size_t)h * a.max_sel;
  int count = a.sel_count[h];
  if (count < 0 || count > a.max_sel) {
    if (threadIdx.x == 0 && part == 0 && s == 0) atomicOr(a.err, OOMB_DEVERR_SEL);
    count = count < 0 ? 0 : a.max_sel;
  }
  if (s >= count) return;
  const int pg = row[s];
  // in range, and strictly above the previous entry and below the next one
  if (pg < 0 || pg >= p.s.n_view || pg >= a.g.max_logical || (s > 0 && row[s - 1] >= pg) ||
      (s + 1 < count && row[s + 1] <= pg)) {
    if (threadIdx.x == 0 && part == 0) atomicOr(a.err, OOMB_DEVERR_SEL);
    return;
  }
  const int phys = a.kv.table[pg];
  if (phys < 0 || phys >= a.g.num_phys) {
    if (threadIdx.x == 0 && part == 0) atomicOr(a.err, OOMB_DEVERR_PAGE);
    return;
  }
  const int64_t p0 = (int64_t)pg * kTile;

  extern __shared__ uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // uniform over the grid: every block leaves here
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.err, OOMB_DEVERR_SMEM);
    return;
  }
  uint8_t* sm = smem_raw;
  BwdBarriers* bar = reinterpret_cast<BwdBarriers*>(sm + kOffBar);
  float* vec = reinterpret_cast<float*>(sm + kOffVec);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort = &bar->abort;

  // query tiles that can see the page: those between the first and the last one whose union
  // meets it (tiles between them that do not see it are masked whole)
  if (threadIdx.x == 0) {
    bar->t_first = INT32_MAX;
    bar->t_last = -1;
  }
  __syncthreads();
  {
    int first = INT32_MAX, last = -1;
    for (int t = threadIdx.x; t < p.n_tiles; t += kThreads)
      if (p.tiles[t].hi > p0 && p.tiles[t].lo < p0 + kTile) {
        first = min(first, t);
        last = max(last, t);
      }
    if (last >= 0) {
      atomicMin(&bar->t_first, first);
      atomicMax(&bar->t_last, last);
    }
  }
  __syncthreads();
  const int t0 = bar->t_first;
  if (bar->t_last < 0) return;
  // steps (query tile t0 + su / G, query head su % G) for su in [u0, u0 + n_steps); a block
  // with no step (fewer steps than blocks) still stages a zero partial for the reduction
  const int all_steps = (bar->t_last - t0 + 1) * G;
  const int u0 = (int)((int64_t)all_steps * part / p.n_split);
  const int n_steps = (int)((int64_t)all_steps * (part + 1) / p.n_split) - u0;

  if (threadIdx.x == 0) {
    mbar_init(&bar->kv_full, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar->hs_full[i], 1);
      mbar_init(&bar->hs_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], kSoftmaxThreads / 32);  // one arrival per softmax warp
      mbar_init(&bar->dq_full[i], 1);
      mbar_init(&bar->dq_free[i], 4);                    // one arrival per read-out warp
    }
    mbar_init(&bar->acc_full, 1);
    mbar_init(&bar->staged, (uint32_t)p.n_split);
    mbar_init(&bar->reduced, (uint32_t)p.n_split);
    bar->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every CTA of the cluster has initialised its barriers once all have arrived here;
  // the epilogue waits for that before its first arrival on a peer's barrier
  cluster_arrive();
  const uint32_t tmem = bar->tmem_base;
  bool ok_acc = n_steps > 0;  // softmax warps: this CTA's dK/dV accumulators are complete

  if (n_steps <= 0) {
    // no step: nothing to load or compute
  } else if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tdo);
      const int64_t blk = a.kv.staged ? (int64_t)(a.kv.stage_h0 + h) * a.kv.stage_stride + s : (int64_t)phys * Hkv + h;
      const int row = (int)(blk * kTile);
      mbar_arrive_expect_tx(&bar->kv_full, 2 * kTileBytes);
      tma_load_2d(sm + kOffK, &tk, &bar->kv_full, 0, row);
      tma_load_2d(sm + kOffK + kHalfBytes, &tk, &bar->kv_full, 64, row);
      tma_load_2d(sm + kOffV, &tv, &bar->kv_full, 0, row);
      tma_load_2d(sm + kOffV + kHalfBytes, &tv, &bar->kv_full, 64, row);
    }
    int v = 0;
    if (lane == 0) {
      for (; v < 2 * n_steps; ++v) {
        const int slot = v % kRing;
        if (v >= kRing && !mbar_wait(&bar->hs_empty[slot], ((v / kRing) - 1) & 1, a.err, abort)) break;
        const int su = u0 + (v >> 1), hh = v & 1;
        const int t = t0 + su / G, g = su % G;
        const int hq = h * G + g;
        const int q0 = t * kTile + hh * kHalf;
        uint8_t* dst = sm + kOffRing + slot * 2 * kHalfTile;
        float* vs = vec + slot * 2 * kHalf;
        mbar_arrive_expect_tx(&bar->hs_full[slot], 2 * kHalfTile + 2 * kHalf * 4);
        tma_load_3d(dst, &tq, &bar->hs_full[slot], 0, hq, q0);
        tma_load_3d(dst + kHalfBox, &tq, &bar->hs_full[slot], 64, hq, q0);
        tma_load_3d(dst + kHalfTile, &tdo, &bar->hs_full[slot], 0, hq, q0);
        tma_load_3d(dst + kHalfTile + kHalfBox, &tdo, &bar->hs_full[slot], 64, hq, q0);
        // LSE * log2(e) and D of the 64 rows (padded rows hold +inf and 0)
        bulk_load(vs, p.lse2 + (size_t)hq * p.n_pad + q0, kHalf * 4, &bar->hs_full[slot]);
        bulk_load(vs + kHalf, p.Dbuf + (size_t)hq * p.n_pad + q0, kHalf * 4, &bar->hs_full[slot]);
      }
    }
    if (lane == 0) {  // drain the copies still in flight before the CTA may exit
      for (int vv = (v > kRing ? v - kRing : 0); vv < v; ++vv)
        mbar_wait(&bar->hs_full[vv % kRing], (vv / kRing) & 1, a.err, nullptr);
      mbar_wait(&bar->kv_full, 0, a.err, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_bf16_f32(128, 64, false, false);   // S^T, dP^T
      const uint32_t id_acc = idesc_bf16_f32(128, 128, false, true);  // dV, dK (A from TMEM)
      const uint32_t id_dq = idesc_bf16_f32(128, 64, true, true);     // dQ^T
      const uint32_t aK = smem_u32(sm + kOffK), aV = smem_u32(sm + kOffV);
      bool ok = mbar_wait(&bar->kv_full, 0, a.err, abort);
      bool first_acc = true;
      // S^T, dP^T of half-step v = 2u + hh into the half's TMEM region
      auto issue_sdp = [&](int u, int hh) -> bool {
        const int v = 2 * u + hh, slot = v % kRing;
        if (!mbar_wait(&bar->hs_full[slot], (v / kRing) & 1, a.err, abort)) return false;
        if (u > 0 && !mbar_wait(&bar->dq_free[hh], (u - 1) & 1, a.err, abort)) return false;  // dQ^T read out
        tc_fence_after();
        const uint32_t aQ = smem_u32(sm + kOffRing + slot * 2 * kHalfTile);
        const uint32_t adO = aQ + kHalfTile;
        const uint32_t tS = tmem + hh * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ss(tS, desc_kmajor(aK, kk), desc_kmajor(aQ, kk, kHalfBox), id_s, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tS + 64, desc_kmajor(aV, kk), desc_kmajor(adO, kk, kHalfBox), id_s, kk > 0);
        mma_commit(&bar->s_full[hh]);
        return true;
      };
      // dQ^T = K^T dS^T, then dV += P^T dO and dK += dS^T Q once the half's softmax is
      // done (dQ^T first, so that its read-out overlaps dV and dK)
      auto issue_acc = [&](int u, int hh) -> bool {
        const int v = 2 * u + hh, slot = v % kRing;
        if (!mbar_wait(&bar->p_full[hh], u & 1, a.err, abort)) return false;
        tc_fence_after();
        const uint32_t aQ = smem_u32(sm + kOffRing + slot * 2 * kHalfTile);
        const uint32_t adO = aQ + kHalfTile;
        const uint32_t tS = tmem + hh * 128;
        const uint32_t adS = smem_u32(sm + kOffDS + hh * kHalfTile);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tS + 64, desc_mnmajor(aK, kk), desc_mnmajor(adS, kk, kHalfBox), id_dq, kk > 0);
        mma_commit(&bar->dq_full[hh]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          // query columns [16 kk, 16 kk + 16): packed P^T / dS^T of column group kk / 2
          const uint32_t a = tS + 32 * (kk >> 1) + 8 * (kk & 1);
          mma_ts(tmem + 256, a, desc_mnmajor(adO, kk, kHalfBox), id_acc, first_acc ? 0u : 1u);
          mma_ts(tmem + 384, a + 16, desc_mnmajor(aQ, kk, kHalfBox), id_acc, first_acc ? 0u : 1u);
          first_acc = false;
        }
        mma_commit(&bar->hs_empty[slot]);
        return true;
      };
      // half b's softmax overlaps the next step's S/dP of half a, and vice versa
      if (ok) ok = issue_sdp(0, 0) && issue_sdp(0, 1);
      for (int u = 0; ok && u < n_steps; ++u) {
        ok = issue_acc(u, 0);
        if (ok && u + 1 < n_steps) ok = issue_sdp(u + 1, 0);
        if (ok) ok = issue_acc(u, 1);
        if (ok && u + 1 < n_steps) ok = issue_sdp(u + 1, 1);
      }
      mma_commit(&bar->acc_full);
      mbar_wait(&bar->acc_full, 0, a.err, nullptr);
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------------ softmax
    const int j = (warp & 3) * 32 + lane;  // key row of the page
    const int hc = (warp - 2) >> 2;        // query columns [32 hc, 32 hc + 32) of each half
    const uint32_t lane_off = tmem_lane_base(warp);
    const int64_t kpos = p0 + j;
    bool ok = true;
    for (int u = 0; ok && u < n_steps; ++u) {
      const int t = t0 + (u0 + u) / G;
      const bool masked = p.tiles[t].clo > p0 || p.tiles[t].chi < p0 + kTile;
      const float slope2 = BIAS ? p.s.slopes[h * G + (u0 + u) % G] * kLog2e : 0.f;
      for (int hh = 0; hh < 2; ++hh) {
        const int v = 2 * u + hh, slot = v % kRing;
        ok = mbar_wait(&bar->s_full[hh], u & 1, a.err, abort) &&
             mbar_wait(&bar->hs_full[slot], (v / kRing) & 1, a.err, abort);
        ok = __all_sync(0xffffffffu, ok);  // TMEM loads and stores below are warp-collective
        if (!ok) break;
        tc_fence_after();
        const uint32_t base = tmem + lane_off + hh * 128 + 32 * hc;
        uint32_t sr[32], dr[32];
        tmem_ld32(base, sr);
        tmem_ld32(base + 64, dr);
        tmem_wait_ld();
        const float4* vs4 = reinterpret_cast<const float4*>(vec + slot * 2 * kHalf) + 8 * hc;  // lse2, D
        const int q0 = t * kTile + hh * kHalf + 32 * hc;  // query row of this thread's column 0
        uint32_t see = 0xffffffffu;                       // columns whose row sees this key
        if (masked) {
          // lane i: the warp's 32 keys that row q0 + i sees, as bits; transposed, lane k has the
          // rows that see its key
          const longlong2 w = p.span[q0 + lane];
          const int64_t k0 = kpos - lane;
          const int b = (int)max((int64_t)0, min((int64_t)(w.x - k0), (int64_t)32));
          const int e = (int)max((int64_t)0, min((int64_t)(w.y - k0), (int64_t)32));
          see = transpose_bits(b >= e ? 0u : (0xffffffffu >> (32 - (e - b))) << b, lane);
        }
        const float f0 = BIAS ? (float)(a.q_start + q0 - kpos) : 0.f;  // distance of column i: |f0 + i|
        uint32_t pk[16], dk[16];
        // P and dA of the columns, four at a time
        auto columns = [&](auto small) {
#pragma unroll
          for (int c4 = 0; c4 < 8; ++c4) {
            const float4 L = vs4[c4], Dv = vs4[16 + c4];
            const float l4[4] = {L.x, L.y, L.z, L.w}, d4[4] = {Dv.x, Dv.y, Dv.z, Dv.w};
            float pr[4], dar[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 4 * c4 + e;
              const float S = __uint_as_float(sr[i]);
              float shift = -l4[e], s2, gate = 1.f;
              if (BIAS) shift = fmaf(-slope2, fabsf(f0 + (float)i), shift);
              if constexpr (CAP == kWideCap) {
                const float r = rcp_approx(1.f + ex2_approx(p.cap.arg * S));
                s2 = fmaf(r, -2.f * p.cap.cap2, shift);
                gate = fmaf(-r, r, r);
              } else if constexpr (CAP == kLargeCap) {
                const float th = tanh_of<decltype(small)::value ? kDegree3 : kWide>(S, p.cap);
                s2 = fmaf(th, p.cap.cap2, shift);
                gate = fmaf(-th, th, 1.f);
              } else {
                s2 = fmaf(S, p.scale_log2, shift);
              }
              pr[e] = ex2_approx(s2);
              dar[e] = pr[e] * (__uint_as_float(dr[i]) - d4[e]);
              if constexpr (CAP != kNoCap) dar[e] *= gate;
            }
            pk[2 * c4] = pack_bf16x2(pr[0], pr[1]);
            pk[2 * c4 + 1] = pack_bf16x2(pr[2], pr[3]);
            dk[2 * c4] = pack_bf16x2(dar[0], dar[1]);
            dk[2 * c4 + 1] = pack_bf16x2(dar[2], dar[3]);
          }
        };
        bool small = false;
        if constexpr (CAP == kLargeCap) {
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) amax = fmax3_abs(amax, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
          small = __all_sync(0xffffffffu, amax <= p.cap.edge3);
        }
        if (CAP == kLargeCap && small)
          columns(std::true_type{});
        else
          columns(std::false_type{});
        if (masked) {  // cleared afterwards, in the packed words, whatever came out for a pair that is not seen
#pragma unroll
          for (int w = 0; w < 16; ++w) {
            const uint32_t keep = ((see >> (2 * w)) & 1u) * 0x0000ffffu | ((see >> (2 * w + 1)) & 1u) * 0xffff0000u;
            pk[w] &= keep;
            dk[w] &= keep;
          }
        }
        // P^T and dA^T go over this thread's own (already loaded) S^T columns
        tmem_st16(base, pk);
        tmem_st16(base + 16, dk);
        // dA^T row j, query columns [32 hc, 32 hc + 32): four 16-byte chunks of the swizzled tile
        uint8_t* drow = sm + kOffDS + hh * kHalfTile + j * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int chunk = hc * 4 + c;
          uint4 w = make_uint4(dk[4 * c], dk[4 * c + 1], dk[4 * c + 2], dk[4 * c + 3]);
          *reinterpret_cast<uint4*>(drow + ((chunk ^ (j & 7)) * 16)) = w;
        }
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[hh]);
      }
    }
    ok_acc = ok;
  } else {
    // ------------------------------------------------------------------ dQ read-out
    // Each thread holds one head-dim column of dQ^T for the half's 64 query rows and adds
    // it into the fp32 accumulator with global reductions: for a given row the warp's 32
    // lanes cover 32 consecutive columns (one 128-byte line), and no shared memory is used.
    const int col = (warp & 3) * 32 + lane;  // head-dim column == TMEM lane of dQ^T
    const uint32_t lane_off = tmem_lane_base(warp);
    bool ok = true;
    for (int u = 0; ok && u < n_steps; ++u) {
      const int t = t0 + (u0 + u) / G, g = (u0 + u) % G;
      const int hq = h * G + g;
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t r[64];
        ok = __all_sync(0xffffffffu, mbar_wait(&bar->dq_full[hh], u & 1, a.err, abort));
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tmem + lane_off + hh * 128 + 64, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tmem_ld32(tmem + lane_off + hh * 128 + 96, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->dq_free[hh]);  // dQ^T is in registers: its columns are free
        const int q0 = t * kTile + hh * kHalf;
        const int nrows = min(kHalf, a.n_q - q0);
        float* dst = p.dq_acc + ((size_t)hq * a.n_q + q0) * kD + col;
#pragma unroll
        for (int rr = 0; rr < kHalf; ++rr)
          if (rr < nrows) atomicAdd(dst + (size_t)rr * kD, __uint_as_float(r[rr]));
      }
    }
  }

  // ------------------------------------------------------------------ dK/dV epilogue
  if (warp >= 2 && warp < 10) {
    const int et = threadIdx.x - 64;  // 0..255
    const int j = (warp & 3) * 32 + lane;  // key row == TMEM lane
    const int hc = (warp - 2) >> 2;        // dV / dK columns [64 hc, 64 hc + 64)
    const uint32_t lane_off = tmem_lane_base(warp);
    // the pool rows this CTA will own: key rows [r0, r1) of the block's dV and dK, pulled
    // into L2 while the partials are staged
    const uint32_t n = (uint32_t)p.n_split;
    const int rank = (int)cluster_ctarank();
    const int r0 = kTile * rank / (int)n, r1 = kTile * (rank + 1) / (int)n;
    const size_t blk = a.grad_staged ? (size_t)(a.kv.stage_h0 + h) * a.kv.stage_stride + s : (size_t)phys * Hkv + h;
    float4* gdv = reinterpret_cast<float4*>(a.dv_pool + blk * kTile * kD);
    float4* gdk = reinterpret_cast<float4*>(a.dk_pool + blk * kTile * kD);
    if (et == 0) {
      prefetch_l2(gdv + (size_t)r0 * (kD / 4), (uint32_t)(r1 - r0) * kD * 4);
      prefetch_l2(gdk + (size_t)r0 * (kD / 4), (uint32_t)(r1 - r0) * kD * 4);
    }
    // (1) stage this CTA's partial (zero when it had no step or its pipeline gave up)
    const bool have = __all_sync(0xffffffffu, ok_acc && mbar_wait(&bar->acc_full, 0, a.err, abort));
    if (have) tc_fence_after();
#pragma unroll 1
    for (int cc = 0; cc < 2; ++cc) {
      uint32_t a[32], b[32];
      if (have) {
        tmem_ld32(tmem + lane_off + 256 + 64 * hc + cc * 32, a);
        tmem_ld32(tmem + lane_off + 384 + 64 * hc + cc * 32, b);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = b[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = 16 * hc + 8 * cc + e;  // float4 column of dV; 32 + c of dK
        *reinterpret_cast<float4*>(sm + kOffStage + stage_off(j, c)) =
            make_float4(__uint_as_float(a[4 * e]), __uint_as_float(a[4 * e + 1]), __uint_as_float(a[4 * e + 2]),
                        __uint_as_float(a[4 * e + 3]));
        *reinterpret_cast<float4*>(sm + kOffStage + stage_off(j, 32 + c)) =
            make_float4(p.scale_da * __uint_as_float(b[4 * e]), p.scale_da * __uint_as_float(b[4 * e + 1]),
                        p.scale_da * __uint_as_float(b[4 * e + 2]), p.scale_da * __uint_as_float(b[4 * e + 3]));
      }
    }
    fence_acq_rel_cluster();
    named_bar_sync(1, kSoftmaxThreads);
    cluster_wait();  // every peer's barriers are initialised
    if (et == 0)
      for (uint32_t q = 0; q < n; ++q) mbar_arrive_cluster(mapa_shared(smem_u32(&bar->staged), q));
    // (2) reduce key rows [r0, r1) over the cluster's partials, in rank order, into the pool
    if (__all_sync(0xffffffffu, mbar_wait_cluster(&bar->staged, 0, a.err))) {
      const uint32_t base = smem_u32(sm + kOffStage);
      const int n_items = (r1 - r0) * 64;  // (row, float4 column); a warp: one row, 32 consecutive float4
      // kBatch items per thread in flight: pool loads (from L2, prefetched above) and the
      // partials of every rank are all issued before the first add
      for (int i0 = et; i0 < n_items; i0 += kBatch * kSoftmaxThreads) {
        float4 x[kBatch], t[kBatch];
        float4* g[kBatch];
        uint32_t off[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int idx = min(i0 + u * kSoftmaxThreads, n_items - 1);  // clamped duplicates are not stored
          const int jj = r0 + idx / 64, c = idx % 64;
          off[u] = stage_off(jj, c);
          g[u] = (c < 32 ? gdv : gdk) + (size_t)jj * (kD / 4) + (c & 31);
          x[u] = *g[u];
          t[u] = ld_dsmem_f4(mapa_shared(base + off[u], 0));
        }
        for (uint32_t q = 1; q < n; ++q) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const float4 v = ld_dsmem_f4(mapa_shared(base + off[u], q));
            t[u].x += v.x;
            t[u].y += v.y;
            t[u].z += v.z;
            t[u].w += v.w;
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (i0 + u * kSoftmaxThreads < n_items) {
            x[u].x += t[u].x;
            x[u].y += t[u].y;
            x[u].z += t[u].z;
            x[u].w += t[u].w;
            *g[u] = x[u];
          }
        }
      }
    }
    // (3) this CTA has read every peer's staging; wait until its own was read by all
    fence_acq_rel_cluster();
    named_bar_sync(1, kSoftmaxThreads);
    if (et == 0)
      for (uint32_t q = 0; q < n; ++q) mbar_arrive_cluster(mapa_shared(smem_u32(&bar->reduced), q));
    mbar_wait_cluster(&bar->reduced, 0, a.err);
  } else {
    cluster_wait();  // every thread that arrived also waits once (long complete by now)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Blocks [0, n_tiles): the row ranges of one query tile.  The others, one warp per (row, head)
// of the padded range: D = rowsum(dO * O) and LSE * log2(e) into [Hq, n_pad] buffers (rows
// without keys and padded rows: LSE = +inf, so P = 0; cap2 is taken off) and the row of the fp32 dQ
// accumulator zeroed.  D comes from O as the forward rounded it to bf16, the only form of it that a
// caller keeps: off by 2^-8 |dO| |O| at most, as much as the rounded P of the products.
__global__ void __launch_bounds__(256) score_bwd_prep(const __grid_constant__ ScoreArgs s, float cap2, int n_pad,
                                                      int n_tiles, float* __restrict__ Dbuf, float* __restrict__ lse2,
                                                      float* __restrict__ dq_acc, longlong2* __restrict__ span,
                                                      TileSpan* __restrict__ tiles) {
  const AttnArgs& a = s.a;
  const int lane = threadIdx.x % 32;
  if ((int)blockIdx.x < n_tiles) {
    __shared__ TileSpan part[4];
    const int i = (int)blockIdx.x * kTile + (int)threadIdx.x, w = threadIdx.x / 32;
    if (threadIdx.x < kTile) {
      int64_t b = 0, e = INT64_MAX;  // padded rows ask for no masking (their P is 0)
      TileSpan t = {INT64_MAX, 0, 0, INT64_MAX};
      if (i < a.n_q) {
        row_span(s, i, b, e);
        if (e > b) t = {b, e, b, e}; else t = {INT64_MAX, 0, b, e};
      }
      span[i] = make_longlong2(b, e);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t.lo = min(t.lo, __shfl_xor_sync(0xffffffffu, t.lo, o));
        t.hi = max(t.hi, __shfl_xor_sync(0xffffffffu, t.hi, o));
        t.clo = max(t.clo, __shfl_xor_sync(0xffffffffu, t.clo, o));
        t.chi = min(t.chi, __shfl_xor_sync(0xffffffffu, t.chi, o));
      }
      if (lane == 0) part[w] = t;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      TileSpan t = part[0];
      for (int k = 1; k < 4; ++k) {
        t.lo = min(t.lo, part[k].lo);
        t.hi = max(t.hi, part[k].hi);
        t.clo = max(t.clo, part[k].clo);
        t.chi = min(t.chi, part[k].chi);
      }
      tiles[blockIdx.x] = t;
    }
    return;
  }
  const int64_t w = ((int64_t)(blockIdx.x - n_tiles) * blockDim.x + threadIdx.x) / 32;
  const int Hq = a.g.Hq;
  if (w >= (int64_t)n_pad * Hq) return;
  const int i = (int)(w / Hq), hq = (int)(w % Hq);
  if (i >= a.n_q) {
    if (lane == 0) {
      Dbuf[(size_t)hq * n_pad + i] = 0.f;
      lse2[(size_t)hq * n_pad + i] = INFINITY;
    }
    return;
  }
  const size_t off = ((size_t)i * Hq + hq) * kD + lane * 4;
  const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.o) + off);
  const uint2 y = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.dout) + off);
  const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x);
  const __nv_bfloat162* y2 = reinterpret_cast<const __nv_bfloat162*>(&y);
  float d = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 u = __bfloat1622float2(x2[e]), v = __bfloat1622float2(y2[e]);
    d += u.x * v.x + u.y * v.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) {
    const float l = a.lse_in[(size_t)hq * a.n_q + i];
    Dbuf[(size_t)hq * n_pad + i] = d;
    lse2[(size_t)hq * n_pad + i] = l == -INFINITY ? INFINITY : l * kLog2e - cap2;
  }
  reinterpret_cast<float4*>(dq_acc + ((size_t)hq * a.n_q + i) * kD)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// dq[i][hq][:] = bf16(scale * dq_acc[hq][i][:]).  One warp per (row, head).
__global__ void __launch_bounds__(256) score_bwd_convert(const float* __restrict__ dq_acc, int n_q, int Hq, float scale,
                                                         __nv_bfloat16* __restrict__ dq) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x % 32;
  if (w >= (int64_t)n_q * Hq) return;
  const int i = (int)(w / Hq), hq = (int)(w % Hq);
  const float4 x = reinterpret_cast<const float4*>(dq_acc + ((size_t)hq * n_q + i) * kD)[lane];
  uint2 out;
  out.x = pack_bf16x2(x.x * scale, x.y * scale);
  out.y = pack_bf16x2(x.z * scale, x.w * scale);
  *reinterpret_cast<uint2*>(dq + ((size_t)i * Hq + hq) * kD + lane * 4) = out;
}

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, unsigned blocks, int n_split, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)n_split;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <CapForm CAP, bool BIAS>
cudaError_t launch_main(ScoreBwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t st) {
  static size_t smem_set[kMaxDevices] = {};
  static int slots[kMaxDevices][kMaxCluster + 1] = {};  // clusters of n blocks resident at once
  const void* fn = (const void*)score_bwd_tc<CAP, BIAS>;
  cudaError_t e = set_smem_limit(fn, kSmemBytes, smem_set);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  if (!slots[dev][1]) {
    int tmp[kMaxCluster + 1] = {};
    for (int n = 1; n <= kMaxCluster; ++n) {
      const cudaLaunchConfig_t cfg = cluster_config(&attr, (unsigned)n * 64, n, nullptr);
      e = cudaOccupancyMaxActiveClusters(&tmp[n], fn, &cfg);
      if (e != cudaSuccess) return e;
    }
    for (int n = kMaxCluster; n >= 1; --n) slots[dev][n] = tmp[n];
  }
  const AttnArgs& a = p.s.a;
  const int64_t own0 = a.q_start / kTile;
  const int n_own = (int)((a.q_start + a.n_q + kTile - 1) / kTile - own0);
  p.n_split = bwd_split(a.max_sel, n_own, p.n_tiles, a.g.G, a.g.Hkv, slots[dev]);
  const cudaLaunchConfig_t cfg =
      cluster_config(&attr, (unsigned)a.max_sel * (unsigned)p.n_split * (unsigned)a.g.Hkv, p.n_split, st);
  e = cudaLaunchKernelEx(&cfg, score_bwd_tc<CAP, BIAS>, tq, tdo, tk, tv, p);
  count_launches(1);
  return e;
}

}  // namespace

size_t score_bwd_tc_workspace_bytes(const Geometry& g, int n_q) {
  const size_t n_pad = (size_t)(n_q + kTile - 1) / kTile * kTile;
  return 2 * align_up((size_t)g.Hq * n_pad * 4, 256) + align_up((size_t)g.Hq * n_q * kD * 4, 256) +
         align_up(n_pad * sizeof(longlong2), 256) + align_up(n_pad / kTile * sizeof(TileSpan), 256);
}

cudaError_t launch_score_bwd_tc(const ScoreArgs& s, cudaStream_t st) {
  const AttnArgs& a = s.a;
  const int n_tiles = (a.n_q + kTile - 1) / kTile, n_pad = n_tiles * kTile;
  char* ws = reinterpret_cast<char*>(a.ws);
  auto take = [&](size_t bytes) {
    char* at = ws;
    ws += align_up(bytes, 256);
    return at;
  };
  float* Dbuf = reinterpret_cast<float*>(take((size_t)a.g.Hq * n_pad * 4));
  float* lse2 = reinterpret_cast<float*>(take((size_t)a.g.Hq * n_pad * 4));
  float* dq_acc = reinterpret_cast<float*>(take((size_t)a.g.Hq * a.n_q * kD * 4));
  longlong2* span = reinterpret_cast<longlong2*>(take((size_t)n_pad * sizeof(longlong2)));
  TileSpan* tiles = reinterpret_cast<TileSpan*>(take((size_t)n_tiles * sizeof(TileSpan)));
  const CapForm form = !(s.cap > 0.f) ? kNoCap : s.cap <= kCapLimit ? kWideCap : kLargeCap;
  const int64_t warps = (int64_t)a.n_q * a.g.Hq, warps_pad = (int64_t)n_pad * a.g.Hq;
  score_bwd_prep<<<(unsigned)(n_tiles + (warps_pad + 7) / 8), 256, 0, st>>>(
      s, form == kWideCap ? s.cap * kLog2e : 0.f, n_pad, n_tiles, Dbuf, lse2, dq_acc, span, tiles);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tdo, tk, tv;
  if (!make_tmap_heads(&tq, a.q, a.n_q, a.g.Hq, kHalf) || !make_tmap_heads(&tdo, a.dout, a.n_q, a.g.Hq, kHalf) ||
      !make_tmap_rows(&tk, a.kv.k, kv_rows(a)) || !make_tmap_rows(&tv, a.kv.v, kv_rows(a)))
    return cudaErrorInvalidValue;
  ScoreBwdParams p;
  p.s = s;
  p.cap = make_cap(s.cap, a.scale);
  p.lse2 = lse2;
  p.Dbuf = Dbuf;
  p.span = span;
  p.tiles = tiles;
  p.dq_acc = dq_acc;
  p.n_pad = n_pad;
  p.n_tiles = n_tiles;
  p.scale_da = form == kWideCap ? 4.f * a.scale : a.scale;
  p.scale_log2 = a.scale * kLog2e;
  const bool bias = s.slopes != nullptr;
  if (form == kWideCap)
    e = bias ? launch_main<kWideCap, true>(p, tq, tdo, tk, tv, st)
             : launch_main<kWideCap, false>(p, tq, tdo, tk, tv, st);
  else if (form == kLargeCap)
    e = bias ? launch_main<kLargeCap, true>(p, tq, tdo, tk, tv, st)
             : launch_main<kLargeCap, false>(p, tq, tdo, tk, tv, st);
  else
    e = bias ? launch_main<kNoCap, true>(p, tq, tdo, tk, tv, st) : launch_main<kNoCap, false>(p, tq, tdo, tk, tv, st);
  if (e != cudaSuccess) return e;
  score_bwd_convert<<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(dq_acc, a.n_q, a.g.Hq, p.scale_da,
                                                                 reinterpret_cast<__nv_bfloat16*>(a.dq));
  count_launches(2);
  return cudaGetLastError();
}

}  // namespace oomb
