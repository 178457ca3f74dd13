// The four matrix products of the loss over a vocabulary (head_loss.cu), on the tensor cores with
// tcgen05 in pairs of SMs, each with its own epilogue:
//
//   kLse   z = X W^T, a tile of 256 rows and 256 columns: row maxima and sums of exponentials
//   kDz    the same product again: dz = g (exp(z' - lse) - [target]) (1 - (z'/cap)^2), stored
//   kDx    dx = dz W over a piece of the vocabulary
//   kDw    dw = dz^T X over the rows with a target
//
// Operands are bf16.  fp32 operands are three bf16 parts of 8 bits each (h + m + l = all 24 bits) and
// a product is the six products of parts that are above 2^-24 of it, the small ones first, so that
// the accumulator is small while they are added.
//
// A tile is 256 x 256 over the two CTAs of a cluster: each holds 128 rows of A and 128 of the 256
// columns' rows of B, so a CTA loads 32 KB for 64 steps of K instead of the 48 KB that a tile of
// its own of the same shape would take; that is what keeps the loads below L2's rate.  Six stages
// of a ring; two accumulators of 256 columns in tensor memory, so that a tile's epilogue (eight
// warps, a thread a row, whose results go through shared memory to be written in lines) runs while the
// next tile's product does.  Persistent: a cluster takes
// tiles c, c + clusters, ... in groups of kGroup row tiles, which share the columns' tiles in L2.
#pragma once
#include "head_loss.h"
#include "head_plan.h"
#include "tc_common.cuh"

namespace oomb {
namespace head {

enum Mode { kLse = 0, kDz = 1, kDx = 2, kDw = 3 };

constexpr uint32_t kOperand = kHalf * kStep * 2;     // 16 KB
constexpr int kThreads = 320;                        // producer, issuer, 8 epilogue warps
constexpr int kEpilogueWarps = 8;
constexpr int kMaxStages = 9;
// Tiles of TN columns: kTile, or kNarrow where there are few tiles.
template <int TN>
struct Shape {
  static constexpr int half = TN / 2;                           // columns of an epilogue warp, rows of B a CTA loads
  static constexpr uint32_t b_bytes = half * kStep * 2;
  static constexpr uint32_t stage = kOperand + b_bytes;
  static constexpr int stages = TN == 256 ? 6 : kMaxStages;
  static constexpr uint32_t turn = kEpilogueWarps * 32 * 33 * 4;  // where the epilogue turns rows into lines
  static constexpr uint32_t smem = stages * stage + turn + 1024;
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tile_full[2], tile_empty[2], done;
  uint32_t tmem;
  int abort;
};

// ---- tcgen05 in pairs
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on this barrier in both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Whether a barrier's phase has been passed; does not wait.
__device__ __forceinline__ bool passed(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same, on this CTA's barrier only.
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Tile of this CTA's shared memory whose bytes are counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load2(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Parts multiplied in pass p of six, the smallest products first.
__device__ __forceinline__ int part_a(int passes, int p) { return passes == 1 ? 0 : (0x021010 >> (4 * (5 - p))) & 15; }
__device__ __forceinline__ int part_b(int passes, int p) { return passes == 1 ? 0 : (0x201100 >> (4 * (5 - p))) & 15; }

// Place of tile t among tms x tns tiles: groups of kGroup row tiles, row tiles first within one.
__device__ __forceinline__ void place(int t, int tms, int tns, int kGroup, int& tm, int& tn) {
  const int per = kGroup * tns, g = t / per, r = t - g * per, rows = min(kGroup, tms - g * kGroup);
  tn = r / rows;
  tm = g * kGroup + (r - tn * rows);
}

__device__ __forceinline__ void store16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// z = cap tanh(z / cap) of 32 columns, known to 3e-7 of itself.  u = z / cap: below 0.4 from the series, since
// a cap far above the logits multiplies what is lost elsewhere; above from one exponential and one
// reciprocal, which are 2^-23 or so off one.  Where all of a warp's are below, only the series is
// formed, two columns an instruction (1601 rows on 50001 x 2048 under a cap of 30: 301 us to 262, both
// directions 1044 to 1008).
__device__ __forceinline__ void cap_logits(float (&z)[32], float cap, float inv_cap) {
  // of v^5 to v^1, v = u^2; the next term is 6e-8 of the sum at 0.4
  constexpr float c4 = -1382.f / 155925.f, c3 = 62.f / 2835.f, c2 = -17.f / 315.f, c1 = 2.f / 15.f, c0 = -1.f / 3.f;
  const uint64_t inv2 = f32x2(inv_cap, inv_cap);
  auto series = [&](uint64_t x) {
    const uint64_t u = mul2(x, inv2), v = mul2(u, u);
    uint64_t q = fma2(v, f32x2(c4, c4), f32x2(c3, c3));
    q = fma2(q, v, f32x2(c2, c2));
    q = fma2(q, v, f32x2(c1, c1));
    q = fma2(q, v, f32x2(c0, c0));
    return fma2(mul2(x, v), q, x);
  };
  auto either = [&](float x, float of_series) {
    const float u = x * inv_cap;
    const float t = cap * fmaf(-2.f, rcp_approx(1.f + ex2_approx(u * (2.f * tc::kLog2e))), 1.f);
    return fabsf(u) < 0.4f ? of_series : t;
  };
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; i += 2) m[i / 2 & 3] = fmax3(m[i / 2 & 3], fabsf(z[i]), fabsf(z[i + 1]));
  // (a NaN is no maximum, and stays one in either form)
  if (__all_sync(0xffffffffu, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * inv_cap < 0.4f)) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) f32x2_split(series(f32x2(z[i], z[i + 1])), z[i], z[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float s0, s1;
      f32x2_split(series(f32x2(z[i], z[i + 1])), s0, s1);
      z[i] = either(z[i], s0);
      z[i + 1] = either(z[i + 1], s1);
    }
  }
}

// Maximum and sum of exponentials of a row's columns, base 2.
struct RowSum {
  float m = -INFINITY, s = 0.f;
  // n: how many of the 32 columns exist
  __device__ __forceinline__ void add(float (&z)[32], int n) {
    if (n <= 0) return;
    float mx = m;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      z[i] = i < n ? z[i] * tc::kLog2e : -INFINITY;
      mx = fmaxf(mx, z[i]);
    }
    const float to = mx == -INFINITY ? 0.f : mx;  // nothing above -infinity yet (a NaN is no maximum, but stays one)
    s *= ex2_approx(m - to);
    m = mx;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i & 3] += ex2_approx(z[i] - to);
    s += (t[0] + t[1]) + (t[2] + t[3]);
  }
};

// CHUNKED: K is cut in pieces of p.chunk steps whose sums are added in fp32 in registers.  The tensor
// cores cut a partial sum's last bits instead of rounding them, always towards zero: 6e-6 of a logit
// over K = 3584 is lost, which a loss in fp32 would show, and 4e-7 over 256; of sums of one sign 1.8e-7 of the
// partial sum for every 16 products (a dw over 65536 rows: 3.8e-4).  The host asks for pieces wherever the
// output would show it.
template <int MODE, bool CHUNKED, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    head_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
              const __grid_constant__ GemmArgs p) {
  constexpr bool kAmn = MODE == kDw, kBmn = MODE == kDx || MODE == kDw;
  static_assert(TN == 256 || !kBmn, "a narrow tile's half of B is no whole swizzled row");
  using S = Shape<TN>;
  constexpr int kStages = S::stages, kCols = S::half;
  constexpr uint32_t kStageBytes = S::stage;
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bar;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  volatile int* abort = &bar.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.tile_full[i], 1);
      mbar_init(&bar.tile_empty[i], 2 * kEpilogueWarps);
    }
    mbar_init(&bar.done, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  if (warp == 1) tmem_alloc2(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("fence.proxy.async;" ::: "memory");  // what earlier kernels stored is read by copies
  const int count = *p.count;
  const int tms = MODE == kDw ? p.tms : (count + kTile - 1) / kTile;
  const int steps_all = MODE == kDw ? (count + kStep - 1) / kStep : p.steps;
  const int clusters = gridDim.x / 2, first = blockIdx.x / 2;
  // K in parts: kDx in as many as the rows with a target ask for, kDw in as many as the host says
  const int all_splits = MODE == kDx ? p.count[1] : MODE == kDw ? p.dw_splits : 1;
  const int splits = MODE == kDx ? min(all_splits, max(1, steps_all)) : all_splits;
  const bool last = MODE == kDx ? p.last && all_splits == 1 : all_splits == 1;  // else the sums are kept
  const int tiles = tms * p.tns * splits;
  // steps of K of a tile: its split's share
  auto range = [&](int t, int& k0, int& k1) {
    const int s = t / (tms * p.tns);
    k0 = (int)((int64_t)steps_all * s / splits);
    k1 = (int)((int64_t)steps_all * (s + 1) / splits);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&bar.full[0]), 0), empty0 = smem_u32(&bar.empty[0]);
      int s = 0, it = 0;
      uint32_t phase = 1;  // of the stage before: the first round finds the stages empty
      bool ok = true;
      for (int t = first; ok && t < tiles; t += clusters) {
        int tm, tn, k0, k1;
        place(t % (tms * p.tns), tms, p.tns, p.group, tm, tn);
        range(t, k0, k1);
        const int ra = tm * kTile + (int)rank * kHalf, rb = tn * TN + (int)rank * kCols;
        const int chunk = CHUNKED ? p.chunk : max(1, k1 - k0);
        for (int c0 = k0; ok && c0 < k1; c0 += chunk) {
          const int c1 = min(k1, c0 + chunk);
          for (int q = 0; ok && q < p.passes; ++q) {
            const int pa = part_a(p.passes, q), pb = part_b(p.passes, q);
            for (int k = c0; k < c1; ++k) {
              if (it >= kStages && !passed(empty0 + 8 * s, phase)) {
                ok = mbar_wait(&bar.empty[s], phase, p.err, abort);
                if (!ok) break;
              }
              if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], 2 * kStageBytes);
              const uint32_t a = base + s * kStageBytes, b = a + kOperand, f = full0 + 8 * s;
              if (kAmn) {
                tma_load2(a, &ta, f, ra, k * kStep, pa);
                tma_load2(a + kOperand / 2, &ta, f, ra + 64, k * kStep, pa);
              } else {
                tma_load2(a, &ta, f, k * kStep, ra, pa);
              }
              if (kBmn) {
                tma_load2(b, &tb, f, rb, p.row_b + k * kStep, pb);
                tma_load2(b + kOperand / 2, &tb, f, rb + 64, p.row_b + k * kStep, pb);
              } else {
                tma_load2(b, &tb, f, k * kStep, p.row_b + rb, pb);
              }
              ++it;
              if (++s == kStages) {
                s = 0;
                phase ^= 1;
              }
            }
          }
        }
      }
      // Every stage handed on has been read (so its copies have landed and the commits that tell it
      // have arrived) before the CTA may end; a pair that gave up waits for its copies.
      const int left = min(it, kStages);
      for (int i = 0; i < left; ++i) {
        const int j = it - left + i;
        if (ok)
          mbar_wait(&bar.empty[j % kStages], (uint32_t)((j / kStages) & 1), p.err, nullptr);
        else if (rank == 0)
          mbar_wait(&bar.full[j % kStages], (uint32_t)((j / kStages) & 1), p.err, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    // One thread issues them all, so its instructions a step have to take less time than the step's
    // products (512 cycles of a wide tile): descriptors are added to, not formed, and a barrier that has
    // been passed already costs one test (4096 rows on 131072 x 3584: 2295 to 2276 us).
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(kTile, TN, kAmn, kBmn);
      constexpr uint64_t kNextA = (kAmn ? 2048 : 32) >> 4, kNextB = (kBmn ? 2048 : 32) >> 4;  // 16 columns of K on
      const uint64_t a0 = kAmn ? tc::desc_mnmajor(base, 0, kOperand / 2) : tc::desc_kmajor(base, 0);
      const uint64_t b0 =
          kBmn ? tc::desc_mnmajor(base + kOperand, 0, kOperand / 2) : tc::desc_kmajor(base + kOperand, 0);
      const uint32_t full0 = smem_u32(&bar.full[0]), empty0 = smem_u32(&bar.empty[0]);
      uint64_t da = a0, db = b0;
      int s = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += clusters) {
        int k0, k1;
        range(t, k0, k1);
        const int chunk = CHUNKED ? p.chunk : max(1, k1 - k0);
        int c0 = k0;
        do {  // one turn without products where K is empty
          const int buf = n & 1;
          if (n >= 2) ok = mbar_wait(&bar.tile_empty[buf], (uint32_t)((n / 2 - 1) & 1), p.err, abort);
          tc_fence_after();
          const uint32_t d = tmem + buf * kTile;
          uint32_t acc = 0;
          for (int k = (min(k1, c0 + chunk) - c0) * p.passes; ok && k > 0; --k) {
            if (!passed(full0 + 8 * s, phase)) {
              ok = mbar_wait(&bar.full[s], phase, p.err, abort);
              if (!ok) break;
            }
            tc_fence_after();
            mma2(d, da, db, idesc, acc);
            mma2(d, da + kNextA, db + kNextB, idesc, 1);
            mma2(d, da + 2 * kNextA, db + 2 * kNextB, idesc, 1);
            mma2(d, da + 3 * kNextA, db + 3 * kNextB, idesc, 1);
            acc = 1;
            commit2(empty0 + 8 * s);
            da += kStageBytes >> 4;
            db += kStageBytes >> 4;
            if (++s == kStages) {
              s = 0;
              phase ^= 1;
              da = a0;
              db = b0;
            }
          }
          if (ok) commit2(smem_u32(&bar.tile_full[buf]));
          ++n;
          c0 += chunk;
        } while (ok && c0 < k1);
      }
      // every MMA has ended before tensor memory is given back
      commit_own(&bar.done);
      mbar_wait(&bar.done, 0, p.err, nullptr);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int half = (warp - 2) >> 2, r0 = (warp & 3) * 32;
    const uint32_t tcol = tmem + tc::tmem_lane_base(warp) + half * kCols;
    const float inv_cap = p.cap > 0.f ? 1.f / p.cap : 0.f;
    float* turn = reinterpret_cast<float*>(raw + (base - smem_u32(raw)) + kStages * kStageBytes) + (warp - 2) * 32 * 33;
    int n = 0;  // accumulators read
    bool ok = true;
    for (int t = first; t < tiles; t += clusters) {
      int tm, tn, k0, k1;
      place(t % (tms * p.tns), tms, p.tns, p.group, tm, tn);
      range(t, k0, k1);
      const int split = t / (tms * p.tns);
      const int row0 = tm * kTile + (int)rank * kHalf + r0, row = row0 + lane;
      const int col0 = tn * TN + half * kCols;
      // what the row needs, on its way while the product runs
      int target = -1, out_row = 0;
      float lse2 = 0.f, g = 1.f;
      if (MODE != kDw && row < count) {
        out_row = p.rows[row];
        if (MODE == kLse || MODE == kDz) {
          const int64_t tt = p.targets[out_row] - p.v0;
          target = tt >= 0 && tt < p.cols ? (int)tt : -1;
        }
        if (MODE == kDz) {
          lse2 = p.lse[out_row] * tc::kLog2e;
          if (p.d_loss) g = p.d_loss[out_row];
        }
      }
      RowSum sum;

      // what becomes of 32 columns of the row, from col on
      const bool none = MODE == kLse && row0 >= count;  // no row of the warp has a target
      auto finish = [&](float (&z)[32], int col) {
        if (none) return;
        if constexpr (MODE == kLse) {
          if (p.cap > 0.f) cap_logits(z, p.cap, inv_cap);
          // the target's logit is known better (stage_x) and joins the sum there
          if (target >= col && target < col + 32)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (col + i == target) z[i] = -INFINITY;
          sum.add(z, p.cols - col);
          return;
        }
        if constexpr (MODE == kDz) {
          // rows without a target and columns behind the last one are zeros
          const bool live = row < count;
          if (p.cap > 0.f) cap_logits(z, p.cap, inv_cap);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float f = g;
            if (p.cap > 0.f) {
              const float th = z[i] * inv_cap;
              f *= fmaf(-th, th, 1.f);
            }
            float q = ex2_approx(fmaf(z[i], tc::kLog2e, -lse2));
            if (col + i == target) q -= 1.f;
            z[i] = live && col + i < p.cols ? q * f : 0.f;
          }
        }
        // 32 rows of 32 columns, a row a lane, become lines: neighbouring lanes on neighbouring columns
        const int n_rows = min(32, (MODE == kDz ? p.n : MODE == kDx ? count : p.cols) - row0);
        const int n_cols = min(32, (MODE == kDz ? p.pitch : p.out_cols) - col);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) turn[lane * 33 + i] = z[i];
        __syncwarp();
        if (n_rows <= 0 || n_cols <= 0) return;
        // dz of bf16 operands keeps 8 bits, as an operand of the next two products: 0.0017 of its size, which is what the
        // rounding of a bf16 output is too (both: 0.0024).  A second part would double dx = dz W and dw = dz^T X (by their
        // rate, 8192 rows on 131072 x 3584 backward from 13.8 to 21 ms).
        if constexpr (MODE == kDz) {  // (the pitch is a multiple of 64)
          const int c = lane % 4 * 8;
#pragma unroll
          for (int r = lane / 4; r < 32; r += 8) {
            if (r >= n_rows) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = turn[r * 33 + c + e];
#pragma unroll
            for (int part = 0; part < (CHUNKED ? 3 : 1); ++part) {
              if (part > 0 && p.passes == 1) break;
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
                f[2 * e] -= __uint_as_float(w[e] << 16);
                f[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
              }
              store16(p.dz + ((size_t)part * p.n + row0 + r) * p.pitch + col + c, w[0], w[1], w[2], w[3]);
            }
          }
        } else {
          if ((MODE == kDx && p.add) || !last) {
            // sums of the pieces before (kDx), of this split
            const int c = lane % 8 * 4;
#pragma unroll
            for (int r = lane / 8; r < 32; r += 4) {
              if (r >= n_rows || c >= n_cols) break;
              float* acc = p.acc + ((size_t)split * (MODE == kDx ? p.n : p.cols) + row0 + r) * p.acc_pitch + col + c;
              float4 o = MODE == kDx && p.add ? *reinterpret_cast<const float4*>(acc) : make_float4(0.f, 0.f, 0.f, 0.f);
              o.x += turn[r * 33 + c];
              o.y += turn[r * 33 + c + 1];
              o.z += turn[r * 33 + c + 2];
              o.w += turn[r * 33 + c + 3];
              if (!last) {
                *reinterpret_cast<float4*>(acc) = o;
              } else {
                turn[r * 33 + c] = o.x;
                turn[r * 33 + c + 1] = o.y;
                turn[r * 33 + c + 2] = o.z;
                turn[r * 33 + c + 3] = o.w;
              }
            }
            if (!last) return;
            __syncwarp();
          }
          auto place_of = [&](int r) {
            const int to = MODE == kDx ? __shfl_sync(0xffffffffu, out_row, r) : p.v0 + row0 + r;
            return (size_t)to * p.out_cols + col;
          };
          const bool vec = p.out_vec && n_cols == 32;
          if (vec && !p.out_fp32) {
            const int c = lane % 4 * 8;
#pragma unroll
            for (int r = lane / 4; r < 32; r += 8) {
              const size_t at = place_of(r);
              if (r < n_rows) {
                const float* f = turn + r * 33 + c;
                store16(reinterpret_cast<__nv_bfloat16*>(p.out) + at + c, pack_bf16x2(p.scale * f[0], p.scale * f[1]),
                        pack_bf16x2(p.scale * f[2], p.scale * f[3]), pack_bf16x2(p.scale * f[4], p.scale * f[5]),
                        pack_bf16x2(p.scale * f[6], p.scale * f[7]));
              }
            }
          } else if (vec) {
            // rows whose old values are asked for together: one at a time, 790 rows on 57899 x 1664 in bf16 with
            // dw added in fp32 took 732 us backward, so 451 (1666 wide, below: 1518, 657)
            constexpr int B = CHUNKED ? 2 : 8;
            const int c = lane % 8 * 4;
#pragma unroll
            for (int r0 = lane / 8; r0 < 32; r0 += 4 * B) {
              float4 old[B];
#pragma unroll
              for (int u = 0; u < B; ++u) {
                old[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (MODE == kDw && p.accumulate && r0 + 4 * u < n_rows)
                  old[u] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.out) + place_of(r0 + 4 * u) + c);
              }
#pragma unroll
              for (int u = 0; u < B; ++u) {
                const int r = r0 + 4 * u;
                const size_t at = place_of(r);
                if (r >= n_rows) continue;
                const float* f = turn + r * 33 + c;
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at + c) =
                    make_float4(fmaf(p.scale, f[0], old[u].x), fmaf(p.scale, f[1], old[u].y),
                                fmaf(p.scale, f[2], old[u].z), fmaf(p.scale, f[3], old[u].w));
              }
            }
          } else {
            constexpr int B = CHUNKED ? 4 : 16;
            for (int r0 = 0; r0 < n_rows; r0 += B) {
              float old[B];
#pragma unroll
              for (int u = 0; u < B; ++u) {
                const size_t at = place_of(r0 + u) + lane;
                old[u] = 0.f;
                if (MODE == kDw && p.accumulate && p.out_fp32 && r0 + u < n_rows && lane < n_cols)
                  old[u] = reinterpret_cast<const float*>(p.out)[at];
              }
#pragma unroll
              for (int u = 0; u < B; ++u) {
                const size_t at = place_of(r0 + u) + lane;
                if (r0 + u >= n_rows || lane >= n_cols) continue;
                const float f = turn[(r0 + u) * 33 + lane];
                if (p.out_fp32)
                  reinterpret_cast<float*>(p.out)[at] = fmaf(p.scale, f, old[u]);
                else
                  reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(p.scale * f);
              }
            }
          }
        }
      };

      // waits for the next accumulator; 32 columns of it; gives it back
      auto next = [&]() {
        ok = mbar_wait(&bar.tile_full[n & 1], (uint32_t)((n / 2) & 1), p.err, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) tc_fence_after();
        return ok;
      };
      auto give_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bar.tile_empty[n & 1]), 0));
        ++n;
      };
      const bool nothing = k1 <= k0;  // no products: the accumulator holds something else
      if constexpr (CHUNKED) {
        float run[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols; ++c) run[c / 32][c % 32] = 0.f;
        int c0 = k0;
        do {
          if (!next()) break;
          if (!nothing)
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              uint32_t v[16];
              tmem_ld16(tcol + (n & 1) * kTile + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) run[c / 32][c % 32 + i] += __uint_as_float(v[i]);
            }
          give_back();
          c0 += p.chunk;
        } while (c0 < k1);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) finish(run[c], col0 + 32 * c);
      } else {
        if (!next()) break;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld32(tcol + (n & 1) * kTile + c, v);
          tmem_wait_ld();
          if (c == kCols - 32) give_back();
          float(&z)[32] = reinterpret_cast<float(&)[32]>(v);
          if (nothing)
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0.f;
          finish(z, col0 + c);
        }
      }
      __syncwarp();
      if (MODE == kLse && row < count && col0 < p.cols)
        p.part[(size_t)row * p.parts + p.part0 + (col0 / kCols)] = make_float2(sum.m, sum.s);
    }
  }
  // the pair ends together: neither's shared memory or tensor memory goes while the other may use it
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
  cluster_arrive();
  cluster_wait();
}

}  // namespace head
}  // namespace oomb
