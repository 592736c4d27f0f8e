// diff_fwd.cu -- differential attention, forward, 16-bit inputs, sm_103a.
//
// Mathematics.  Head pair h has two score maps over one set of values:
//     P_m = softmax(tau Q_m K_m^T + mask),  m = 1, 2   (64 columns each)
//     O   = (P_1 - lambda_h P_2) V                     (128 columns)
// lambda multiplies the second map only after its normalisation, and neither
// row sum is known before the last key, so the two maps keep their own running
// maximum, sum and unnormalised accumulator O_m = P_m V and meet once, in the
// epilogue: O = O_1 / l_1 - lambda O_2 / l_2.  Saved for the backward pass: the
// two logsumexps and O_2 / l_2 (D_1 and D_2 follow from dO with O and O_2).
//
// Work per visible (query, key) pair: 2 x 128 flops of scores, 2 x 256 of
// P V (512 if the maps could be joined before the product), two exponentials.
// What bounds it: the softmax warps' instructions and the latency of the chain
// S -> softmax -> P V within one map; the two maps are independent chains and
// cover one another.  The exponentials do not: two a pair at the 30 per clock and
// SM that a loop of them reaches are a quarter of the time.
//
// Mapping.  An item is one 128-row query tile of one head pair; the two maps take
// the places that two query tiles have in the d = 128 kernel (fwd_tc.cu):
//   * warps 0-3 / 4-7: softmax of map 1 / 2, one thread per query row;
//   * warp 8: claims items and streams them with TMA; a ring stage holds K_1, K_2
//     (16 KB each) and V (32 KB), so V crosses L2 -> shared memory once for both
//     maps; the next item's Q, K, V and first scores are under way while this
//     item's epilogue runs;
//   * warp 9 issues S_1, S_2; warps 10 / 11 issue O_m += P_m V.
// Key tiles are worked in two halves of 64 keys; row_softmax.cuh says where S, P
// and O lie.  Measured at GPT-2-medium width (B = 64, N = 1024, causal, bf16): one
// CTA per item, whole tiles with P over S (the next S waits for the product that
// reads P) 362 us; persistent CTAs, one on each SM, 324; 64-key halves with P over
// S 292, with P in columns of its own 260 (138 GFLOP under the mask: 529 TFLOP/s;
// tensor pipe a third busy, issue slots 45 %).  P through shared memory
// instead of over S: 312 (the store and its proxy fence cost the softmax warps
// more than the shorter chain gains); an S issuer for each map: 267.
// Epilogue: warpgroup x forms columns 64 x .. 64 x + 63 of O and O_2 for every
// row from both accumulators (any warp of a lane quarter can read them), after
// the row sums are exchanged through shared memory; both leave as TMA stores.
//
// Keys behind seqlens_k[b] may hold anything, NaN included: their scores are
// replaced, and their V rows are zeroed in shared memory before the product
// (0 x NaN would not be 0).
#include <algorithm>

#include "row_softmax.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;
constexpr float kLn2 = 0.6931471805599453f;

struct DCfg {
  static constexpr int NS = 2;                           // K / V stages
  static constexpr int kTB = 16384;                      // one [128 rows][64 columns] box
  static constexpr int kQ = 0;                           // Q_1, Q_2
  static constexpr int kK = 2 * kTB;                     // NS x (K_1, K_2)
  static constexpr int kV = kK + NS * 2 * kTB;           // NS x 2 boxes
  static constexpr int kO = kV + NS * 2 * kTB;           // O's two boxes, then O_2's
  static constexpr int kInv = kO + 4 * kTB;              // 2 x 128 floats: 1 / l_m of every row
  static constexpr int kItem = kInv + 1024;              // the two published items
  static constexpr int kBar = kItem + 64;
  static constexpr int kBytes = kBar + 512;
};
static_assert(DCfg::kBytes <= 232448, "shared memory over the per-block limit");

struct DBars {
  uint64_t item_full[2], item_empty[2];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_free[2];                         // [map]
  uint64_t p_full[2][2], pv_done[2][2];                  // [map][half]
  uint64_t done[3];
  uint64_t k_full[DCfg::NS], v_full[DCfg::NS], k_empty[DCfg::NS], v_empty[DCfg::NS];
  uint64_t meet, meet_x[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DBars) <= 512, "barrier block overflows its shared-memory slot");

// Query tile qt of head pair h of batch b, and its key tiles lo .. lo + n - 1
// (n = -1: no more items).
struct FItem { int b, h, hk, qt, Lk, lo, n; float lam; };
static_assert(sizeof(FItem) == 32, "an item overflows its mailbox slot");

template <bool kWin>
__device__ __forceinline__ FItem make_item(const DiffFwdArgs& a, int u) {
  FItem it;
  const int BH = a.B * a.H;
  const int level = u / BH, bh = u - level * BH;
  it.qt = a.nq - 1 - level;                    // heaviest tiles first
  it.b = bh / a.H;
  it.h = bh - it.b * a.H;
  it.hk = it.h / a.group;
  it.Lk = a.N;
  if (a.seqlens_k != nullptr) it.Lk = max(0, min(a.N, a.seqlens_k[it.b]));
  int lim = (it.Lk + kTile - 1) / kTile;
  if (a.causal) lim = min(lim, it.qt + 1);
  it.lo = kWin ? max(0, it.qt * kTile - a.window + 1) / kTile : 0;
  it.n = max(0, lim - it.lo);
  it.lam = a.lam[it.h];
  return it;
}

template <typename T, bool kWin>
__global__ void __launch_bounds__(kThreads, 1)
diff_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                const __grid_constant__ CUtensorMap tmO2, const DiffFwdArgs a) {
  using C = DCfg;
  constexpr int NS = C::NS;
  constexpr int TB = C::kTB;
  extern __shared__ __align__(1024) uint8_t smem[];
  // The 128-byte swizzle needs 1024-byte aligned tiles: refuse (every thread
  // alike, before any barrier or allocation) if the runtime placed the
  // dynamic shared memory otherwise.
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  DBars* bars = reinterpret_cast<DBars*>(smem + C::kBar);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const int total = a.nq * a.B * a.H;
  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->item_full[x], 1);
      mbar_init(&bars->item_empty[x], 11);     // warps 0-7 and 9-11
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->s_free[x], 128);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&bars->p_full[x][j], 128);
        mbar_init(&bars->pv_done[x][j], 1);
      }
      mbar_init(&bars->meet_x[x], 4);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars->done[i], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_empty[s], 2);
    }
    mbar_init(&bars->meet, 8);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  constexpr int ab = Cvt<T>::kAB;
  // the next item (all lanes of a warp together); n = -1: none left
  int kc = 0;
  auto fetch = [&]() -> FItem {
    const int slot = kc & 1;
    FItem it;
    it.n = -1;
    if (!warp_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl)) return it;
    it = *reinterpret_cast<const FItem*>(smem + C::kItem + slot * 32);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    ++kc;
    return it;
  };
  // Register split of the 384 x 168 launch budget, as in fwd_tc.cu:
  // 8 x 32 x 224 + 4 x 32 x 56 = 64512 = 384 x 168.

  if (warp >= 8) {
    regs_dec<56>();
    if (warp == 8) {
      // ===================== items and TMA =====================
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        int nk = 0, nv = 0, ni = 0;            // K and V stages and Q tiles loaded
        bool ok = true;
        // the first item is the CTA's own index, the others come from the counter
        int u = (int)blockIdx.x;
        for (int kf = 0; ok; ++kf, u = (int)gridDim.x + atomicAdd(a.sched, 1)) {
          const int slot = kf & 1;
          FItem it;
          it.n = -1;
          if (u < total) it = make_item<kWin>(a, u);
          if (kf >= 2 && !(ok = mbar_wait(&bars->item_empty[slot], (uint32_t)((kf >> 1) - 1) & 1u, ctl))) break;
          *reinterpret_cast<FItem*>(smem + C::kItem + slot * 32) = it;
          mbar_arrive(&bars->item_full[slot]);
          if (it.n < 0) break;
          if (it.n == 0) continue;
          if (ni >= 1 && !(ok = mbar_wait(&bars->q_empty, (uint32_t)(ni - 1) & 1u, ctl))) break;
          mbar_expect_tx(&bars->q_full, 2 * TB);
          for (int x = 0; x < 2; ++x)
            tma_load_4d(smem + C::kQ + x * TB, &tmQ, &bars->q_full, 0, it.qt * kTile, 2 * it.h + x, it.b);
          ++ni;
          for (int s = 0; s < it.n; ++s) {
            const int st = nk % NS;
            const uint32_t ph = (uint32_t)(nk / NS) & 1u;
            const int row = (it.lo + s) * kTile;
            // a stage's first use needs no wait
            if (nk >= NS && !(ok = mbar_wait(&bars->k_empty[st], ph ^ 1u, ctl))) break;
            mbar_expect_tx(&bars->k_full[st], 2 * TB);
            for (int x = 0; x < 2; ++x)
              tma_load_4d(smem + C::kK + (st * 2 + x) * TB, &tmK, &bars->k_full[st], 0, row, 2 * it.hk + x, it.b);
            ++nk;
            if (nv >= NS && !(ok = mbar_wait(&bars->v_empty[st], ph ^ 1u, ctl))) break;
            mbar_expect_tx(&bars->v_full[st], 2 * TB);
            for (int x = 0; x < 2; ++x)
              tma_load_4d(smem + C::kV + (st * 2 + x) * TB, &tmV, &bars->v_full[st], 64 * x, row, it.hk, it.b);
            ++nv;
          }
        }
        // Before leaving, make sure no load is still writing shared memory.
        for (int j = max(0, nk - NS); j < nk; ++j) mbar_wait(&bars->k_full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
        for (int j = max(0, nv - NS); j < nv; ++j) mbar_wait(&bars->v_full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
        if (ni > 0) mbar_wait(&bars->q_full, (uint32_t)(ni - 1) & 1u, ctl);
      }
    } else if (warp == 9) {
      // ===================== S issuer (both maps) =====================
      constexpr uint32_t idS = idesc_f16(128, 64, ab, 0, 0);
      const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQ), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kK), 16, 1024);
      int g = 0, ni = 0;                       // steps, items with steps
      bool ok = true;
      while (ok) {
        const FItem it = fetch();
        if (it.n < 0) break;
        if (it.n == 0) continue;
        if (lane == 0) {
          ok = mbar_wait(&bars->q_full, (uint32_t)ni & 1u, ctl);
          for (int s = 0; s < it.n && ok; ++s, ++g) {
            const int st = g % NS;
            if (!(ok = mbar_wait(&bars->k_full[st], (uint32_t)(g / NS) & 1u, ctl))) break;
#pragma unroll
            for (int jx = 0; jx < 4; ++jx) {
              const int j = jx >> 1, x = jx & 1;       // half by half, map by map
              // S of half h = 2 g + j overwrites that of half h - 1 once the softmax has read it
              if (ok && g + j > 0) ok = mbar_wait(&bars->s_free[x], (uint32_t)(j ^ 1), ctl);
              // and follows the product of half h - 2, so that S(h) tells the softmax P is free as well
              if (ok && g > 0) ok = mbar_wait(&bars->pv_done[x][j], (uint32_t)(g - 1) & 1u, ctl);
              if (!ok) break;
              tc_fence_after();
              const uint64_t qd = qd0 + (uint64_t)((x * TB) >> 4);
              const uint64_t kd = kd0 + (uint64_t)(((st * 2 + x) * TB + j * 8192) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss(tmem + x * kStream, qd + (uint64_t)((k * 32) >> 4), kd + (uint64_t)((k * 32) >> 4), idS,
                       k > 0 ? 1u : 0u);
              mma_commit(&bars->s_full[x]);
            }
            if (ok) mma_commit(&bars->k_empty[st]);
          }
          if (ok) mma_commit(&bars->q_empty);
        }
        ++ni;
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0) {
        mma_commit(&bars->done[0]);
        mbar_wait(&bars->done[0], 0, ctl);
      }
    } else {
      // ===================== P V issuer of map x (the whole warp walks the steps) =====================
      const int x = warp - 10;
      constexpr uint32_t idPV = idesc_f16(128, 128, ab, 0, 1);
      const uint64_t vd0 = sdesc_sw128(smem_u32(smem + C::kV), 16384, 1024);
      const uint32_t tP = tmem + x * kStream + kColP, tO = tmem + x * kStream + kColO;
      int g = 0;
      bool ok = true;
      while (ok) {
        const FItem it = fetch();
        if (it.n < 0) break;
        for (int s = 0; s < it.n && ok; ++s, ++g) {
          const int st = g % NS;
          if (!(ok = warp_wait(&bars->v_full[st], (uint32_t)(g / NS) & 1u, ctl))) break;
          const int live = it.Lk - (it.lo + s) * kTile;         // V rows of this tile that count
          if (live < kTile) {
            // both maps' issuers write the same zeros, each before its own product
            uint8_t* vb = smem + C::kV + st * 2 * TB;
            for (int o = live * 128 + lane * 16; o < TB; o += 512) {
              *reinterpret_cast<uint4*>(vb + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(vb + TB + o) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // P follows the softmax warps' reads of the last item's O
            if (ok) ok = warp_wait(&bars->p_full[x][j], (uint32_t)g & 1u, ctl);
            if (!ok) break;
            if (lane == 0) {
              tc_fence_after();
              const uint64_t vd = vd0 + (uint64_t)((st * 2 * TB + j * 8192) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tO, tP + j * 32 + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idPV, (s > 0 || j > 0 || k > 0) ? 1u : 0u);
              mma_commit(&bars->pv_done[x][j]);
              if (j == 1) mma_commit(&bars->v_empty[st]);
            }
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        mma_commit(&bars->done[1 + x]);
        mbar_wait(&bars->done[1 + x], 0, ctl);
      }
    }
  } else {
    regs_inc<224>();
    // ===================== softmax warps =====================
    const int x = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;          // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + x * kStream + lane_off, tO = tS + kColO;
    const float sl2 = a.scale_log2;
    float* inv_sh = reinterpret_cast<float*>(smem + C::kInv);
    uint8_t* ob = smem + C::kO + x * TB;        // columns 64 x .. of O
    uint8_t* ob2 = ob + 2 * TB;                 // and of O_2
    WarpMeet meet{&bars->meet, 0}, meet_x{&bars->meet_x[x], 0};
    int g = 0;
    bool ok = true;
    while (ok) {
      const FItem it = fetch();
      if (it.n < 0) break;
      const int i = it.qt * kTile + r;          // global query row
      const int jmax = a.causal ? min(it.Lk - 1, i) : (it.Lk - 1);
      const int jmin = kWin ? i - a.window + 1 : 0;
      RowSoftmax w;
      for (int s = 0; s < it.n && ok; ++s, ++g) {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          if (!(ok = warp_wait(&bars->s_full[x], (uint32_t)j, ctl))) break;      // half h = 2 g + j
          tc_fence_after();
          const int key0 = (it.lo + s) * kTile + j * 64;
          ok = w.template step<T, 128, kWin>(
              tS, tS + kColP + j * 32, tO, jmax - key0, jmin - key0, sl2, s == 0 && j == 0,
              [&] { mbar_arrive(&bars->s_free[x]); },
              [&]() -> bool {       // the product of half h - 1
                const bool done = warp_wait(&bars->pv_done[x][j ^ 1], (uint32_t)(j ? g : g - 1) & 1u, ctl);
                tc_fence_after();
                return done;
              });
          if (!ok) break;
          mbar_arrive(&bars->p_full[x][j]);
        }
      }
      if (!ok) break;
      // ---- epilogue: O = O_1 / l_1 - lambda O_2 / l_2, columns 64 x .. of both tensors
      uint32_t r1[2][32], r2[2][32];
      float inv1 = 0.f, inv2 = 0.f;
      if (it.n > 0) {
        inv_sh[x * 128 + r] = w.l_rnd > 0.f ? 1.f / w.l_rnd : 0.f;
        // The last product of this warpgroup's own map; the other map may be
        // phases behind, where a parity wait would pass at once, so its end is
        // learned from the barrier both warpgroups meet at.
        if (!(ok = warp_wait(&bars->pv_done[x][1], (uint32_t)(g - 1) & 1u, ctl))) break;
        tc_fence_after();
        tc_fence_before();
        if (!(ok = meet.sync(ctl))) break;
        tc_fence_after();
        inv1 = inv_sh[r];
        inv2 = inv_sh[128 + r];
        const uint32_t t1 = tmem + lane_off + kColO + x * 64, t2 = t1 + kStream;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          tmem_ld32(t1 + hf * 32, r1[hf]);
          tmem_ld32(t2 + hf * 32, r2[hf]);
        }
        tmem_wait_ld();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          reg_fence32(r1[hf]);
          reg_fence32(r2[hf]);
        }
        // both accumulators are read: the next item's products may overwrite
        // them once both warpgroups are here
        tc_fence_before();
        if (!(ok = meet.sync(ctl))) break;
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) r1[c >> 5][c & 31] = r2[c >> 5][c & 31] = 0u;
      }
      // the last item's stores have read the staging boxes
      if (r == 0) bulk_wait_read0();
      if (!(ok = meet_x.sync(ctl))) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t u1[4], u2[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int c = 8 * j + 2 * t;
          const float a2 = __uint_as_float(r2[c >> 5][c & 31]) * inv2, b2 = __uint_as_float(r2[c >> 5][(c & 31) + 1]) * inv2;
          u1[t] = Cvt<T>::pack(__uint_as_float(r1[c >> 5][c & 31]) * inv1 - it.lam * a2,
                               __uint_as_float(r1[c >> 5][(c & 31) + 1]) * inv1 - it.lam * b2);
          u2[t] = Cvt<T>::pack(a2, b2);
        }
        const uint32_t off = r * 128 + (((j ^ r) & 7) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(smem_u32(ob + off)), "r"(u1[0]), "r"(u1[1]), "r"(u1[2]), "r"(u1[3]) : "memory");
        if (a.has_o2)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(smem_u32(ob2 + off)), "r"(u2[0]), "r"(u2[1]), "r"(u2[2]), "r"(u2[3]) : "memory");
      }
      fence_proxy_async_smem();
      if (!(ok = meet_x.sync(ctl))) break;
      if (r == 0) {
        tma_store_4d(&tmO, ob, x * 64, it.qt * kTile, it.h, it.b);
        if (a.has_o2) tma_store_4d(&tmO2, ob2, x * 64, it.qt * kTile, it.h, it.b);
        bulk_commit();
      }
      if (i < a.N)
        a.lse[((size_t)it.b * 2 * a.H + 2 * it.h + x) * a.N + i] =
            w.l_true > 0.f ? (w.m_run + lg2(w.l_true)) * kLn2 : -INFINITY;
    }
    if (r == 0) bulk_wait_read0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, bool kWin>
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
                     const CUtensorMap& o2, const DiffFwdArgs& a, cudaStream_t s) {
  auto kern = diff_fwd_kernel<T, kWin>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DCfg::kBytes);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const long long total = (long long)a.nq * a.B * a.H;
  kern<<<(unsigned)std::min<long long>(total, std::max(sms, 1)), kThreads, DCfg::kBytes, s>>>(q, k, v, o, o2, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_fwd(int dtype, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& o, const CUtensorMap& o2, const DiffFwdArgs& a, cudaStream_t s) {
  if (dtype == FA_DT_BF16)
    return a.window > 0 ? launch_t<__nv_bfloat16, true>(q, k, v, o, o2, a, s)
                        : launch_t<__nv_bfloat16, false>(q, k, v, o, o2, a, s);
  return a.window > 0 ? launch_t<__half, true>(q, k, v, o, o2, a, s) : launch_t<__half, false>(q, k, v, o, o2, a, s);
}

}  // namespace fa
