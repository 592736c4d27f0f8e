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
// What bounds it: the softmax warps (two exponentials a pair against 16 per
// clock and SM) and the latency of the chain S -> softmax -> P V within one
// map; the two maps are independent chains and cover one another.
//
// Mapping.  An item is one 128-row query tile of one head pair; the two maps take
// the places that two query tiles have in the d = 128 kernel (fwd_tc.cu):
//   * warps 0-3 / 4-7: softmax of map 1 / 2, one thread per query row;
//   * warp 8: claims items and streams them with TMA; a ring stage holds K_1, K_2
//     (16 KB each) and V (32 KB), so V crosses L2 -> shared memory once for both
//     maps; Q has two buffers, so the next item's Q, K, V and first scores are
//     under way while this item's epilogue runs;
//   * warp 9 issues S_1, S_2; warps 10 / 11 issue O_m += P_m V.
// Tensor memory per map (256 columns): S 128 | O 128.  There is no room for P
// beside S, so P (16 bit) overwrites S and the next S must wait for the product
// that reads P: with whole 128-key tiles that makes one serial chain S -> softmax
// -> P V per map (324 us at the size below).  The tile is therefore worked in two
// halves of 64 keys with a place each, (S | P over it) 64 columns: while the
// softmax works on one half, the other half's P V and next S run.
// The CTAs are persistent, one on each SM: with one CTA per item the pipeline's
// fill and drain took a third of the time at short causal rows (GPT-2-medium
// width, B = 64, N = 1024: 362 us).
// Epilogue: warpgroup x forms columns 64 x .. 64 x + 63 of O and O_2 for every
// row from both accumulators (any warp of a lane quarter can read them), after
// the row sums are exchanged through shared memory.
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
  static constexpr int kQ = 0;                           // 2 x (Q_1, Q_2)
  static constexpr int kK = 4 * kTB;                     // NS x (K_1, K_2)
  static constexpr int kV = kK + NS * 2 * kTB;           // NS x 2 boxes
  static constexpr int kInv = kV + NS * 2 * kTB;         // 2 x 128 floats: 1 / l_m of every row
  static constexpr int kBar = kInv + 1024;
  static constexpr int kBytes = kBar + 512;
};
static_assert(DCfg::kBytes <= 232448, "shared memory over the per-block limit");

struct DBars {
  uint64_t item_full[2], item_empty[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // [map][half]
  uint64_t done[3];
  uint64_t k_full[DCfg::NS], v_full[DCfg::NS], k_empty[DCfg::NS], v_empty[DCfg::NS];
  uint64_t meet;
  int item[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DBars) <= 512, "barrier block overflows its shared-memory slot");

// Item u: query tile qt of head pair h of batch b, and its key tiles lo .. lo + n - 1.
struct FItem { int b, h, hk, qt, Lk, lo, n; };

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
  return it;
}

// 32 columns of one row: two 32-byte stores where the layout allows them
template <typename T>
__device__ __forceinline__ void store32(T* p, const uint32_t (&w)[16], int v8) {
#pragma unroll
  for (int c = 0; c < 16; c += 8) {
    if (v8) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                   :: "l"(p + 2 * c), "r"(w[c]), "r"(w[c + 1]), "r"(w[c + 2]), "r"(w[c + 3]), "r"(w[c + 4]),
                      "r"(w[c + 5]), "r"(w[c + 6]), "r"(w[c + 7]) : "memory");
    } else {
      reinterpret_cast<uint4*>(p + 2 * c)[0] = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
      reinterpret_cast<uint4*>(p + 2 * c)[1] = make_uint4(w[c + 4], w[c + 5], w[c + 6], w[c + 7]);
    }
  }
}

template <typename T, bool kWin>
__global__ void __launch_bounds__(kThreads, 1)
diff_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const DiffFwdArgs a) {
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->item_full[x], 1);
      mbar_init(&bars->item_empty[x], 11);     // warps 0-7 and 9-11
      mbar_init(&bars->q_full[x], 1);
      mbar_init(&bars->q_empty[x], 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&bars->s_full[x][j], 1);
        mbar_init(&bars->p_full[x][j], 128);
        mbar_init(&bars->pv_done[x][j], 1);
      }
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars->done[i], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_empty[s], 2);
    }
    mbar_init(&bars->meet, 256);
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
  volatile int* item_u = bars->item;
  // the next item's index (all lanes of a warp together), or -1
  int kc = 0;
  auto fetch = [&]() -> int {
    const int slot = kc & 1;
    if (!warp_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl)) return -1;
    const int u = item_u[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    ++kc;
    return u;
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
        int nk = 0, nv = 0, ni = 0;            // K and V stages and Q buffers loaded
        bool ok = true;
        // the first item is the CTA's own index, the others come from the counter
        int u = (int)blockIdx.x;
        for (int kf = 0; ok; ++kf, u = (int)gridDim.x + atomicAdd(a.sched, 1)) {
          const int slot = kf & 1;
          if (kf >= 2 && !(ok = mbar_wait(&bars->item_empty[slot], (uint32_t)((kf >> 1) - 1) & 1u, ctl))) break;
          item_u[slot] = u < total ? u : -1;
          mbar_arrive(&bars->item_full[slot]);
          if (u >= total) break;
          const FItem it = make_item<kWin>(a, u);
          if (it.n == 0) continue;
          const int qb = ni & 1;
          if (ni >= 2 && !(ok = mbar_wait(&bars->q_empty[qb], (uint32_t)((ni >> 1) - 1) & 1u, ctl))) break;
          mbar_expect_tx(&bars->q_full[qb], 2 * TB);
          for (int x = 0; x < 2; ++x)
            tma_load_4d(smem + C::kQ + (qb * 2 + x) * TB, &tmQ, &bars->q_full[qb], 0, it.qt * kTile, 2 * it.h + x, it.b);
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
        for (int j = max(0, ni - 2); j < ni; ++j) mbar_wait(&bars->q_full[j & 1], (uint32_t)(j >> 1) & 1u, ctl);
      }
    } else if (warp == 9) {
      // ===================== S issuer (both maps) =====================
      constexpr uint32_t idS = idesc_f16(128, 64, ab, 0, 0);
      const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQ), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kK), 16, 1024);
      int g = 0, ni = 0;                       // steps, items with steps
      bool ok = true;
      int u;
      while (ok && (u = fetch()) >= 0) {
        const FItem it = make_item<kWin>(a, u);
        if (it.n == 0) continue;
        if (lane == 0) {
          const int qb = ni & 1;
          ok = mbar_wait(&bars->q_full[qb], (uint32_t)(ni >> 1) & 1u, ctl);
          for (int s = 0; s < it.n && ok; ++s, ++g) {
            const int st = g % NS;
            if (!(ok = mbar_wait(&bars->k_full[st], (uint32_t)(g / NS) & 1u, ctl))) break;
#pragma unroll
            for (int jx = 0; jx < 4; ++jx) {
              const int j = jx >> 1, x = jx & 1;       // half by half, map by map
              // S_xj(g) overwrites P_xj(g-1) once its product has read it
              if (ok && g > 0) ok = mbar_wait(&bars->pv_done[x][j], (uint32_t)(g - 1) & 1u, ctl);
              if (!ok) break;
              tc_fence_after();
              const uint64_t qd = qd0 + (uint64_t)(((qb * 2 + x) * TB) >> 4);
              const uint64_t kd = kd0 + (uint64_t)(((st * 2 + x) * TB + j * 8192) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss(tmem + x * 256 + j * 64, qd + (uint64_t)((k * 32) >> 4), kd + (uint64_t)((k * 32) >> 4), idS,
                       k > 0 ? 1u : 0u);
              mma_commit(&bars->s_full[x][j]);
            }
            if (ok) mma_commit(&bars->k_empty[st]);
          }
          if (ok) mma_commit(&bars->q_empty[qb]);
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
      const uint32_t tP = tmem + x * 256, tO = tmem + x * 256 + 128;
      int g = 0;
      bool ok = true;
      int u;
      while (ok && (u = fetch()) >= 0) {
        const FItem it = make_item<kWin>(a, u);
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
            // P_xj(g) follows the softmax warps' reads of the last item's O
            if (ok) ok = warp_wait(&bars->p_full[x][j], (uint32_t)g & 1u, ctl);
            if (!ok) break;
            if (lane == 0) {
              tc_fence_after();
              const uint64_t vd = vd0 + (uint64_t)((st * 2 * TB + j * 8192) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tO, tP + j * 64 + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idPV, (s > 0 || j > 0 || k > 0) ? 1u : 0u);
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
    const uint32_t tS = tmem + x * 256 + lane_off, tO = tS + 128;
    const float sl2 = a.scale_log2;
    float* inv_sh = reinterpret_cast<float*>(smem + C::kInv);
    // barrier of both warpgroups (bounded, so that a warp that gave up leaves none behind)
    GroupSync meet{&bars->meet, 0};
    int g = 0;
    bool ok = true;
    int u;
    while (ok && (u = fetch()) >= 0) {
      const FItem it = make_item<kWin>(a, u);
      const int i = it.qt * kTile + r;          // global query row
      const int jmax = a.causal ? min(it.Lk - 1, i) : (it.Lk - 1);
      const int jmin = kWin ? i - a.window + 1 : 0;
      RowSoftmax w;
      for (int s = 0; s < it.n; ++s, ++g) {
        const int kv = it.lo + s;
#pragma unroll 1
        for (int j = 0; j < 2 && ok; ++j) {
          if (!(ok = warp_wait(&bars->s_full[x][j], (uint32_t)g & 1u, ctl))) break;
          tc_fence_after();
          // the last product into O: the other half's, of this tile or the one before
          auto o_ready = [&]() -> bool {
            const bool done = warp_wait(&bars->pv_done[x][j ^ 1], (uint32_t)(j ? g : g - 1) & 1u, ctl);
            tc_fence_after();
            return done;
          };
          const int key0 = kv * kTile + j * 64;
          if (!(ok = w.template step<T, 64, 128, kWin>(tS + j * 64, tO, jmax - key0, jmin - key0, sl2, s == 0 && j == 0,
                                                       o_ready)))
            break;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[x][j]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- epilogue: O = O_1 / l_1 - lambda O_2 / l_2, columns 64 x .. of both tensors
      const bool row_ok = i < a.N;
      const size_t orow = (size_t)it.b * a.ost.b + (size_t)it.h * a.ost.h + (size_t)i * a.ost.n + x * 64;
      T* op = static_cast<T*>(a.o) + orow;
      T* op2 = static_cast<T*>(a.o2) + orow;
      float inv1 = 0.f, inv2 = 0.f;
      if (it.n > 0) {
        inv_sh[x * 128 + r] = w.l_rnd > 0.f ? 1.f / w.l_rnd : 0.f;
        // The last product of this warpgroup's own map; the other map may be
        // phases behind, where a parity wait would pass at once, so its end is
        // learned from the barrier both warpgroups meet at.
        if (!(ok = warp_wait(&bars->pv_done[x][1], (uint32_t)(g - 1) & 1u, ctl))) break;
        tc_fence_after();
        tc_fence_before();
        if (!(ok = __all_sync(0xffffffffu, meet.sync(ctl)))) break;
        tc_fence_after();
        inv1 = inv_sh[r];
        inv2 = inv_sh[128 + r];
      }
      const float lam = a.lam[it.h];
      const uint32_t t1 = tmem + lane_off + 128 + x * 64, t2 = t1 + 256;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t r1[32], r2[32];
        if (it.n > 0) {
          tmem_ld32(t1 + hf * 32, r1);
          tmem_ld32(t2 + hf * 32, r2);
          tmem_wait_ld();
          reg_fence32(r1);
          reg_fence32(r2);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) r1[c] = r2[c] = 0u;
        }
        uint32_t w1[16], w2[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float a2 = __uint_as_float(r2[2 * c]) * inv2, b2 = __uint_as_float(r2[2 * c + 1]) * inv2;
          w1[c] = Cvt<T>::pack(__uint_as_float(r1[2 * c]) * inv1 - lam * a2,
                               __uint_as_float(r1[2 * c + 1]) * inv1 - lam * b2);
          w2[c] = Cvt<T>::pack(a2, b2);
        }
        if (hf == 1 && it.n > 0) {
          // both accumulators are read: the next item's products may overwrite
          // them once every thread of both warpgroups is here
          tc_fence_before();
          if (!(ok = __all_sync(0xffffffffu, meet.sync(ctl)))) break;
        }
        if (row_ok) {
          store32(op + hf * 32, w1, a.o_v8);
          if (a.o2 != nullptr) store32(op2 + hf * 32, w2, a.o_v8);
        }
      }
      if (!ok) break;
      if (row_ok)
        a.lse[((size_t)it.b * 2 * a.H + 2 * it.h + x) * a.N + i] =
            w.l_true > 0.f ? (w.m_run + lg2(w.l_true)) * kLn2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, bool kWin>
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const DiffFwdArgs& a,
                     cudaStream_t s) {
  auto kern = diff_fwd_kernel<T, kWin>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DCfg::kBytes);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const long long total = (long long)a.nq * a.B * a.H;
  kern<<<(unsigned)std::min<long long>(total, std::max(sms, 1)), kThreads, DCfg::kBytes, s>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_fwd(int dtype, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const DiffFwdArgs& a, cudaStream_t s) {
  if (dtype == FA_DT_BF16)
    return a.window > 0 ? launch_t<__nv_bfloat16, true>(q, k, v, a, s) : launch_t<__nv_bfloat16, false>(q, k, v, a, s);
  return a.window > 0 ? launch_t<__half, true>(q, k, v, a, s) : launch_t<__half, false>(q, k, v, a, s);
}

}  // namespace fa
