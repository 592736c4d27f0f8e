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
// Mapping.  One CTA = one 128-row query tile of one head pair; the two maps
// take the places that two query tiles have in the d = 128 kernel (fwd_tc.cu):
//   * warps 0-3 / 4-7: softmax of map 1 / 2, one thread per query row;
//   * warp 8: TMA producer; a ring stage holds K_1, K_2 (16 KB each) and V
//     (32 KB), so V crosses L2 -> shared memory once for both maps;
//   * warp 9 issues S_1, S_2; warps 10 / 11 issue O_m += P_m V.
// Tensor memory per map (256 columns): S 128 | O 128; P (16 bit) overwrites the
// first 64 columns of S, so the next S of a map waits for its P V.
// Epilogue: warpgroup x forms columns 64 x .. 64 x + 63 of O and O_2 for every
// row from both accumulators (any warp of a lane quarter can read them), after
// the row sums are exchanged through shared memory.
//
// Keys behind seqlens_k[b] may hold anything, NaN included: their scores are
// replaced, and their V rows are zeroed in shared memory before the product
// (0 x NaN would not be 0).
#include "row_softmax.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;
constexpr float kLn2 = 0.6931471805599453f;

struct DCfg {
  static constexpr int NS = 3;                           // K / V stages
  static constexpr int kTB = 16384;                      // one [128 rows][64 columns] box
  static constexpr int kQ = 0;                           // Q_1, Q_2; the O boxes at the end
  static constexpr int kK = 2 * kTB;                     // NS x (K_1, K_2); the O_2 boxes at the end
  static constexpr int kV = kK + NS * 2 * kTB;           // NS x 2 boxes
  static constexpr int kInv = kV + NS * 2 * kTB;         // 2 x 128 floats: 1 / l_m of every row
  static constexpr int kBar = kInv + 1024;
  static constexpr int kBytes = kBar + 512;
};
static_assert(DCfg::kBytes <= 232448, "shared memory over the per-block limit");

struct DBars {
  uint64_t q_full;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t done[3];
  uint64_t k_full[DCfg::NS], v_full[DCfg::NS], k_empty[DCfg::NS], v_empty[DCfg::NS];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DBars) <= 512, "barrier block overflows its shared-memory slot");

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

  // ---- work item: (b, head pair, query tile); heaviest tiles launch first
  const int BH = a.B * a.H;
  const int qt = a.nq - 1 - (int)(blockIdx.x / BH);
  const int bh = (int)(blockIdx.x % BH);
  const int b = bh / a.H, h = bh % a.H;
  const int hk = h / a.group;
  int Lk = a.N;
  if (a.seqlens_k != nullptr) Lk = max(0, min(a.N, a.seqlens_k[b]));
  int lim = (Lk + kTile - 1) / kTile;
  if (a.causal) lim = min(lim, qt + 1);
  const int lo = kWin ? max(0, qt * kTile - a.window + 1) / kTile : 0;
  const int n = max(0, lim - lo);              // key tiles lo .. lo + n - 1

  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[x], 128);
      mbar_init(&bars->pv_done[x], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars->done[i], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_empty[s], 2);
    }
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
  // Register split of the 384 x 168 launch budget, as in fwd_tc.cu:
  // 8 x 32 x 224 + 4 x 32 x 56 = 64512 = 384 x 168.

  if (warp >= 8) {
    regs_dec<56>();
    if (warp == 8) {
      // ===================== TMA producer =====================
      if (lane == 0 && n > 0) {
        mbar_expect_tx(&bars->q_full, 2 * TB);
        tma_load_4d(smem + C::kQ, &tmQ, &bars->q_full, 0, qt * kTile, 2 * h, b);
        tma_load_4d(smem + C::kQ + TB, &tmQ, &bars->q_full, 0, qt * kTile, 2 * h + 1, b);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        bool ok = true;
        for (int s = 0; s < n && ok; ++s) {
          const int st = s % NS;
          const uint32_t ph = (uint32_t)(s / NS) & 1u;
          const int row = (lo + s) * kTile;
          // a stage's first use needs no wait
          if (s >= NS && !(ok = mbar_wait(&bars->k_empty[st], ph ^ 1u, ctl))) break;
          mbar_expect_tx(&bars->k_full[st], 2 * TB);
          tma_load_4d(smem + C::kK + st * 2 * TB, &tmK, &bars->k_full[st], 0, row, 2 * hk, b);
          tma_load_4d(smem + C::kK + st * 2 * TB + TB, &tmK, &bars->k_full[st], 0, row, 2 * hk + 1, b);
          if (s >= NS && !(ok = mbar_wait(&bars->v_empty[st], ph ^ 1u, ctl))) {
            // K of this step is in flight: it lands before the CTA leaves
            mbar_wait(&bars->k_full[st], ph, ctl);
            break;
          }
          mbar_expect_tx(&bars->v_full[st], 2 * TB);
          tma_load_4d(smem + C::kV + st * 2 * TB, &tmV, &bars->v_full[st], 0, row, hk, b);
          tma_load_4d(smem + C::kV + st * 2 * TB + TB, &tmV, &bars->v_full[st], 64, row, hk, b);
        }
        // Before leaving, make sure no load is still writing shared memory.
        for (int j = max(0, n - NS); j < n; ++j) {
          mbar_wait(&bars->k_full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
          mbar_wait(&bars->v_full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
        }
        mbar_wait(&bars->q_full, 0, ctl);
      }
    } else if (warp == 9) {
      // ===================== S issuer (both maps) =====================
      if (lane == 0 && n > 0) {
        constexpr uint32_t idS = idesc_f16(128, 128, ab, 0, 0);
        const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQ), 16, 1024);
        const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kK), 16, 1024);
        bool ok = mbar_wait(&bars->q_full, 0, ctl);
        for (int s = 0; s < n && ok; ++s) {
          const int st = s % NS;
          if (!(ok = mbar_wait(&bars->k_full[st], (uint32_t)(s / NS) & 1u, ctl))) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // S_x(s) overwrites P_x(s-1) once P V_x(s-1) has read it
            if (s > 0 && !(ok = mbar_wait(&bars->pv_done[x], (uint32_t)(s - 1) & 1u, ctl))) break;
            tc_fence_after();
            const uint64_t qd = qd0 + (uint64_t)((x * TB) >> 4);
            const uint64_t kd = kd0 + (uint64_t)(((st * 2 + x) * TB) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + x * 256, qd + (uint64_t)((k * 32) >> 4), kd + (uint64_t)((k * 32) >> 4), idS,
                     k > 0 ? 1u : 0u);
            mma_commit(&bars->s_full[x]);
          }
          if (ok) mma_commit(&bars->k_empty[st]);
        }
        mma_commit(&bars->done[0]);
        mbar_wait(&bars->done[0], 0, ctl);
      }
    } else if (n > 0) {
      // ===================== P V issuer of map x (the whole warp walks the steps) =====================
      const int x = warp - 10;
      constexpr uint32_t idPV = idesc_f16(128, 128, ab, 0, 1);
      const uint64_t vd0 = sdesc_sw128(smem_u32(smem + C::kV), 16384, 1024);
      const uint32_t tP = tmem + x * 256, tO = tmem + x * 256 + 128;
      bool ok = true;
      for (int s = 0; s < n && ok; ++s) {
        const int st = s % NS;
        if (!(ok = warp_wait(&bars->v_full[st], (uint32_t)(s / NS) & 1u, ctl))) break;
        const int live = Lk - (lo + s) * kTile;         // V rows of this tile that count
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
        if (!(ok = warp_wait(&bars->p_full[x], (uint32_t)s & 1u, ctl))) break;
        if (lane == 0) {
          tc_fence_after();
          const uint64_t vd = vd0 + (uint64_t)((st * 2 * TB) >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(tO, tP + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idPV, (s > 0 || k > 0) ? 1u : 0u);
          mma_commit(&bars->pv_done[x]);
          mma_commit(&bars->v_empty[st]);
        }
        __syncwarp();
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
    const int i = qt * kTile + r;               // global query row
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + x * 256 + lane_off, tO = tS + 128;
    const float sl2 = a.scale_log2;
    const int jmax = a.causal ? min(Lk - 1, i) : (Lk - 1);
    const int jmin = kWin ? i - a.window + 1 : 0;

    RowSoftmax w;
    bool ok = true;
    for (int s = 0; s < n; ++s) {
      const int kv = lo + s;
      if (!(ok = warp_wait(&bars->s_full[x], (uint32_t)s & 1u, ctl))) break;
      tc_fence_after();
      w.template step<T, 128, kWin>(tS, tO, jmax - kv * kTile, jmin - kv * kTile, sl2, s == 0);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->p_full[x]);
    }

    // ---- epilogue: O = O_1 / l_1 - lambda O_2 / l_2, columns 64 x .. of both tensors
    float* inv_sh = reinterpret_cast<float*>(smem + C::kInv);
    inv_sh[x * 128 + r] = w.l_rnd > 0.f ? 1.f / w.l_rnd : 0.f;
    // The last product of this warpgroup's own map; the other map may be phases
    // behind, where a parity wait would pass at once, so its end is learned from
    // the barrier both warpgroups meet at.
    bool fin = ok;
    if (ok && n > 0) {
      fin = warp_wait(&bars->pv_done[x], (uint32_t)(n - 1) & 1u, ctl);
      tc_fence_after();
    }
    tc_fence_before();
    if (!named_bar_or(1, 256, !fin || bars->abort)) {
      tc_fence_after();
      const float inv1 = inv_sh[r], inv2 = inv_sh[128 + r];
      const float lam = a.lam[h];
      const bool row_ok = i < a.N;
      const uint32_t t1 = tmem + lane_off + 128 + x * 64, t2 = t1 + 256;
      uint8_t* ob = smem + C::kQ + x * TB;       // Q and K are dead once every product is done
      uint8_t* ob2 = smem + C::kK + x * TB;
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        float o[32], o2[32];
        if (n > 0) {
          uint32_t r1[32], r2[32];
          tmem_ld32(t1 + hf * 32, r1);
          tmem_ld32(t2 + hf * 32, r2);
          tmem_wait_ld();
          reg_fence32(r1);
          reg_fence32(r2);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            o2[c] = __uint_as_float(r2[c]) * inv2;
            o[c] = __uint_as_float(r1[c]) * inv1 - lam * o2[c];
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = o2[c] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t u[4], u2[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            u[t] = Cvt<T>::pack(o[j * 8 + 2 * t], o[j * 8 + 2 * t + 1]);
            u2[t] = Cvt<T>::pack(o2[j * 8 + 2 * t], o2[j * 8 + 2 * t + 1]);
          }
          const uint32_t off = r * 128 + ((((hf * 4 + j) ^ r) & 7) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(smem_u32(ob + off)), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
          if (a.has_o2)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         :: "r"(smem_u32(ob2 + off)), "r"(u2[0]), "r"(u2[1]), "r"(u2[2]), "r"(u2[3]) : "memory");
        }
      }
      fence_proxy_async_smem();
      named_bar_sync(2 + x, 128);
      if (r == 0) {
        tma_store_4d(&tmO, ob, x * 64, qt * kTile, h, b);
        if (a.has_o2) tma_store_4d(&tmO2, ob2, x * 64, qt * kTile, h, b);
        bulk_commit();
        bulk_wait_read0();
      }
      if (row_ok)
        a.lse[((size_t)b * 2 * a.H + 2 * h + x) * a.N + i] = w.l_true > 0.f ? (w.m_run + lg2(w.l_true)) * kLn2 : -INFINITY;
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
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
                     const CUtensorMap& o2, const DiffFwdArgs& a, cudaStream_t s) {
  auto kern = diff_fwd_kernel<T, kWin>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DCfg::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.nq * a.B * a.H), kThreads, DCfg::kBytes, s>>>(q, k, v, o, o2, a);
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
