// prefix_tc.cu -- many query rows against the shared prefix, on the tensor-memory
// products.
//
// Mathematics: prefix.cu.  Here a K/V head's B G T query rows are many, so the
// prefix part is a plain dense attention of R rows against P keys, bound by the
// softmax and the tensor rate rather than HBM.  The register products of
// prefix.cu reach about a quarter of the tcgen05 rate and re-read K and V from
// L2 for every 64 rows.
//
// Mapping, as in the d = 128 forward (fwd_tc.cu): one CTA = 256 rows (two
// 128-row slots) and one key split, every K / V tile loaded once for both slots;
// warps 0-7 softmax (one thread a row), warp 8 TMA, warps 9 and 10 the S products
// and 11 and 12 the P V products of slot 0 and 1 (products of one issuer complete
// one after the other, 8 for each half tile of S at d = 128: one issuer for both
// slots took 39 us where two take 34, 1,024 rows x 32,769 keys x 2 heads, 1.0
// PFLOP/s).  Folded (kFold), the slots have the same rows and a key split each.
// A row's place in q follows from (sequence, head, token), so the softmax threads
// gather their own Q row into the swizzled tile.  Splits are sized so that one
// wave of CTAs covers the GPU; each leaves (max, sums, O unnormalised) in float32
// for the join.  Starting the own keys' kernel or the join beside this one
// (griddepcontrol.launch_dependents) gains nothing: from the first instruction on
// it halves this kernel's speed, from its last tile on it changes no total.
// Tiles are worked in two 64-key halves; row_softmax.cuh says where S, P and O lie.
#include "prefix.cuh"
#include "row_softmax.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;   // warps 0-7 softmax, 8 TMA, 9 / 10 S issuers, 11 / 12 P V issuers, 13-15 idle

template <int D, int DV> struct TCfg {                   // columns of q and k, and of v and o
  static constexpr int kTB = 128 * D * 2;                // one [128 rows][D] tile of Q or K
  static constexpr int kVB = 128 * DV * 2;               // one [128 rows][DV] tile of V
  static constexpr int NS = DV == 64 ? 5 : D == 64 ? 4 : 2;   // K / V stages
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTB;
  static constexpr int kV = kK + NS * kTB;
  static constexpr int kBar = kV + NS * kVB;
  static constexpr int kBytes = kBar + 512;
};
template <int D, int DV> constexpr bool fits() { return TCfg<D, DV>::kBytes <= 232448; }
static_assert(fits<64, 64>() && fits<128, 128>() && fits<64, 128>(), "shared memory over the per-block limit");

struct TBars {
  uint64_t q_full;
  uint64_t s_full[2], s_free[2];                         // [slot]
  uint64_t p_full[2][2], pv_done[2][2];                  // [slot][half]
  uint64_t done[4];
  uint64_t k_full[5], v_full[5], k_empty[5], v_empty[5];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(TBars) <= 512, "barrier block overflows its shared-memory slot");

template <typename T, int D, int DV, bool kFold>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PArgs a) {
  using C = TCfg<D, DV>;
  // stages; folded, the even ones are slot 0's, the odd ones slot 1's
  constexpr int NS = kFold ? C::NS & ~1 : C::NS, TB = C::kTB, VB = C::kVB;
  constexpr bool kDiff = D != DV;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {       // the 128-byte swizzle's tiles: see diff_fwd.cu
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  TBars* bars = reinterpret_cast<TBars*>(smem + C::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item: row tiles of the same keys run together and share them in L2
  const int rts = kFold ? 1 : a.pt, sps = kFold ? (a.np + 1) / 2 : a.np;
  int it = (int)blockIdx.x;
  const int rt = it % rts;
  it /= rts;
  const int sp0 = (kFold ? 2 : 1) * (it % sps);           // split of slot 0
  const int hk = it / sps;
  // slots at work: two that share the keys if there are rows, or two splits of one row tile
  const int nact = (kFold ? sp0 + 1 < a.np : rt * 256 + 128 < a.R) ? 2 : 1;
  auto split = [&](int x) { return kFold ? sp0 + x : sp0; };
  auto tiles = [&](int x) { return (min(a.P, (split(x) + 1) * a.pchunk) - split(x) * a.pchunk + kTile - 1) / kTile; };
  // ring place of tile s of slot x
  auto place = [&](int s, int x) { return kFold ? 2 * s + x : s; };

  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 128 * nact);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->s_free[x], 128);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&bars->p_full[x][j], 128);
        mbar_init(&bars->pv_done[x][j], 1);
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars->done[i], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], kFold ? 1 : nact);
      mbar_init(&bars->v_empty[s], kFold ? 1 : nact);
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
  // Register split of the 512 x 128 launch budget:
  // 8 x 32 x 200 + 8 x 32 x 56 = 65536 = 512 x 128.

  if (warp >= 8) {
    regs_dec<56>();
    if (warp == 8) {
      // ===================== TMA producer =====================
      if (lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        // a tile is four 32-row boxes per 64 columns
        auto load = [&](int base, int boxes, const CUtensorMap* m, uint64_t* bar, int row, int head) {
#pragma unroll
          for (int c = 0; c < boxes; ++c)
#pragma unroll
            for (int x = 0; x < kTile / kKT; ++x)
              tma_load_4d(smem + base + c * 16384 + x * kKT * 128, m, bar, c * 64, row + x * kKT, head, 0);
        };
        bool ok = true;
        const int n = tiles(0);                            // slot 1 has as many or fewer
        int nk[2] = {0, 0}, nv[2] = {0, 0};
        for (int s = 0; s < n && ok; ++s) {
#pragma unroll
          for (int x = 0; x < (kFold ? 2 : 1); ++x) {
            if (x >= nact || s >= tiles(x)) continue;
            const int g = place(s, x), st = g % NS, row = split(x) * a.pchunk + s * kTile;
            const uint32_t ph = (uint32_t)(g / NS) & 1u;
            // a stage's first use needs no wait
            if (g >= NS && !(ok = mbar_wait(&bars->k_empty[st], ph ^ 1u, ctl))) break;
            mbar_expect_tx(&bars->k_full[st], TB);
            load(C::kK + st * TB, D / 64, &tmK, &bars->k_full[st], row, hk);
            ++nk[x];
            if (g >= NS && !(ok = mbar_wait(&bars->v_empty[st], ph ^ 1u, ctl))) break;
            mbar_expect_tx(&bars->v_full[st], VB);
            load(C::kV + st * VB, DV / 64, &tmV, &bars->v_full[st], row, value_head<kDiff>(hk));
            ++nv[x];
          }
        }
        // Before leaving, make sure no load is still writing shared memory.
        constexpr int kOwn = kFold ? NS / 2 : NS;          // stages of a slot
        for (int x = 0; x < (kFold ? 2 : 1); ++x) {
          for (int s = max(0, nk[x] - kOwn); s < nk[x]; ++s)
            mbar_wait(&bars->k_full[place(s, x) % NS], (uint32_t)(place(s, x) / NS) & 1u, ctl);
          for (int s = max(0, nv[x] - kOwn); s < nv[x]; ++s)
            mbar_wait(&bars->v_full[place(s, x) % NS], (uint32_t)(place(s, x) / NS) & 1u, ctl);
        }
      }
    } else if (warp <= 10) {
      // ===================== S issuer of slot x =====================
      const int x = warp - 9;
      if (lane == 0 && x < nact) {
        constexpr uint32_t idS = idesc_f16(128, 64, ab, 0, 0);
        const uint64_t qd0 = sdesc_sw128(smem_u32(smem + C::kQ), 16, 1024);
        const uint64_t kd0 = sdesc_sw128(smem_u32(smem + C::kK), 16, 1024);
        bool ok = mbar_wait(&bars->q_full, 0, ctl);
        const int n = tiles(x);
        for (int s = 0; s < n && ok; ++s) {
          const int g = place(s, x), st = g % NS;
          if (!(ok = mbar_wait(&bars->k_full[st], (uint32_t)(g / NS) & 1u, ctl))) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // S of half h = 2 s + j overwrites that of half h - 1 once the softmax has read it
            if (ok && s + j > 0) ok = mbar_wait(&bars->s_free[x], (uint32_t)(j ^ 1), ctl);
            // and follows the product of half h - 2, so that S(h) tells the softmax P is free as well
            if (ok && s > 0) ok = mbar_wait(&bars->pv_done[x][j], (uint32_t)(s - 1) & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
            const uint64_t qd = qd0 + (uint64_t)((x * TB) >> 4), kd = kd0 + (uint64_t)((st * TB + j * 8192) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t o = (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
              mma_ss(tmem + x * kStream, qd + o, kd + o, idS, k > 0 ? 1u : 0u);
            }
            mma_commit(&bars->s_full[x]);
          }
          if (ok) mma_commit(&bars->k_empty[st]);
        }
        mma_commit(&bars->done[x]);
        mbar_wait(&bars->done[x], 0, ctl);
      }
    } else if (warp <= 12 && warp - 11 < nact) {
      // ===================== P V issuer of slot x =====================
      const int x = warp - 11;
      if (lane == 0) {
        constexpr uint32_t idPV = idesc_f16(128, DV, ab, 0, 1);
        const uint64_t vd0 = sdesc_sw128(smem_u32(smem + C::kV), 16384, 1024);
        const uint32_t tP = tmem + x * kStream + kColP, tO = tmem + x * kStream + kColO;
        bool ok = true;
        const int n = tiles(x);
        for (int s = 0; s < n && ok; ++s) {
          const int g = place(s, x), st = g % NS;
          if (!(ok = mbar_wait(&bars->v_full[st], (uint32_t)(g / NS) & 1u, ctl))) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (ok) ok = mbar_wait(&bars->p_full[x][j], (uint32_t)s & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint64_t)((st * VB + j * 8192) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tO, tP + j * 32 + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idPV, (s > 0 || j > 0 || k > 0) ? 1u : 0u);
            mma_commit(&bars->pv_done[x][j]);
          }
          if (!ok) break;
          mma_commit(&bars->v_empty[st]);
        }
        mma_commit(&bars->done[2 + x]);
        mbar_wait(&bars->done[2 + x], 0, ctl);
      }
    }
  } else {
    regs_inc<200>();
    // ===================== softmax warps =====================
    const int x = warp >> 2;
    if (x < nact) {
      const int quarter = warp & 3;
      const int r = quarter * 32 + lane;          // row within the slot = TMEM lane
      const int row = kFold ? r : rt * 256 + x * 128 + r;
      const int n = tiles(x), k0 = split(x) * a.pchunk;
      const uint32_t tS = tmem + x * kStream + ((uint32_t)(quarter * 32) << 16), tO = tS + kColO;
      // this thread's Q row into the swizzled tile
      {
        uint8_t* qb = smem + C::kQ + x * TB + r * 128;
        const int b = row / a.r, rem = row - b * a.r;
        const int j = rem / a.T, t = rem - j * a.T;
        const uint4* src =
            row < a.R ? reinterpret_cast<const uint4*>(prefix_row<T, kDiff>(a, hk, b, j, t)) : nullptr;
        uint4 v[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) v[c] = src != nullptr ? src[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(qb + (c >> 3) * 16384 + (((c ^ r) & 7) << 4)) = v[c];
        fence_proxy_async_smem();
        mbar_arrive(&bars->q_full);
      }
      RowSoftmax w;
      bool ok = true;
      for (int s = 0; s < n && ok; ++s) {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          if (!(ok = warp_wait(&bars->s_full[x], (uint32_t)j, ctl))) break;      // half h = 2 s + j
          tc_fence_after();
          ok = w.template step<T, DV, false>(
              tS, tS + kColP + j * 32, tO, a.P - 1 - (k0 + s * kTile + j * 64), 0, a.scale_log2, s == 0 && j == 0,
              [&] { mbar_arrive(&bars->s_free[x]); },
              [&]() -> bool {       // the product of half h - 1
                const bool done = warp_wait(&bars->pv_done[x][j ^ 1], (uint32_t)(j ? s : s - 1) & 1u, ctl);
                tc_fence_after();
                return done;
              });
          if (!ok) break;
          mbar_arrive(&bars->p_full[x][j]);
        }
      }
      // ---- this row's maximum, sums and unnormalised O
      if (ok && warp_wait(&bars->pv_done[x][1], (uint32_t)(n - 1) & 1u, ctl)) {
        tc_fence_after();
        const long long pr = ((long long)split(x) * a.Hkv + hk) * a.R + row;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
          reg_fence32(o);
          if (row < a.R) {
            float* dst = a.part + pr * DV + c;           // 32-byte aligned: see launch_prefix
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                           :: "l"(dst + e), "r"(o[e]), "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]),
                              "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7]) : "memory");
          }
        }
        if (row < a.R) a.stat[pr] = make_float4(w.m_run, w.l_true, w.l_rnd, 0.f);
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, int DV, bool kFold>
cudaError_t launch_f(const CUtensorMap& k, const CUtensorMap& v, const PArgs& a, cudaStream_t s) {
  auto kern = prefix_tc_kernel<T, D, DV, kFold>;
  constexpr int bytes = TCfg<D, DV>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.Hkv * (kFold ? (a.np + 1) / 2 : a.pt * a.np)), kThreads, bytes, s>>>(k, v, a);
  return cudaGetLastError();
}

template <typename T, int D, int DV>
cudaError_t launch_t(const CUtensorMap& k, const CUtensorMap& v, const PArgs& a, cudaStream_t s) {
  if constexpr (D == 64) if (a.fold) return launch_f<T, D, DV, true>(k, v, a, s);
  return launch_f<T, D, DV, false>(k, v, a, s);
}

}  // namespace

cudaError_t launch_prefix_tc(int dtype, int d, const CUtensorMap& k, const CUtensorMap& v, const PArgs& a,
                             cudaStream_t s) {
  using B16 = __nv_bfloat16;
  const bool bf = dtype == FA_DT_BF16;
  if (a.lam != nullptr) return bf ? launch_t<B16, 64, 128>(k, v, a, s) : launch_t<__half, 64, 128>(k, v, a, s);
  if (d == 128) return bf ? launch_t<B16, 128, 128>(k, v, a, s) : launch_t<__half, 128, 128>(k, v, a, s);
  return bf ? launch_t<B16, 64, 64>(k, v, a, s) : launch_t<__half, 64, 64>(k, v, a, s);
}

}  // namespace fa
