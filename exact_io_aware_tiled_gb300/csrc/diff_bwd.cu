// diff_bwd.cu -- differential attention, backward, 16-bit inputs, sm_103a.
//
// Mathematics (O = (P_1 - lambda P_2) V, P_m rebuilt from Q_m, K_m and the saved
// logsumexps).  Both maps meet the same dP, because they share V and dO:
//     dP   = dO V^T,   D_m = rowsum(P_m o dP) = dO . O_m
//     dS_1 = P_1 o (dP - D_1),   dS_2 = -lambda P_2 o (dP - D_2)
//     dV   = (P_1 - lambda P_2)^T dO     one product for both maps
//     dQ_m = tau dS_m K_m,   dK_m = tau dS_m^T Q_m,   dlambda = -sum P_2 o dP
// Per visible pair: 2 x 128 flops of scores, 256 each of dP, dV, dQ and dK
// (1280 in all) and two exponentials.  Two separate backward passes at d = 128
// (Q, K padded) would do 2560.  dlambda is summed from the float32 P_2 and dP,
// not from rounded outputs: it is a long sum of both signs.
//
// Roundings: P_1 - lambda P_2, dS_1 and dS_2 become 16-bit operands of the products
// that take them, half a step of each element; dQ, dK and dV are rounded once at
// the end (0.0024 relative in bf16, both together).  P, dP, D and all sums are float32.
//
// Tiles: 128 keys x 64 query rows a step, keys on the tensor-memory lanes, as in
// the d = 128 backward (bwd_tc128.cu), whose roles and barriers this kernel
// keeps, except that dQ goes from registers into the float32 accumulator by
// 128-byte-per-warp adds instead of through a staging tile and a TMA reduce: the
// 32 KB that frees hold a second pair of K tiles, so an item's first scores do
// not wait for the last item's products.  Tensor memory (512 columns):
//   S_1^T 0-63 | S_2^T 64-127 | dP^T 128-191 | dQ^T 192-255 | dK_1, dK_2 256-383 | dV 384-511
// W^T = (P_1 - lambda P_2)^T, the 16-bit operand of dV, lies over S_1^T (the 16
// queries of warpgroup w in the first 8 of its own 16 columns), so S_1 of the
// next step waits for dV; S_2 is issued before it and covers the wait.
//
// dQ^T has 64 rows (head dims) per map, half of what the tensor core's M = 128
// takes.  Both maps share one accumulator: lanes 0-63 hold dQ_1^T, 64-127
// dQ_2^T.  The A operand of map 1 is (K_1 | Z) and of map 2 (Z | K_2), Z a tile
// of zeros that lies between K_1 and K_2 in shared memory, so each product adds
// zeros to the other map's half.  That doubles this product's multiplies (+20 %
// of the total) and keeps everything within 512 columns and one drain.
//
// What bounds it: the chain S -> P -> dS -> dQ of a step and the compute warps'
// instructions (two exponentials and two dS per pair), not the tensor core.
// Measured at GPT-2-medium width (B = 64, N = 1024, causal, bf16): 574 us, 344
// GFLOP under the mask: 599 TFLOP/s; tensor pipe 29 %, issue slots 36 %.
// dQ by a separate drain warpgroup 655-830 us (its registers come from the compute
// warps); dQ loaded before this step's dS is published, so that the next product
// starts earlier, 702; dS in two buffers against one pair of K tiles 631; sleeping
// waits in the compute warps 591.
//
// Keys behind seqlens_k[b] may hold anything: their P and dP are replaced, and
// their K rows are zeroed in shared memory before dQ reads them.
#include <algorithm>
#include <type_traits>

#include "register_mma.cuh"

namespace fa {
namespace {

constexpr int kThreads = 640;
constexpr int kCompute = 512;   // threads of warps 0-15
constexpr int kQS = 64;         // query rows per step
constexpr int NQ = 2;           // Q / dO stages
constexpr float kLog2e = 1.4426950408889634f;

struct DSmem {
  // K_1 of two items | zeros | K_2 of two items, 16 KB each
  static constexpr int kK1 = 0, kZ = 32768, kK2 = 49152;
  static constexpr int kV = 81920;                  // 32 KB: V [2 boxes][128 keys][64]
  static constexpr int kQ = kV + 32768;             // NQ x (Q_1, Q_2: 8 KB each)
  static constexpr int kDO = kQ + NQ * 16384;       // NQ x 16 KB: dO [2 boxes][64 q][64]
  static constexpr int kDS = kDO + NQ * 16384;      // dS_1^T, dS_2^T [128 keys][64 q], 16 KB each
  static constexpr int kLD = kDS + 32768;           // NQ x 4 x 64 floats: -LSE_1, -LSE_2, e_1, e_2
  static constexpr int kItem = kLD + NQ * 1024;     // the two published work items
  static constexpr int kBar = kItem + 64;
  static constexpr int kBytes = kBar + 320;
  static constexpr int kDyn = kBytes + 1024;
};
static_assert(DSmem::kDyn <= 232448, "shared memory over the per-block limit");

struct DBars {
  uint64_t item_full[2], item_empty[2];
  uint64_t k_full[2], k_empty[2], v_full, v_empty;
  uint64_t q_full[NQ], q_empty[NQ];
  uint64_t s_full, p_full, dp_full, ds_full, dq_full, dq_free, dkv_full, pt_free;
  uint64_t dsm_free;
  uint64_t done[3];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DBars) <= 320, "barrier block overflows its shared-memory slot");

constexpr uint32_t kColS1 = 0, kColS2 = 64, kColDP = 128, kColDQ = 192, kColDK = 256, kColDV = 384;

// One work item: key tile jt of K/V pair hk of batch b, and its steps: the two
// 64-row halves of every query tile that sees the key tile, for each of the
// group's query head pairs.
struct DItem {
  int b, hk, jt, Lk;
  int n;                  // query tiles per query head pair
  int i0;                 // first query tile
  int h0;                 // first query head pair of the group
  int steps;              // 64-row steps
};

__device__ __forceinline__ DItem make_item(const DiffBwdArgs& a, int u) {
  DItem it;
  const int bk = u / a.nq;
  it.jt = u - bk * a.nq;
  it.b = bk / a.H_kv;
  it.hk = bk - it.b * a.H_kv;
  it.Lk = a.N;
  if (a.seqlens_k != nullptr) it.Lk = max(0, min(a.N, a.seqlens_k[it.b]));
  it.i0 = a.causal ? it.jt : 0;
  it.h0 = it.hk * a.group;
  int qlast = a.nq - 1;
  // under a window of w keys, key j is seen by queries j .. j + w - 1 (the sum in 64 bits: w may be any int)
  if (a.window > 0) qlast = (int)min((long long)qlast, ((long long)it.jt * kTile + kTile - 1 + a.window - 1) / kTile);
  it.n = it.jt * kTile < it.Lk ? max(0, qlast - it.i0 + 1) : 0;
  it.steps = 2 * it.n * a.group;
  return it;
}

struct StepPos {
  int qu = 0, hq = 0, hf = 0;
  __device__ __forceinline__ void next(const DItem& it) {
    if (++hf == 2) {
      hf = 0;
      if (++qu == it.n) { qu = 0; ++hq; }
    }
  }
};

template <typename T, bool kWin>
__global__ void __launch_bounds__(kThreads, 1)
diff_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                const DiffBwdArgs a) {
  using L = DSmem;
  // bf16: tau is folded into dS, so dQ and dK leave the tensor core scaled; not
  // for fp16, whose smaller range would push small dS values into subnormals.
  constexpr bool kFold = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DBars* bars = reinterpret_cast<DBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int total = a.nq * a.B * a.H_kv;
  WaitCtl ctl{a.status, &bars->abort};

  // the zero tile between K_1 and K_2
  for (int o = threadIdx.x * 16; o < 16384; o += kThreads * 16)
    *reinterpret_cast<uint4*>(smem + L::kZ + o) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 3 + kCompute);   // warps 17-19 and the compute threads
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 2);  // the S^T and the dQ^T products read K
    }
    mbar_init(&bars->v_full, 1);
    mbar_init(&bars->v_empty, 1);       // the dP^T products read V
    for (int s = 0; s < NQ; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->p_full, kCompute);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->ds_full, kCompute);
    mbar_init(&bars->dq_full, 1);
    mbar_init(&bars->dq_free, kCompute);
    mbar_init(&bars->dkv_full, 1);
    mbar_init(&bars->pt_free, 1);
    mbar_init(&bars->dsm_free, 2);     // dK and dQ^T both read the shared dS^T tiles
    for (int i = 0; i < 3; ++i) mbar_init(&bars->done[i], 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // the kernels before are done (the launch overlaps the end of the last of them)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp >= 16) {
    constexpr int ab = Cvt<T>::kAB;
    constexpr uint32_t idST = idesc_f16(128, 64, ab, 0, 0);    // S^T, dP^T (both operands K-major)
    constexpr uint32_t idV = idesc_f16(128, 128, ab, 0, 1);    // dV (A in tensor memory, B MN-major)
    constexpr uint32_t idK = idesc_f16(128, 64, ab, 0, 1);     // dK_m (A K-major, B MN-major)
    constexpr uint32_t idQ = idesc_f16(128, 64, ab, 1, 1);     // dQ^T (A = (K_1 | Z)^T or (Z | K_2)^T, B = dS^T, MN-major)
    const uint32_t sK1 = smem_u32(smem + L::kK1), sZ = smem_u32(smem + L::kZ), sK2 = smem_u32(smem + L::kK2);
    const uint32_t sV = smem_u32(smem + L::kV);
    const uint32_t sQ = smem_u32(smem + L::kQ), sDO = smem_u32(smem + L::kDO);
    const uint32_t sDS = smem_u32(smem + L::kDS);
    volatile int* item_u = reinterpret_cast<volatile int*>(smem + L::kItem);
    int kc = 0;
    auto fetch = [&]() -> int {
      const int slot = kc & 1;
      if (!mbar_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl)) return -1;
      const int v = item_u[slot];
      mbar_arrive(&bars->item_empty[slot]);
      ++kc;
      return v;
    };
    if (warp == 16) {
      // ===================== items and TMA =====================
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmDO);
        int g = 0, nkv = 0;
        bool ok = true;
        int kf = 0;
        auto publish = [&]() -> int {
          const int slot = kf & 1;
          if (!mbar_wait(&bars->item_empty[slot], ((uint32_t)(kf >> 1) & 1u) ^ 1u, ctl)) return -2;
          int v = atomicAdd(a.sched, 1);
          if (v >= total) v = -1;
          item_u[slot] = v;
          mbar_arrive(&bars->item_full[slot]);
          ++kf;
          return v;
        };
        int nv = 0;                       // V loads issued
        while (ok) {
          const int u = publish();
          if (u < 0) break;
          const DItem it = make_item(a, u);
          if (it.steps == 0) continue;
          // K: two buffers, so the next item's K lands while this item's last products run
          const int kb = nkv & 1;
          if (!(ok = mbar_wait(&bars->k_empty[kb], ((uint32_t)(nkv >> 1) & 1u) ^ 1u, ctl))) break;
          mbar_expect_tx(&bars->k_full[kb], 32768);
          tma_load_4d(smem + L::kK1 + kb * 16384, &tmK, &bars->k_full[kb], 0, it.jt * kTile, 2 * it.hk, it.b);
          tma_load_4d(smem + L::kK2 + kb * 16384, &tmK, &bars->k_full[kb], 0, it.jt * kTile, 2 * it.hk + 1, it.b);
          ++nkv;
          StepPos sp;
          sp.hq = it.h0;
          for (int t = 0; t < it.steps; ++t, sp.next(it)) {
            const int st = g % NQ;
            if (!(ok = mbar_wait(&bars->q_empty[st], ((uint32_t)(g / NQ) & 1u) ^ 1u, ctl))) break;
            const int q0 = (it.i0 + sp.qu) * kTile + sp.hf * kQS;
            const size_t ld_row = (((size_t)it.b * a.H + sp.hq) * a.npad + (size_t)q0) * 4;
            mbar_expect_tx(&bars->q_full[st], 32768 + 1024);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tma_load_4d(smem + L::kQ + st * 16384 + c * 8192, &tmQ, &bars->q_full[st], 0, q0, 2 * sp.hq + c, it.b);
              tma_load_4d(smem + L::kDO + st * 16384 + c * 8192, &tmDO, &bars->q_full[st], c * 64, q0, sp.hq, it.b);
            }
            bulk_load(smem + L::kLD + st * 1024, a.rows + ld_row, 1024, &bars->q_full[st]);
            ++g;
            if (t == 0) {
              // V: one buffer, free once the last item's dP^T products are done
              if (!(ok = mbar_wait(&bars->v_empty, ((uint32_t)nv & 1u) ^ 1u, ctl))) break;
              mbar_expect_tx(&bars->v_full, 32768);
#pragma unroll
              for (int c = 0; c < 2; ++c)
                tma_load_4d(smem + L::kV + c * 16384, &tmV, &bars->v_full, c * 64, it.jt * kTile, it.hk, it.b);
              ++nv;
            }
          }
        }
        // before leaving, make sure no load is still writing shared memory
        for (int t = max(0, g - NQ); t < g; ++t) mbar_wait(&bars->q_full[t % NQ], (uint32_t)(t / NQ) & 1u, ctl);
        for (int t = max(0, nkv - 2); t < nkv; ++t) mbar_wait(&bars->k_full[t & 1], (uint32_t)(t >> 1) & 1u, ctl);
        if (nv > 0) mbar_wait(&bars->v_full, (uint32_t)(nv - 1) & 1u, ctl);
      }
    } else if (warp == 17) {
      // ===================== S^T / dP^T issuer =====================
      if (lane == 0) {
        int g = 0, nkv = 0;
        bool ok = true;
        int u;
        while (ok && (u = fetch()) >= 0) {
          const DItem it = make_item(a, u);
          if (it.steps == 0) continue;
          const int kb = nkv & 1;
          if (!(ok = mbar_wait(&bars->k_full[kb], (uint32_t)(nkv >> 1) & 1u, ctl))) break;
          for (int t = 0; t < it.steps && ok; ++t, ++g) {
            const int st = g % NQ;
            // S_2^T(g) once part 1 of step g-1 has read S_2^T(g-1); S_1^T(g) also
            // once dV(g-1) has read W^T(g-1), which lies over S_1^T(g-1)
            if (g > 0 && !(ok = mbar_wait(&bars->p_full, (uint32_t)(g - 1) & 1u, ctl))) break;
            if (!(ok = mbar_wait(&bars->q_full[st], (uint32_t)(g / NQ) & 1u, ctl))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + kColS2, sdesc_sw128(sK2 + kb * 16384 + k * 32, 16, 1024),
                     sdesc_sw128(sQ + st * 16384 + 8192 + k * 32, 16, 1024), idST, k > 0 ? 1u : 0u);
            if (g > 0 && !(ok = mbar_wait(&bars->pt_free, (uint32_t)(g - 1) & 1u, ctl))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + kColS1, sdesc_sw128(sK1 + kb * 16384 + k * 32, 16, 1024),
                     sdesc_sw128(sQ + st * 16384 + k * 32, 16, 1024), idST, k > 0 ? 1u : 0u);
            mma_commit(&bars->s_full);
            if (t == it.steps - 1) mma_commit(&bars->k_empty[kb]);   // this item's S^T are done with K
            // dP^T(g) = V dO_g^T once part 2 of step g-1 has read dP^T(g-1)
            if (g > 0 && !(ok = mbar_wait(&bars->ds_full, (uint32_t)(g - 1) & 1u, ctl))) break;
            if (t == 0 && !(ok = mbar_wait(&bars->v_full, (uint32_t)nkv & 1u, ctl))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ss(tmem + kColDP, sdesc_sw128(sV + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024),
                     sdesc_sw128(sDO + st * 16384 + (k >> 2) * 8192 + (k & 3) * 32, 16, 1024), idST, k > 0 ? 1u : 0u);
            mma_commit(&bars->dp_full);
          }
          mma_commit(&bars->v_empty);     // this item's dP^T are done with V
          ++nkv;
        }
        mma_commit(&bars->done[0]);
        mbar_wait(&bars->done[0], 0, ctl);
      }
    } else if (warp == 18) {
      // ===================== dV / dK issuer =====================
      if (lane == 0) {
        int g = 0;
        bool ok = true;
        int u;
        while (ok && (u = fetch()) >= 0) {
          const DItem it = make_item(a, u);
          if (it.steps == 0) continue;
          for (int t = 0; t < it.steps && ok; ++t, ++g) {
            const int st = g % NQ;
            const uint32_t qb = sQ + st * 16384, db = sDO + st * 16384;
            // dV += W^T dO_g: A = W^T (16 queries per 16 columns of S_1's place), B = dO MN-major
            if (!(ok = mbar_wait(&bars->p_full, (uint32_t)g & 1u, ctl) &&
                       mbar_wait(&bars->q_full[st], (uint32_t)(g / NQ) & 1u, ctl))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + kColDV, tmem + kColS1 + k * 16, sdesc_sw128(db + k * 2048, 8192, 1024), idV,
                     (t > 0 || k > 0) ? 1u : 0u);
            mma_commit(&bars->pt_free);
            // dK_m += dS_m^T Q_m: A = dS^T K-major (32 bytes per 16 queries), B = Q MN-major
            if (!(ok = mbar_wait(&bars->ds_full, (uint32_t)g & 1u, ctl))) break;
            tc_fence_after();
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss(tmem + kColDK + m * 64, sdesc_sw128(sDS + m * 16384 + k * 32, 16, 1024),
                       sdesc_sw128(qb + m * 8192 + k * 2048, 8192, 1024), idK, (t > 0 || k > 0) ? 1u : 0u);
            mma_commit(&bars->dsm_free);
            mma_commit(&bars->q_empty[st]);
          }
          mma_commit(&bars->dkv_full);
        }
        mma_commit(&bars->done[1]);
        mbar_wait(&bars->done[1], 0, ctl);
      }
    } else {
      // ===================== dQ^T issuer (warp 19, all lanes) =====================
      int g = 0, nkv = 0;
      bool ok = true;
      while (ok) {
        const int slot = kc & 1;
        if (!(ok = warp_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl))) break;
        const int u = item_u[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
        ++kc;
        if (u < 0) break;
        const DItem it = make_item(a, u);
        if (it.steps == 0) continue;
        const int kb = nkv & 1;
        const int live = it.Lk - it.jt * kTile;       // K rows of this tile that count
        if (live < kTile) {
          if (!(ok = warp_wait(&bars->k_full[kb], (uint32_t)(nkv >> 1) & 1u, ctl))) break;
          for (int o = live * 128 + lane * 16; o < 16384; o += 512) {
            *reinterpret_cast<uint4*>(smem + L::kK1 + kb * 16384 + o) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + L::kK2 + kb * 16384 + o) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ++nkv;
        for (int t = 0; t < it.steps && ok; ++t, ++g) {
          if (!(ok = warp_wait(&bars->ds_full, (uint32_t)g & 1u, ctl))) break;
          if (g > 0 && !(ok = warp_wait(&bars->dq_free, (uint32_t)(g - 1) & 1u, ctl))) break;
          if (lane == 0) {
            tc_fence_after();
            // the second 64 rows of A lie one leading offset behind the first: zeros
            // behind K_1, K_2 behind the zeros
            const uint32_t a1 = sK1 + kb * 16384, a2 = sK2 + kb * 16384;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ss(tmem + kColDQ, sdesc_sw128(a1 + k * 2048, sZ - a1, 1024), sdesc_sw128(sDS + k * 2048, 8192, 1024), idQ,
                     k > 0 ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ss(tmem + kColDQ, sdesc_sw128(sZ + k * 2048, a2 - sZ, 1024),
                     sdesc_sw128(sDS + 16384 + k * 2048, 8192, 1024), idQ, 1u);
            mma_commit(&bars->dq_full);
            mma_commit(&bars->dsm_free);
          }
          __syncwarp();
        }
        if (lane == 0) mma_commit(&bars->k_empty[kb]);   // this item's dQ^T products are done with K
        __syncwarp();
      }
      if (lane == 0) {
        mma_commit(&bars->done[2]);
        mbar_wait(&bars->done[2], 0, ctl);
      }
    }
  } else {
    // ===================== softmax-gradient warpgroups =====================
    const int wg = warp >> 2;                 // query columns 16 wg .. 16 wg + 15 of the step
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;        // key row, or (dQ^T) map r / 64 and head dim r % 64 = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tl = tmem + lane_off;
    const float sl2 = a.scale_log2;
    const float c1 = kFold ? a.scale : 1.f;
    const int c0 = wg * 16;                   // first query column of this warpgroup
    bool ok = true;

    // dQ_t: row r of the stacked dQ^T, this warpgroup's 16 queries -> x tau (fp16)
    // -> added to the float32 accumulator.  A warp's 32 lanes are 32 consecutive
    // head dims of one query, so every add instruction is one 128-byte line.
    // (qn: rows of the step that exist, counted from this warpgroup's first.)
    auto drain_dq = [&](int t, float* dst, int qn) -> bool {
      if (!warp_wait(&bars->dq_full, (uint32_t)t & 1u, ctl)) return false;
      tc_fence_after();
      uint32_t g[16];
      tmem_ld16(tl + kColDQ + c0, g);
      tmem_wait_ld();
      reg_fence16(g);
      tc_fence_before();
      mbar_arrive(&bars->dq_free);
      auto add = [&](int c) {
        const float v = kFold ? __uint_as_float(g[c]) : __uint_as_float(g[c]) * a.scale;
        asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" :: "l"(dst + c * 64), "f"(v) : "memory");
      };
      if (qn >= 16) {
#pragma unroll
        for (int c = 0; c < 16; ++c) add(c);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c < qn) add(c);
      }
      return true;
    };
    // this thread's place in the accumulator for the step whose dQ is drained next
    float* dq_dst = nullptr;
    int dq_n = 0;

    // dK (x tau for fp16) and dV of an item: columns 32 wg .. 32 wg + 31 of the
    // stacked (dK_1 | dK_2) row and of the dV row, in two halves of 16
    auto store_dkv = [&](const DItem& it, int half, const uint32_t (&kraw)[16], const uint32_t (&vraw)[16],
                         bool have) {
      const int j = it.jt * kTile + r;
      if (j >= a.N) return;
      const size_t koff = (size_t)it.b * a.kst.b + (size_t)(2 * it.hk + (wg >> 1)) * a.kst.h + (size_t)j * a.kst.n +
                          (wg & 1) * 32 + half * 16;
      const size_t voff =
          (size_t)it.b * a.vst.b + (size_t)it.hk * a.vst.h + (size_t)j * a.vst.n + wg * 32 + half * 16;
      uint32_t wk[8], wv[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float ks = kFold ? 1.f : a.scale;   // bf16: dK is already scaled
        wk[c] = Cvt<T>::pack(have ? __uint_as_float(kraw[2 * c]) * ks : 0.f,
                             have ? __uint_as_float(kraw[2 * c + 1]) * ks : 0.f);
        wv[c] = Cvt<T>::pack(have ? __uint_as_float(vraw[2 * c]) : 0.f, have ? __uint_as_float(vraw[2 * c + 1]) : 0.f);
      }
      if (a.dkv_v8) {
        // one 32-byte store per tensor: whole sectors in one instruction
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(static_cast<T*>(a.dk) + koff), "r"(wk[0]), "r"(wk[1]), "r"(wk[2]), "r"(wk[3]),
                        "r"(wk[4]), "r"(wk[5]), "r"(wk[6]), "r"(wk[7]) : "memory");
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(static_cast<T*>(a.dv) + voff), "r"(wv[0]), "r"(wv[1]), "r"(wv[2]), "r"(wv[3]),
                        "r"(wv[4]), "r"(wv[5]), "r"(wv[6]), "r"(wv[7]) : "memory");
        return;
      }
      uint4* dk = reinterpret_cast<uint4*>(static_cast<T*>(a.dk) + koff);
      uint4* dv = reinterpret_cast<uint4*>(static_cast<T*>(a.dv) + voff);
      dk[0] = make_uint4(wk[0], wk[1], wk[2], wk[3]);
      dk[1] = make_uint4(wk[4], wk[5], wk[6], wk[7]);
      dv[0] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
      dv[1] = make_uint4(wv[4], wv[5], wv[6], wv[7]);
    };

    volatile int* item_u = reinterpret_cast<volatile int*>(smem + L::kItem);
    int kc = 0;
    auto fetch = [&]() -> int {
      const int slot = kc & 1;
      if (!warp_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl)) return -1;
      const int v = item_u[slot];
      mbar_arrive(&bars->item_empty[slot]);
      ++kc;
      return v;
    };
    int t = 0;        // global step
    int nit = 0;      // items with steps (dkv_full phases)
    int u;
    while (ok && (u = fetch()) >= 0) {
      const DItem it = make_item(a, u);
      float* part = a.dlam_part + (size_t)u * a.group * 16 + warp;
      if (it.steps == 0) {            // no query tile sees this key tile: dK = dV = 0, nothing for dlambda
        const uint32_t zero[16] = {};
        store_dkv(it, 0, zero, zero, false);
        store_dkv(it, 1, zero, zero, false);
        for (int g = lane; g < a.group; g += 32) part[g * 16] = 0.f;
        continue;
      }
      const int j = it.jt * kTile + r;          // global key
      const bool key_ok = j < it.Lk;
      StepPos sp;
      sp.hq = it.h0;
      float lam = a.lam[it.h0];
      float dl0 = 0.f, dl1 = 0.f;               // sum of P_2 o dP of this thread, current head pair
      for (int tt = 0; tt < it.steps && ok; ++tt, ++t, sp.next(it)) {
        const int st = t % NQ;
        const int q0 = (it.i0 + sp.qu) * kTile + sp.hf * kQS;   // first query row of the step
        const uint32_t s_ld = smem_u32(smem + L::kLD + st * 1024) + c0 * 4;
        // query column c of the step is hidden from this key under causal iff
        // c < qlo, and outside its sliding window iff c >= qhe
        const int qlo = a.causal ? (j - q0) : -1;
        const int qhe = kWin ? (int)min((long long)j + a.window - q0, (long long)kQS) : kQS;
        const bool any_mask = !key_ok || qlo > c0 || (kWin && qhe < c0 + 16);

        // ---- part 1: P_1, P_2 (float32, kept) and W = P_1 - lambda P_2
        if (!(ok = warp_wait(&bars->s_full, (uint32_t)t & 1u, ctl) &&
                   warp_wait(&bars->q_full[st], (uint32_t)(t / NQ) & 1u, ctl))) break;
        tc_fence_after();
        uint32_t s1[16], s2[16];
        tmem_ld16(tl + kColS1 + c0, s1);
        tmem_ld16(tl + kColS2 + c0, s2);
        tmem_wait_ld();
        reg_fence16(s1);
        reg_fence16(s2);
        float p1[16], p2[16];
        uint32_t w[8];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int cc = q4 * 4;
          const float4 l1 = lds128(s_ld + cc * 4), l2 = lds128(s_ld + 256 + cc * 4);
          fma2(p1[cc], p1[cc + 1], __uint_as_float(s1[cc]), __uint_as_float(s1[cc + 1]), sl2, sl2, l1.x, l1.y);
          fma2(p1[cc + 2], p1[cc + 3], __uint_as_float(s1[cc + 2]), __uint_as_float(s1[cc + 3]), sl2, sl2, l1.z, l1.w);
          fma2(p2[cc], p2[cc + 1], __uint_as_float(s2[cc]), __uint_as_float(s2[cc + 1]), sl2, sl2, l2.x, l2.y);
          fma2(p2[cc + 2], p2[cc + 3], __uint_as_float(s2[cc + 2]), __uint_as_float(s2[cc + 3]), sl2, sl2, l2.z, l2.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p1[cc + e] = ex2(p1[cc + e]);
            p2[cc + e] = ex2(p2[cc + e]);
          }
          if (any_mask) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!key_ok || c0 + cc + e < qlo || (kWin && c0 + cc + e >= qhe)) p1[cc + e] = p2[cc + e] = 0.f;
          }
          float w0, w1, w2, w3;
          fma2(w0, w1, p2[cc], p2[cc + 1], -lam, -lam, p1[cc], p1[cc + 1]);
          fma2(w2, w3, p2[cc + 2], p2[cc + 3], -lam, -lam, p1[cc + 2], p1[cc + 3]);
          w[q4 * 2] = Cvt<T>::pack(w0, w1);
          w[q4 * 2 + 1] = Cvt<T>::pack(w2, w3);
        }
        // over this warpgroup's own columns of S_1^T, which are in registers
        tmem_st8(tl + kColS1 + c0, w);
        if (!(ok = warp_wait(&bars->dp_full, (uint32_t)t & 1u, ctl))) break;
        tc_fence_after();
        uint32_t dp[16];
        tmem_ld16(tl + kColDP + c0, dp);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full);

        // ---- part 2: dS_1, dS_2 from dP^T into the shared tiles once dK and
        //      dQ^T of the previous step have read them
        if (t >= 1 && !(ok = warp_wait(&bars->dsm_free, (uint32_t)(t - 1) & 1u, ctl))) break;
        tmem_wait_ld();
        reg_fence16(dp);
        if (!key_ok) {          // V behind the sequence may hold NaN
#pragma unroll
          for (int c = 0; c < 16; ++c) dp[c] = 0u;
        }
        const float c2 = -lam * c1;
        uint32_t d1w[8], d2w[8];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int cc = q4 * 4;
          // e_1 = -c_1 D_1, e_2 = -c_2 D_2
          const float4 e1 = lds128(s_ld + 512 + cc * 4), e2 = lds128(s_ld + 768 + cc * 4);
          const float g0 = __uint_as_float(dp[cc]), g1 = __uint_as_float(dp[cc + 1]);
          const float g2 = __uint_as_float(dp[cc + 2]), g3 = __uint_as_float(dp[cc + 3]);
          fma2(dl0, dl1, p2[cc], p2[cc + 1], g0, g1, dl0, dl1);
          fma2(dl0, dl1, p2[cc + 2], p2[cc + 3], g2, g3, dl0, dl1);
          float y0, y1, y2, y3;
          fma2(y0, y1, g0, g1, c1, c1, e1.x, e1.y);
          fma2(y2, y3, g2, g3, c1, c1, e1.z, e1.w);
          mul2(y0, y1, y0, y1, p1[cc], p1[cc + 1]);
          mul2(y2, y3, y2, y3, p1[cc + 2], p1[cc + 3]);
          d1w[q4 * 2] = Cvt<T>::pack(y0, y1);
          d1w[q4 * 2 + 1] = Cvt<T>::pack(y2, y3);
          fma2(y0, y1, g0, g1, c2, c2, e2.x, e2.y);
          fma2(y2, y3, g2, g3, c2, c2, e2.z, e2.w);
          mul2(y0, y1, y0, y1, p2[cc], p2[cc + 1]);
          mul2(y2, y3, y2, y3, p2[cc + 2], p2[cc + 3]);
          d2w[q4 * 2] = Cvt<T>::pack(y0, y1);
          d2w[q4 * 2 + 1] = Cvt<T>::pack(y2, y3);
        }
        // this warpgroup's 16 queries are the 16-byte pieces 2 wg, 2 wg + 1 of the key's 128-byte rows
        const uint32_t dsb = smem_u32(smem + L::kDS + r * 128);
#pragma unroll
        for (int pc2 = 0; pc2 < 2; ++pc2) {
          const uint32_t off = ((((2 * wg + pc2) ^ r) & 7) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(dsb + off), "r"(d1w[pc2 * 4]), "r"(d1w[pc2 * 4 + 1]), "r"(d1w[pc2 * 4 + 2]),
                          "r"(d1w[pc2 * 4 + 3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(dsb + 16384 + off), "r"(d2w[pc2 * 4]), "r"(d2w[pc2 * 4 + 1]), "r"(d2w[pc2 * 4 + 2]),
                          "r"(d2w[pc2 * 4 + 3]) : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);

        // ---- the head pair's last step of this item: its part of dlambda
        if (sp.hf == 1 && sp.qu == it.n - 1) {
          float s = dl0 + dl1;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) part[(sp.hq - it.h0) * 16] = s;
          dl0 = dl1 = 0.f;
          if (tt + 1 < it.steps) lam = a.lam[sp.hq + 1];
        }
        // ---- drain dQ of the previous step
        if (t > 0 && !(ok = drain_dq(t - 1, dq_dst, dq_n))) break;
        dq_dst = a.dqacc + (((size_t)it.b * 2 * a.H + 2 * sp.hq + (r >> 6)) * a.N + q0 + c0) * 64 + (r & 63);
        dq_n = a.N - q0 - c0;
      }
      if (!ok) break;
      // ---- item end: dK, dV out of tensor memory (the next item's first dV /
      //      dK follow this thread's next p_full / ds_full arrivals)
      if (!(ok = warp_wait(&bars->dkv_full, (uint32_t)nit & 1u, ctl))) break;
      ++nit;
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t kraw[16], vraw[16];
        tmem_ld16(tl + kColDK + wg * 32 + half * 16, kraw);
        tmem_ld16(tl + kColDV + wg * 32 + half * 16, vraw);
        tmem_wait_ld();
        reg_fence16(kraw);
        reg_fence16(vraw);
        store_dkv(it, half, kraw, vraw, true);
      }
      tc_fence_before();
    }
    if (ok && t > 0) ok = drain_dq(t - 1, dq_dst, dq_n);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// D_1 and D_2 of every query row from dO . O and dO . O_2 (D_1 = dO . O +
// lambda D_2; diff_d1_kernel replaces it where lambda is large), the logsumexps in log2 units, all in the 64-row groups that a
// step loads in one piece; the dQ accumulator is cleared on the way.  Eight
// threads a row, 16 columns each.  Bound by HBM: three 256-byte rows read, two
// 256-byte accumulator rows written.
template <typename T>
__global__ void diff_prep_kernel(const T* __restrict__ o, const T* __restrict__ o2, Strides ost,
                                 const T* __restrict__ dout, Strides dst, const float* __restrict__ lse,
                                 const float* __restrict__ lam, int H, int N, int npad, long long total, float c1,
                                 float* __restrict__ rows, float* __restrict__ dqacc, int* __restrict__ sched) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *sched = 0;   // work counter of the main kernel
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 3;
  const int part = threadIdx.x & 7;
  const bool live = row < total;
  const long long bh = live ? row / npad : 0;
  const int i = live ? (int)(row - bh * npad) : N;
  const int b = (int)(bh / H), h = (int)(bh % H);
  float d = 0.f, d2 = 0.f;
  if (live && i < N) {
    const size_t oo = (size_t)b * ost.b + (size_t)h * ost.h + (size_t)i * ost.n;
    const size_t od = (size_t)b * dst.b + (size_t)h * dst.h + (size_t)i * dst.n;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int c = part * 8 + m * 64;
      const uint4 uo = *reinterpret_cast<const uint4*>(o + oo + c), u2 = *reinterpret_cast<const uint4*>(o2 + oo + c);
      const uint4 ud = *reinterpret_cast<const uint4*>(dout + od + c);
      const uint32_t wo[4] = {uo.x, uo.y, uo.z, uo.w}, w2[4] = {u2.x, u2.y, u2.z, u2.w}, wd[4] = {ud.x, ud.y, ud.z, ud.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float g0 = Cvt<T>::lo(wd[t]), g1 = Cvt<T>::hi(wd[t]);
        d += g0 * Cvt<T>::lo(wo[t]) + g1 * Cvt<T>::hi(wo[t]);
        d2 += g0 * Cvt<T>::lo(w2[t]) + g1 * Cvt<T>::hi(w2[t]);
      }
      // heads 2h, 2h + 1 of the accumulator [B,2H,N,64]: this thread's 8 columns of map m
      float4* z = reinterpret_cast<float4*>(dqacc + (((size_t)bh * 2 + m) * N + i) * 64 + part * 8);
      z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    d += __shfl_xor_sync(0xffffffffu, d, s);
    d2 += __shfl_xor_sync(0xffffffffu, d2, s);
  }
  if (live && part < 4) {
    // part 0, 1: -LSE of map 1, 2 in log2 units (P = exp2(S tau log2e - LSE) is one
    // packed FMA, which cannot negate an operand); part 2, 3: e_1 = -c_1 D_1, e_2 = lambda c_1 D_2
    float v;
    if (part < 2) {
      v = -INFINITY;                 // a row without keys, or past N: P = 0
      if (i < N) {
        const float l = lse[((size_t)bh * 2 + part) * N + i];
        if (l != -INFINITY) v = -l * kLog2e;
      }
    } else {
      const float lm = lam[h];
      v = i >= N ? 0.f : part == 2 ? -c1 * (d + lm * d2) : lm * c1 * d2;
    }
    rows[((size_t)row >> 6) * 256 + part * 64 + (row & 63)] = v;
  }
}

// D_1 of the head pairs with |lambda| > kD1Direct, from the products themselves:
//     D_1 = rowsum(P_1 o dP),  P_1 = exp(tau Q_1 K_1^T - LSE_1),  dP = dO V^T,
// all in float32, over the prepass's dO . O + lambda dO . O_2.  There the rounding
// of O and lambda times that of O_2 stay when lambda dO . O_2 cancels, so the
// error of D_1, and of dQ_1 and dK_1, grows with |lambda| while their values do
// not.  Relative error of dQ_1 (bf16, N = 257, causal, normal inputs) with the
// prepass's D_1: lambda 0.5 0.0025, 1 0.0026, 2 0.0031, 4 0.0050, 8 0.010, 30 0.038,
// 100 0.129; with this one 0.0024 throughout, the rounding of dS and of dQ.  So the
// prepass's is kept up to 2.
//
// A CTA takes 64 query rows, 16 a warp, against 64-key tiles of K_1 and V that
// it loads ahead: 384 flops a pair on the register products.  Issue slots (51 %)
// and the products' latency (tensor pipe 35 %) bound it.  The head pairs above the
// limit are gathered first, so that all of them share one order of items, long
// rows first (head after head, the same CTAs had the long rows of each: 630 us
// for 517, 318 for 138 at B = 16).  At GPT-2-medium width (B = 64, N = 1024, causal,
// bf16) 1.9 us where no head pair is above the limit, 80 with one of the eight,
// 517 with all (199 TFLOP/s under the mask; the main kernel takes 574).  This kernel
// and the main one are launched over the end of the one before, which hides the
// 1.9 us: a training step takes 1,011 us as it did without (1,016 launched plainly;
// B = 32, N = 509, fp16, padded: 214 for 216, 220 launched plainly).
constexpr float kD1Direct = 2.f;
constexpr int kD1Threads = 128;
constexpr int kD1Stage = 8192 + 16384;           // K_1 [64 keys][64], V [2 boxes][64 keys][64]

struct D1Args {
  const void *q, *k, *v, *dout;
  Strides qs, ks, vs, ds;
  const float *lse, *lam;
  const int32_t* seqlens_k;
  int B, H, group, N, npad, causal, window;
  float sl2, c1;
  float* rows;
};

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kD1Threads, 3) diff_d1_kernel(const D1Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ uint32_t masks[kD1Threads / 32];
  __shared__ int heads[kD1Threads];
  const int tiles = (a.N + 63) / 64;
#pragma unroll 1
  for (int h0 = 0; h0 < a.H; h0 += kD1Threads) {
    // those of 128 head pairs that are above the limit, in order
    const bool large = h0 + tid < a.H && fabsf(a.lam[h0 + tid]) > kD1Direct;
    const uint32_t mask = __ballot_sync(0xffffffffu, large);
    if (lane == 0) masks[warp] = mask;
    __syncthreads();
    int nh = 0, before = __popc(mask & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kD1Threads / 32; ++w) {
      nh += __popc(masks[w]);
      if (w < warp) before += __popc(masks[w]);
    }
    if (large) heads[before] = h0 + tid;
    __syncthreads();
    // the prepass has written its rows (the launch overlaps its end)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int wide = a.B * nh;                                   // B H < 2^31
#pragma unroll 1
    for (long long u = blockIdx.x; u < (long long)wide * tiles; u += gridDim.x) {
      const int level = (int)(u / wide), bh = (int)(u - (long long)level * wide);
      const int b = bh / nh, h = heads[bh - b * nh], hk = h / a.group;
      const int i0 = (tiles - 1 - level) * 64;                   // long rows first
      int Lk = a.N;
      if (a.seqlens_k != nullptr) Lk = max(0, min(a.N, a.seqlens_k[b]));
      const int hi = a.causal ? min(Lk, i0 + 64) : Lk;
      const int lo = a.window > 0 ? max(0, i0 - a.window + 1) / 64 * 64 : 0;
      const int n = hi > lo ? (hi - lo + 63) / 64 : 0;
      const T* kb = static_cast<const T*>(a.k) + (int64_t)b * a.ks.b + (int64_t)(2 * hk) * a.ks.h;
      const T* vb = static_cast<const T*>(a.v) + (int64_t)b * a.vs.b + (int64_t)hk * a.vs.h;
      auto load = [&](int t) {
        const uint32_t s = smem_u32(smem + (t & 1) * kD1Stage);
        for (int e = tid; e < 64 * 24; e += kD1Threads) {        // 8 pieces of K_1, 16 of V a key
          const int r = e / 24, c = e - r * 24, j = lo + t * 64 + r;
          const bool live = j < Lk;                              // rows past it may hold anything, or nothing
          const int64_t jj = live ? j : 0;
          const T* src = c < 8 ? kb + jj * a.ks.n + c * 8 : vb + jj * a.vs.n + (c - 8) * 8;
          copy16(s + (c >> 3) * 8192 + sw128_off(r, (c & 7) * 8), src, live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (n > 0) load(0);
      // this thread's two rows of Q_1 and dO, as operands
      uint32_t q[4][4], g[8][4];
      float nl[2], d[2] = {0.f, 0.f};
      const int i = i0 + warp * 16 + (lane >> 2);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int ix = i + 8 * x;
        const bool live = ix < a.N;
        const int64_t in = live ? ix : 0;
        const T* qr = static_cast<const T*>(a.q) + (int64_t)b * a.qs.b + (int64_t)(2 * h) * a.qs.h + in * a.qs.n + 2 * (lane & 3);
        const T* dr = static_cast<const T*>(a.dout) + (int64_t)b * a.ds.b + (int64_t)h * a.ds.h + in * a.ds.n + 2 * (lane & 3);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k][2 * c + x] = live ? *reinterpret_cast<const uint32_t*>(qr + k * 16 + c * 8) : 0u;
#pragma unroll
          for (int k = 0; k < 8; ++k) g[k][2 * c + x] = live ? *reinterpret_cast<const uint32_t*>(dr + k * 16 + c * 8) : 0u;
        }
        nl[x] = live ? -a.lse[((int64_t)b * 2 * a.H + 2 * h) * a.N + in] * kLog2e : 0.f;
      }
      const int lr = lane & 7, lm = lane >> 3;
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        if (t + 1 < n) {
          load(t + 1);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const uint32_t sK = smem_u32(smem + (t & 1) * kD1Stage), sV = sK + 8192;
        const int j0 = lo + t * 64;
#pragma unroll
        for (int m = 0; m < 4; ++m) {                            // 16 keys
          float s[2][4] = {}, dp[2][4] = {};
          // matrices: keys 0-7 / 8-15 (lm >> 1), columns 0-7 / 8-15 (lm & 1)
          const uint32_t row = m * 16 + (lm >> 1) * 8 + lr;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
            ldsm4(w, sK + sw128_off(row, k * 16 + (lm & 1) * 8));
            mma16816<T>(s[0], q[k], w[0], w[1]);
            mma16816<T>(s[1], q[k], w[2], w[3]);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t w[4];
            ldsm4(w, sV + (k >> 2) * 8192 + sw128_off(row, (k & 3) * 16 + (lm & 1) * 8));
            mma16816<T>(dp[0], g[k], w[0], w[1]);
            mma16816<T>(dp[1], g[k], w[2], w[3]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ix = i + 8 * (e >> 1), j = j0 + m * 16 + y * 8 + 2 * (lane & 3) + (e & 1);
              const bool see = j < hi && (!a.causal || j <= ix) && (a.window == 0 || j > ix - a.window);
              const float p = ex2(s[y][e] * a.sl2 + nl[e >> 1]);
              d[e >> 1] += see ? p * dp[y][e] : 0.f;
            }
        }
        __syncthreads();                                         // the tile has been read
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        d[x] += __shfl_xor_sync(0xffffffffu, d[x], 1);
        d[x] += __shfl_xor_sync(0xffffffffu, d[x], 2);
        const int ix = i + 8 * x;
        if ((lane & 3) == 0 && ix < a.N) {
          const long long r = ((long long)b * a.H + h) * a.npad + ix;
          a.rows[(r >> 6) * 256 + 128 + (r & 63)] = -a.c1 * d[x];
        }
      }
    }
  }
}

// dlambda of head pair blockIdx.x: every item's and warp's part, in a fixed order.
// Bound by the latency of its loads: 1,024 threads take an item's 16 sums in four
// 16-byte pieces.
__global__ void __launch_bounds__(1024) diff_dlam_kernel(const float* __restrict__ part, float* __restrict__ dlam, int B,
                                                         int H, int group, int nq) {
  __shared__ float sh[1024];
  const int h = blockIdx.x, hk = h / group, j = h - hk * group, hkv = H / group;
  const int n = B * nq;                       // items of this head pair's K/V pair (total items fit an int)
  float s = 0.f;
#pragma unroll 4
  for (int e = threadIdx.x; e < 4 * n; e += 1024) {
    const int it = e >> 2;
    const int b = it / nq, jt = it - b * nq;
    const float4 v = *reinterpret_cast<const float4*>(
        part + ((((size_t)b * hkv + hk) * nq + jt) * group + j) * 16 + (e & 3) * 4);
    s += (v.x + v.y) + (v.z + v.w);
  }
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int o = 512; o > 0; o >>= 1) {
    if (threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) dlam[h] = -sh[0];
}

// A launch that may begin while the kernel before it in the stream ends: the kernel
// waits (griddepcontrol.wait) before it touches what that one wrote.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                              const A&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, args...);
}

template <typename T, bool kWin>
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dout,
                     const DiffBwdArgs& a, cudaStream_t s) {
  auto kern = diff_bwd_kernel<T, kWin>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DSmem::kDyn);
  if (e != cudaSuccess) return e;
  const long long total = (long long)a.nq * a.B * a.H_kv;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<long long>(total, (long long)std::max(sms, 1));
  return launch_overlapped(kern, grid, kThreads, DSmem::kDyn, s, q, k, v, dout, a);
}

template <typename T>
cudaError_t prep_t(const void* o, const void* o2, Strides ost, const void* dout, Strides dst, const float* lse,
                   const float* lam, int B, int H, int N, int npad, float c1, float* rows, float* dqacc, int* sched,
                   cudaStream_t s) {
  const long long total = (long long)B * H * npad;
  const unsigned grid = (unsigned)((total * 8 + 255) / 256);
  diff_prep_kernel<T><<<grid, 256, 0, s>>>(static_cast<const T*>(o), static_cast<const T*>(o2), ost,
                                           static_cast<const T*>(dout), dst, lse, lam, H, N, npad, total, c1, rows,
                                           dqacc, sched);
  return cudaGetLastError();
}

template <typename T>
cudaError_t d1_t(const D1Args& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaFuncSetAttribute(diff_d1_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kD1Stage);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long most = (long long)a.B * a.H * ((a.N + 63) / 64);
  return launch_overlapped(diff_d1_kernel<T>, (unsigned)std::min<long long>(most, 3ll * std::max(sms, 1)), kD1Threads,
                           2 * kD1Stage, s, a);
}

}  // namespace

cudaError_t launch_diff_d1(int dtype, const void* q, const void* k, const void* v, const void* dout, Strides qst,
                           Strides dst, float c1, const float* lse, const DiffBwdArgs& m, cudaStream_t s) {
  D1Args a{};
  a.q = q; a.k = k; a.v = v; a.dout = dout;
  a.qs = qst; a.ks = m.kst; a.vs = m.vst; a.ds = dst;
  a.lse = lse; a.lam = m.lam;
  a.seqlens_k = m.seqlens_k;
  a.B = m.B; a.H = m.H; a.group = m.group; a.N = m.N; a.npad = m.npad;
  a.causal = m.causal; a.window = m.window;
  a.sl2 = m.scale_log2; a.c1 = c1;
  a.rows = const_cast<float*>(m.rows);
  return dtype == FA_DT_BF16 ? d1_t<__nv_bfloat16>(a, s) : d1_t<__half>(a, s);
}

cudaError_t launch_diff_prep(int dtype, const void* o, const void* o2, Strides ost, const void* dout, Strides dost,
                             const float* lse, const float* lam, int B, int H, int N, int npad, float c1, float* rows,
                             float* dqacc, int* sched, cudaStream_t s) {
  if (dtype == FA_DT_BF16)
    return prep_t<__nv_bfloat16>(o, o2, ost, dout, dost, lse, lam, B, H, N, npad, c1, rows, dqacc, sched, s);
  return prep_t<__half>(o, o2, ost, dout, dost, lse, lam, B, H, N, npad, c1, rows, dqacc, sched, s);
}

cudaError_t launch_diff_bwd(int dtype, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& dout, const DiffBwdArgs& a, cudaStream_t s) {
  if (dtype == FA_DT_BF16)
    return a.window > 0 ? launch_t<__nv_bfloat16, true>(q, k, v, dout, a, s)
                        : launch_t<__nv_bfloat16, false>(q, k, v, dout, a, s);
  return a.window > 0 ? launch_t<__half, true>(q, k, v, dout, a, s) : launch_t<__half, false>(q, k, v, dout, a, s);
}

cudaError_t launch_diff_dlam(const float* part, float* dlam, int B, int H, int group, int nq, cudaStream_t s) {
  diff_dlam_kernel<<<H, 1024, 0, s>>>(part, dlam, B, H, group, nq);
  return cudaGetLastError();
}

}  // namespace fa
