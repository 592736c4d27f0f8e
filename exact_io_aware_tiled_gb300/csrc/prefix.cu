// prefix.cu -- attention of a batch whose sequences share one long prefix, for
// single tokens and short runs of tokens against caches.
//
// Mathematics.  Query t of sequence b sees the P prefix keys that every
// sequence shares and the first L_b - T + t + 1 keys of its own cache:
//     O = (sum_prefix e^{s_j} v_j + sum_own e^{s_j} v_j) / (the same sum of e^{s_j}).
// Softmax sums over disjoint key sets join by their maxima, so the prefix is one
// product of all B g T query rows of a K/V head against one copy of its keys
// (read once for all, not once a sequence), the own keys a small product per
// sequence, and both are split along the keys wherever rows are few.  Every
// split leaves (max, sum, O unnormalised) in float32; a second kernel joins
// them in split order, so results do not depend on which split ends first.
//
// What bounds it: HBM for few rows per key (decode reads each key once), the
// 16-bit tensor rate for many.  This kernel's products are m16n8k16 register
// products: a decode tile has 1 to 64 rows, and at 16 rows a 128-row tensor-
// memory tile would be seven eighths empty.  Measured: 64 sequences of one token,
// 16 heads of 64, 8,193 shared and 1-1,024 own keys (168 MB), 36 us, 4.7 TB/s (0.69
// of the copy rate); 128 sequences, 2 heads of 128, 0-2,047 own keys (134 MB) 31.5 us
// (4.3 TB/s).  More than 32 rows against many shared keys go to prefix_tc.cu (use_tc).
//
// Work items: (prefix, K/V head, row tile, key split) first, then (sequence, K/V
// head, row tile, key split), claimed from a counter by persistent CTAs (two or
// three on an SM).  Warp 4 claims them and streams their 64- or 32-key tiles of K and V
// with TMA, running ahead into the next item while warps 0-3 finish the last;
// each takes 16 rows, and the four split a tile of 16 / 32 / 64 rows into 1 / 2 /
// 4 row groups and the key tiles among 4 / 2 / 1 key groups with running
// maxima of their own, which join at the end of the item.  So a key is read from
// shared memory once per 16 rows that need it, and few rows still use all warps.
#include <algorithm>
#include <cmath>

#include "prefix.cuh"
#include "register_mma.cuh"

namespace fa {
namespace {

constexpr int kPThreads = 160;   // warps 0-3 compute, 4 TMA
constexpr int kSms = 152;        // the plan's SM count: a workspace's size does not depend on the device at hand
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int DV> struct PCfg {               // columns of q and k, and of v and o
  static constexpr int KS = D == 64 ? 64 : 32;       // keys of a stage
  static constexpr int kBox = KS * 128;              // one 64-column box of a stage
  static constexpr int kKTile = KS * D * 2, kVTile = KS * DV * 2;   // one stage
  static constexpr int NS = 4;                       // a multiple of 4: with split keys stage s is warp s % 4's
  static constexpr int kCtas = DV == 64 ? 3 : 2;     // CTAs per SM
  static constexpr int kK = 0;
  static constexpr int kV = NS * kKTile;
  static constexpr int kJoin = kV + NS * kVTile;     // [2][16][DV] O and [2][16] statistics of two warps
  static constexpr int kBar = kJoin + 2 * 16 * (DV * 4 + 16);
  static constexpr int kItem = kBar + 256;           // two published items
  static constexpr int kBytes = kItem + 128;
};
template <int D, int DV> constexpr bool fits() { return PCfg<D, DV>::kCtas * (PCfg<D, DV>::kBytes + 1024) <= 233472; }
static_assert(fits<64, 64>() && fits<128, 128>() && fits<64, 128>(), "the CTAs of one SM exceed its shared memory");

struct PBars {
  uint64_t full[4], empty[4];
  uint64_t item_full[2], item_empty[2], join;
  int abort;
};
static_assert(sizeof(PBars) <= 256, "barrier block overflows its shared-memory slot");

// One work item: rows rt * tile .. of K/V head hk against keys k0 .. kend - 1,
// of the prefix or of sequence b's cache.
struct PItem {
  bool shared;
  int b, hk, rt, sp;
  int k0, kend;          // keys of this split; kend <= the part's filled rows
  int end;               // filled rows of the part
  int rows, tile;
  int nt;                // stages, 0: nothing to do; -1 in the mailbox: no more items
};
static_assert(sizeof(PItem) <= 64, "an item overflows its mailbox slot");

template <int KS>
__device__ __forceinline__ PItem prefix_item(const PArgs& a, int u) {
  PItem it;
  it.shared = u < a.pitems;
  it.b = 0;
  int chunk;
  if (it.shared) {
    it.rt = u % a.pt;            // row tiles of the same keys run together and share them in L2
    u /= a.pt;
    it.sp = u % a.np;
    it.hk = u / a.np;
    it.end = a.P;
    chunk = a.pchunk; it.rows = a.R; it.tile = a.ptile;
  } else {
    u -= a.pitems;
    it.rt = u % a.st;
    u /= a.st;
    it.hk = u % a.Hkv;
    u /= a.Hkv;
    it.b = u % a.B;              // every sequence's first split before any second: the long ones start early
    it.sp = u / a.B;
    it.end = max(0, min(a.M, a.lens[it.b]));
    chunk = a.schunk; it.rows = a.r; it.tile = a.stile;
  }
  it.k0 = it.sp * chunk;
  it.kend = min(it.end, it.k0 + chunk);
  it.nt = it.kend > it.k0 ? (it.kend - it.k0 + KS - 1) / KS : 0;
  return it;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" :: "r"(smem_u32(bar)), "r"(n) : "memory");
}

// State of 16 query rows in one warp: thread (lane / 4, lane % 4) holds rows
// lane / 4 and lane / 4 + 8, columns 2 (lane % 4) + {0, 1} of every 8.
template <typename T, int D, int DV> struct Rows {
  uint32_t q[D / 16][4];
  float o[DV / 8][4];
  float m[2], lt[2], lr[2];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < DV / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    lt[0] = lt[1] = lr[0] = lr[1] = 0.f;
  }
  // base of each of this thread's two rows, or nullptr (zeros)
  __device__ __forceinline__ void load_q(const T* r0, const T* r1, int lane) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int c = k * 16 + 2 * (lane & 3);
      q[k][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c) : 0u;
      q[k][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c) : 0u;
      q[k][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c + 8) : 0u;
      q[k][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c + 8) : 0u;
    }
  }
  // The keys of one stage, key0 and on.  lim: keys at or past it are hidden, per
  // row; kend: V rows at or past it may hold anything.  nx = 1: only rows 0-7 of
  // the 16 exist (one token of up to 8 heads), the others' softmax is left out.
  __device__ __forceinline__ void step(uint32_t sK, uint32_t sV, int key0, const int (&lim)[2], int kend, float sl2,
                                       int lane, int nx) {
    constexpr int NK = PCfg<D, DV>::KS, kBox = PCfg<D, DV>::kBox;
    float s[NK / 8][4];
#pragma unroll
    for (int n = 0; n < NK / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
    const int lr_ = lane & 7, lm = lane >> 3;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int n = 0; n < NK / 16; ++n) {
        // matrices: keys 0-7 / 8-15 (lm >> 1), columns 0-7 / 8-15 (lm & 1)
        const uint32_t row = n * 16 + (lm >> 1) * 8 + lr_;
        const uint32_t col = (k & 3) * 16 + (lm & 1) * 8;
        uint32_t b[4];
        ldsm4(b, sK + (k >> 2) * kBox + sw128_off(row, col));
        mma16816<T>(s[2 * n], q[k], b[0], b[1]);
        mma16816<T>(s[2 * n + 1], q[k], b[2], b[3]);
      }
    }
    const int kl = key0 + 2 * (lane & 3);      // key of s[0][0]
    if (key0 + NK > min(lim[0], lim[1])) {
#pragma unroll
      for (int n = 0; n < NK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kl + n * 8 + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NK / 8; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) mx[x] = max3f(mx[x], s[n][2 * x], s[n][2 * x + 1]);
    }
    float alpha[2], nm[2];
    bool moved = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * sl2;
      // the reference maximum moves only when it is exceeded by 2^8: any
      // reference gives the same quotient, and most steps skip the rescale
      const float m_new = mx[x] > m[x] + 8.f ? mx[x] : m[x];
      alpha[x] = 1.f;
      if (m_new != m[x]) {
        alpha[x] = m[x] == -INFINITY ? 0.f : ex2(m[x] - m_new);
        moved = true;
      }
      m[x] = m_new;
      nm[x] = m_new == -INFINITY ? 0.f : -m_new;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lt[x] *= alpha[x];
        lr[x] *= alpha[x];
#pragma unroll
        for (int n = 0; n < DV / 8; ++n) {
          o[n][2 * x] *= alpha[x];
          o[n][2 * x + 1] *= alpha[x];
        }
      }
    }
    // P in 16 bits, the product's operand type (half a step per weight); the
    // rounded sum normalises O, the unrounded one makes the logsumexp
    uint32_t p[NK / 16][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= nx) {
#pragma unroll
        for (int n = 0; n < NK / 8; ++n) p[n >> 1][(n & 1) * 2 + x] = 0u;
        break;
      }
      float st[2] = {0.f, 0.f}, sr[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NK / 8; ++n) {
        float e0, e1;
        fma2(e0, e1, s[n][2 * x], s[n][2 * x + 1], sl2, sl2, nm[x], nm[x]);
        e0 = ex2(e0);
        e1 = ex2(e1);
        add2(st[0], st[1], e0, e1);
        const uint32_t u = Cvt<T>::pack(e0, e1);
        Cvt<T>::acc2(sr[0], sr[1], u);
        p[n >> 1][(n & 1) * 2 + x] = u;
      }
      lt[x] += st[0] + st[1];
      lr[x] += sr[0] + sr[1];
    }
    // V rows past kend are replaced by zeros (0 x NaN would not be 0)
    if (key0 + NK > kend) pv<true>(sV, p, kend - key0, lane);
    else pv<false>(sV, p, 0, lane);
  }
  template <bool kTail>
  __device__ __forceinline__ void pv(uint32_t sV, const uint32_t (&p)[PCfg<D, DV>::KS / 16][4], int live, int lane) {
    const int lr_ = lane & 7, lm = lane >> 3;
#pragma unroll
    for (int k = 0; k < PCfg<D, DV>::KS / 16; ++k) {
      // register pairs hold keys kp, kp + 1 and kp + 8, kp + 9
      uint32_t z0 = ~0u, z1 = ~0u;
      if (kTail) {
        const int kp = k * 16 + 2 * (lane & 3);
        z0 = (kp < live ? 0xFFFFu : 0u) | (kp + 1 < live ? 0xFFFF0000u : 0u);
        z1 = (kp + 8 < live ? 0xFFFFu : 0u) | (kp + 9 < live ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int n = 0; n < DV / 16; ++n) {
        // matrices: keys 0-7 / 8-15 (lm & 1), columns 0-7 / 8-15 (lm >> 1)
        const uint32_t row = k * 16 + (lm & 1) * 8 + lr_;
        const uint32_t col = (n & 3) * 16 + (lm >> 1) * 8;
        uint32_t b[4];
        ldsm4t(b, sV + (n >> 2) * PCfg<D, DV>::kBox + sw128_off(row, col));
        if (kTail) {
          b[0] &= z0; b[1] &= z1; b[2] &= z0; b[3] &= z1;
        }
        mma16816<T>(o[2 * n], p[k], b[0], b[1]);
        mma16816<T>(o[2 * n + 1], p[k], b[2], b[3]);
      }
    }
  }
  // this warp's rows and statistics into shared memory, and another warp's joined to this one's
  __device__ __forceinline__ void put(float* so, float4* ss, int lane, int nx) const {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= nx) break;
      const int row = (lane >> 2) + 8 * x;
      float* dst = so + row * DV + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < DV / 8; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
      if ((lane & 3) == 0) ss[row] = make_float4(m[x], lt[x], lr[x], 0.f);
    }
  }
  __device__ __forceinline__ void join(const float* so, const float4* ss, int lane, int nx) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= nx) break;
      const int row = (lane >> 2) + 8 * x;
      const float4 st = ss[row];
      const float m_new = fmaxf(m[x], st.x);
      const float fa_ = m[x] == -INFINITY ? 0.f : ex2(m[x] - m_new), fb = st.x == -INFINITY ? 0.f : ex2(st.x - m_new);
      m[x] = m_new;
      lt[x] = lt[x] * fa_ + st.y * fb;
      lr[x] = lr[x] * fa_ + st.z * fb;
      const float* src = so + row * DV + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < DV / 8; ++n) {
        const float2 v = *reinterpret_cast<const float2*>(src + n * 8);
        o[n][2 * x] = o[n][2 * x] * fa_ + v.x * fb;
        o[n][2 * x + 1] = o[n][2 * x + 1] * fa_ + v.y * fb;
      }
    }
  }
  __device__ __forceinline__ void sum_lanes() {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      lt[x] += __shfl_xor_sync(0xffffffffu, lt[x], 1);
      lt[x] += __shfl_xor_sync(0xffffffffu, lt[x], 2);
      lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 1);
      lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 2);
    }
  }
};

template <typename T, int D, int DV>
__global__ void __launch_bounds__(kPThreads, (PCfg<D, DV>::kCtas))
prefix_kernel(const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PArgs a) {
  using C = PCfg<D, DV>;
  constexpr bool kDiff = D != DV;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {       // the 128-byte swizzle's tiles: see diff_fwd.cu
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  PBars* bars = reinterpret_cast<PBars*>(smem + C::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 4);
    }
    mbar_init(&bars->join, 4);
    bars->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == 4) {
    // ===================== items and TMA =====================
    if (lane == 0) {
      prefetch_tmap(&tmKP);
      prefetch_tmap(&tmVP);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      int g = 0;                 // stages loaded
      bool ok = true;
      // the first item is the CTA's own index, the others come from the counter
      int u = (int)blockIdx.x;
      for (int kf = 0; ok; u = (int)gridDim.x + atomicAdd(a.sched, 1)) {
        PItem it;
        it.nt = -1;
        if (u < a.items) {
          it = prefix_item<C::KS>(a, u);
          if (it.nt == 0) continue;           // a split past this sequence's keys: the join does not read it
        }
        const int slot = kf & 1;
        if (kf >= 2 && !(ok = mbar_wait(&bars->item_empty[slot], (uint32_t)((kf >> 1) - 1) & 1u, ctl))) break;
        *reinterpret_cast<PItem*>(smem + C::kItem + slot * 64) = it;
        mbar_arrive(&bars->item_full[slot]);
        ++kf;
        if (it.nt < 0) break;
        const CUtensorMap* mk = it.shared ? &tmKP : &tmK;
        const CUtensorMap* mv = it.shared ? &tmVP : &tmV;
        for (int t = 0; t < it.nt; ++t, ++g) {
          const int st = g % NS;
          if (g >= NS && !(ok = mbar_wait(&bars->empty[st], (uint32_t)(g / NS - 1) & 1u, ctl))) break;
          mbar_expect_tx(&bars->full[st], C::kKTile + C::kVTile);
#pragma unroll
          for (int c = 0; c < DV / 64; ++c)
#pragma unroll
            for (int x = 0; x < C::KS; x += kKT) {
              const int row = it.k0 + t * C::KS + x, at = c * C::kBox + x * 128;
              if (c < D / 64)
                tma_load_4d(smem + C::kK + st * C::kKTile + at, mk, &bars->full[st], c * 64, row, it.hk, it.b);
              tma_load_4d(smem + C::kV + st * C::kVTile + at, mv, &bars->full[st], c * 64, row, value_head<kDiff>(it.hk),
                          it.b);
            }
        }
      }
      // no load may still be writing shared memory when the CTA ends
      for (int j = max(0, g - NS); j < g; ++j) mbar_wait(&bars->full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
    }
    return;
  }

  // ===================== compute warps =====================
  float* so = reinterpret_cast<float*>(smem + C::kJoin);              // [2][16][DV]
  float4* ss = reinterpret_cast<float4*>(so + 2 * 16 * DV);            // [2][16]
  // barrier of the four compute warps: bounded like every wait, so that a warp
  // that gave up leaves none behind
  int nj = 0;
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->join);
    return __all_sync(0xffffffffu, mbar_wait(&bars->join, (uint32_t)nj++ & 1u, ctl));
  };
  int g = 0;
  for (int kc = 0;; ++kc) {
    const int slot = kc & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl))) return;
    const PItem it = *reinterpret_cast<const PItem*>(smem + C::kItem + slot * 64);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    if (it.nt < 0) return;
    // warp = (key group) * rgs + (row group): rgs groups of 16 rows, 4 / rgs of stages
    const int rgs = it.tile >> 4, kgs = 4 / rgs;
    const int rg = warp & (rgs - 1), kg = warp / rgs;
    // This warp's key group counted from the item's first stage: group lk has stages lk,
    // lk + kgs, ... of the item, wherever in the ring the item starts.  The joins go by it,
    // so a result's bits follow from the item alone, not from the items before it.
    const int lk = (kg - g) & (kgs - 1), lw = lk * rgs + rg;
    const int rbase = it.rt * it.tile + rg * 16 + (lane >> 2);
    Rows<T, D, DV> w;
    w.init();
    int lim[2] = {0, 0};
    const T* qr[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rbase + 8 * x;
      qr[x] = nullptr;
      if (row < it.rows) {
        // shared: row (b, j, t) of all sequences; else (j, t) of sequence it.b
        const int b = it.shared ? row / a.r : it.b;
        const int rem = it.shared ? row - b * a.r : row;
        const int j = a.T == 1 ? rem : rem / a.T, t = rem - j * a.T;
        qr[x] = prefix_row<T, kDiff>(a, it.hk, b, j, t);
        lim[x] = it.shared ? a.P : it.end - a.T + t + 1;
      }
    }
    w.load_q(qr[0], qr[1], lane);
    const int left = it.rows - it.rt * it.tile - rg * 16;            // rows of this warp's 16
    const int nx = left <= 0 ? 0 : left <= 8 ? 1 : 2;                 // eights of rows that exist
    for (int t = 0; t < it.nt; ++t, ++g) {
      const int st = g % NS;
      // A stage belongs to one key group for all its phases in an item.  The
      // other warps do not wait on it (they would lag behind its phases); where
      // they next do, in an item split otherwise, the join has brought all
      // warps together.
      if ((st & (kgs - 1)) != kg) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[st], (uint32_t)(g / NS) & 1u, ctl))) return;
      const uint32_t sK = smem_u32(smem + C::kK + st * C::kKTile), sV = smem_u32(smem + C::kV + st * C::kVTile);
      const int key0 = it.k0 + t * C::KS;
      if (nx > 0) w.step(sK, sV, key0, lim, it.kend, a.scale_log2, lane, nx);
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&bars->empty[st], kgs);
    }
    w.sum_lanes();
    // ---- join the key groups: lw 2, 3 into 0, 1, then (one row group) 1 into 0
#pragma unroll 1
    for (int half = 2; half >= rgs; half >>= 1) {
      if (lw >= half && lw < 2 * half) w.put(so + (lw - half) * 16 * DV, ss + (lw - half) * 16, lane, nx);
      if (!meet()) return;
      if (lw < half) w.join(so + lw * 16 * DV, ss + lw * 16, lane, nx);
      if (!meet()) return;
    }
    if (lk != 0) continue;
    // row i of this item in the partial arrays
    const long long prow0 = it.shared ? ((long long)it.sp * a.Hkv + it.hk) * a.R
                                      : a.srow0 + (((long long)it.b * a.Hkv + it.hk) * a.ns + it.sp) * a.r;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rbase + 8 * x;
      if (row >= it.rows) continue;
      float* dst = a.part + (prow0 + row) * DV + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < DV / 8; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(w.o[n][2 * x], w.o[n][2 * x + 1]);
      if ((lane & 3) == 0) a.stat[prow0 + row] = make_float4(w.m[x], w.lt[x], w.lr[x], 0.f);
    }
  }
}

// Joins the splits of each query row: W warps per row (1 for few splits, else 4),
// DV / 32 columns a lane.  The lanes fetch the splits' statistics side by side,
// then every split's row is an independent load.  The differential form joins
// both maps' rows and leaves their difference.  Launched to overlap the end of
// the kernel before it (griddepcontrol.wait before the first read of its rows).
template <typename T, int DV, int W, bool kDiff>
__global__ void __launch_bounds__(128) prefix_join_kernel(const PArgs a, T* __restrict__ o, Strides os,
                                                          float* __restrict__ lse) {
  constexpr int E = DV / 32;
  __shared__ float sh[W == 1 ? 1 : 4][W == 1 ? 1 : DV + 3];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = W == 1 ? (int)(blockIdx.x * 4 + warp) : (int)blockIdx.x;       // B H T < 2^26
  const int w0 = W == 1 ? 0 : warp;
  const int OH = kDiff ? a.H / 2 : a.H;                                          // heads of o
  const bool live = row < a.B * OH * a.T;
  const int bh = live ? row / a.T : 0, t = live ? row - bh * a.T : 0;
  const int b = bh / OH, h = bh - b * OH;
  const int p = h / a.G, j = h - p * a.G;                                        // K/V head (pair) and place in its group
  const int len = max(0, min(a.M, a.lens[b]));
  const int n = live ? a.np + (len + a.schunk - 1) / a.schunk : 0;
  const long long prow = ((long long)b * a.G + j) * a.T + t;             // row of the prefix items
  float out[E] = {};
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
  for (int x = 0; x < (kDiff ? 2 : 1); ++x) {
    const int hk = kDiff ? 2 * p + x : p;
    const long long own = a.srow0 + (((long long)b * a.Hkv + hk) * a.ns) * a.r + (long long)j * a.T + t;
    auto at = [&](int s) -> long long {
      return s < a.np ? ((long long)s * a.Hkv + hk) * a.R + prow : own + (long long)(s - a.np) * a.r;
    };
    float m = -INFINITY, acc[E] = {}, lt = 0.f, lr = 0.f;
    // this warp's splits: w0, w0 + W, ...; 32 statistics at a time
    for (int s0 = w0; s0 < n; s0 += 32 * W) {
      const int cnt = min(32, (n - s0 + W - 1) / W);
      // eight splits' rows at a time, the first eight on their way before the
      // statistics that weigh them are in
      float v[8][E];
      auto fetch8 = [&](int s1) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float* src = a.part + at(s0 + min(s1 + s, cnt - 1) * W) * DV + lane * E;
          if constexpr (E == 2) *reinterpret_cast<float2*>(v[s]) = *reinterpret_cast<const float2*>(src);
          else *reinterpret_cast<float4*>(v[s]) = *reinterpret_cast<const float4*>(src);
        }
      };
      fetch8(0);
      const float4 st = lane < cnt ? a.stat[at(s0 + lane * W)] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      float mx = st.x;
#pragma unroll
      for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
      const float m_new = fmaxf(m, mx);
      const float old = m == -INFINITY ? 0.f : ex2(m - m_new);
      m = m_new;
      const float f = st.x == -INFINITY ? 0.f : ex2(st.x - m);
      float ft = f * st.y, fr = f * st.z;
#pragma unroll
      for (int y = 16; y > 0; y >>= 1) {
        ft += __shfl_xor_sync(0xffffffffu, ft, y);
        fr += __shfl_xor_sync(0xffffffffu, fr, y);
      }
      lt = lt * old + ft;
      lr = lr * old + fr;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= old;
      for (int s1 = 0; s1 < cnt; s1 += 8) {
        if (s1 > 0) fetch8(s1);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float fs = __shfl_sync(0xffffffffu, f, (s1 + s) & 31);
          if (s1 + s < cnt) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += fs * v[s][e];
          }
        }
      }
    }
    if constexpr (W > 1) {
      // the four warps' parts, in warp order
      if (x > 0) __syncthreads();          // the first map's parts have been read
#pragma unroll
      for (int e = 0; e < E; ++e) sh[warp][lane * E + e] = acc[e];
      if (lane == 0) {
        sh[warp][DV] = m; sh[warp][DV + 1] = lt; sh[warp][DV + 2] = lr;
      }
      __syncthreads();
      float mm = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; ++g) mm = fmaxf(mm, sh[g][DV]);
      lt = lr = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float f = sh[g][DV] == -INFINITY ? 0.f : ex2(sh[g][DV] - mm);
        lt += f * sh[g][DV + 1];
        lr += f * sh[g][DV + 2];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * sh[g][lane * E + e];
      }
      m = mm;
    }
    const float inv = lr > 0.f ? 1.f / lr : 0.f;
    const float c = x == 0 ? inv : -a.lam[h] * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] += c * acc[e];
    if (live && lane == 0 && (W == 1 || warp == 0))
      lse[((long long)b * a.H + (kDiff ? 2 * h + x : h)) * a.T + t] = lt > 0.f ? (m + lg2(lt)) * kLn2 : -INFINITY;
  }
  if (!live || (W > 1 && warp != 0)) return;
  T* dst = o + (int64_t)b * os.b + (int64_t)h * os.h + (int64_t)t * os.n + lane * E;
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) w[e] = Cvt<T>::pack(out[2 * e], out[2 * e + 1]);
  if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
  else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

template <typename T, int DV, int W, bool kDiff>
cudaError_t launch_join(const PArgs& a, void* o, Strides os, float* lse, cudaStream_t s) {
  const int rows = a.B * (kDiff ? a.H / 2 : a.H) * a.T;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(W == 1 ? (rows + 3) / 4 : rows));
  c.blockDim = dim3(128);
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, prefix_join_kernel<T, DV, W, kDiff>, a, static_cast<T*>(o), os, lse);
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Whether the shared keys go to the tensor-memory kernel: by the work, 64-row tiles x
// shared keys x d, that has to pay for a launch of its own.  us here / there, 8 heads,
// 512 own keys a sequence.  Well above the limit it wins: d = 128, 33 rows x 65,536
// keys 84 / 68, 256 rows x 65,536 310 / 159; d = 64, 64 rows x 65,536 59 / 52, 256
// rows x 65,536 153 / 104.  At the limit and up to three times it the rule takes the
// slower side by a little: d = 128, 64 rows x 16,384 51 / 52, 65 rows x 8,192 46 / 47;
// d = 64, 65 rows x 16,384 31 / 33, 129 rows x 16,384 51 / 55.  Up to 32 rows the two
// are level without own keys.
bool use_tc(const fa_prefix_params* p, int rows, int heads) {
  return rows > 32 && (long long)heads * ((rows + 63) / 64) * p->P >= (1 << 24) / p->d;
}

// Whether the tensor-memory kernel's two slots take two key splits of the same rows.
// That keeps the second slot busy where the rows fill one, and gives the join twice
// the splits.  us one slot / folded, d = 64, 64 rows: 16 heads x 8,192 keys 17.1 / 17.4,
// x 16,384 26.5 / 23.6, x 65,536 72 / 57.  At d = 128 a slot would have one stage of K
// and V to itself: 91 / 95.
bool use_fold(const fa_prefix_params* p, int rows, int heads) {
  return p->d == 64 && rows <= 128 && (long long)heads * p->P >= 1 << 18;
}

int row_tile(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Row tiles and key splits.  The work of a 64-key unit is tile / 16 warp tiles;
// splits are cut so that the items are about equal in that measure and number
// three for every resident CTA (ragged lengths and the long prefix items even
// out; six cost 4 % more than they even out), but no shorter than four units, the
// prefix's than eight, unless CTAs would be left without an item.
void plan(const fa_prefix_params* p, PArgs& a) {
  constexpr int kU = 64;
  const int maps = p->lam != nullptr ? 2 : 1;      // score heads per head
  a.B = p->B; a.H = maps * p->H; a.Hkv = maps * p->H_kv; a.T = p->T; a.G = p->H / p->H_kv;
  a.lam = p->lam;
  a.P = p->P; a.M = p->M;
  a.r = a.G * a.T;
  a.R = a.B * a.r;
  a.ptile = use_tc(p, a.R, a.Hkv) ? 256 : row_tile(a.R);
  a.stile = row_tile(a.r);
  a.pt = (a.R + a.ptile - 1) / a.ptile;
  a.st = (a.r + a.stile - 1) / a.stile;
  const long long kp = ((long long)a.P + kU - 1) / kU, ks = ((long long)a.M + kU - 1) / kU;
  const int pw = a.ptile / 16, sw = a.stile / 16;
  const long long wp = a.ptile == 256 ? 0 : (long long)a.Hkv * a.pt * kp * pw;
  const long long wsuf = (long long)a.B * a.Hkv * a.st * ks * sw;
  const long long ctas = (long long)kSms * (p->d == 64 && maps == 1 ? PCfg<64, 64>::kCtas : PCfg<128, 128>::kCtas);
  const long long share = (wp + wsuf + 3 * ctas - 1) / (3 * ctas);
  const long long least = std::clamp<long long>(((long long)a.B * a.Hkv * a.st * ks + ctas - 1) / ctas, 2, 4);
  const long long sc = std::max(least, share / sw);
  long long pc = std::max<long long>(8, share / pw);
  // Where the own keys leave room, prefix splits that fill one round exactly: down
  // to two units (1,024 shared keys, 2 heads of 128: 14.4 -> 10.3 us) but not above
  // 64 splits for that (the join reads them one after another), and up to twice the
  // length above rather than a little over one round (72 tokens against 23,400 keys
  // x 12 heads: 19.0 -> 15.9 us).
  const long long own = (long long)a.B * a.Hkv * a.st * ((ks + sc - 1) / sc), heads = (long long)a.Hkv * a.pt;
  if (a.ptile != 256 && heads > 0 && ctas - own >= heads) {
    const long long splits = (ctas - own) / heads, fit = (kp + splits - 1) / splits;
    const long long low = std::clamp<long long>((kp + 63) / 64, 2, 8);
    if (fit <= 2 * pc) pc = std::max({fit, low, share / pw});
  }
  if (a.ptile == 256) {
    a.fold = use_fold(p, a.R, a.Hkv);
    // one CTA a SM: key splits such that one wave covers the heads and row tiles
    // (two splits a CTA where the rows fill one slot)
    const long long groups = (long long)a.Hkv * a.pt;
    const long long splits = (1 + a.fold) * std::max<long long>(1, kSms / groups);
    pc = 2 * std::max<long long>(1, ((kp + 1) / 2 + splits - 1) / splits);
  }
  a.pchunk = (int)(std::min<long long>(pc, 1 << 21) * kU);
  a.schunk = (int)(std::min<long long>(sc, 1 << 21) * kU);
  a.np = (int)((a.P + (long long)a.pchunk - 1) / a.pchunk);
  a.ns = (int)((a.M + (long long)a.schunk - 1) / a.schunk);
  a.pitems = a.ptile == 256 ? 0 : a.Hkv * a.pt * a.np;
  a.items = a.pitems + a.B * a.Hkv * a.st * a.ns;
  a.srow0 = (long long)a.np * a.Hkv * a.R;
}

// The workspace is 16-byte aligned, prefix_tc_kernel's 32-byte stores of partial rows want 32: the launch rounds
// part's address up, and the size leaves room for that.
constexpr size_t kPartAlign = 32;

struct PLayout { size_t status, stat, part, total; };
PLayout playout(const PArgs& a, int d) {      // d: value columns
  PLayout L;
  const size_t rows = (size_t)a.srow0 + (size_t)a.B * a.Hkv * a.ns * a.r;
  L.status = 0;
  L.stat = 256;
  L.part = L.stat + al256(rows * sizeof(float4));
  L.total = L.part + al256(rows * d * sizeof(float)) + kPartAlign;
  return L;
}

template <typename T, int D, int DV>
cudaError_t launch_p(const CUtensorMap (&m)[4], const PArgs& a, void* o, Strides os, float* lse, cudaStream_t s) {
  using C = PCfg<D, DV>;
  constexpr bool kDiff = D != DV;
  auto kern = prefix_kernel<T, D, DV>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  if (a.ptile == 256 && (e = launch_prefix_tc(Cvt<T>::kAB ? FA_DT_BF16 : FA_DT_F16, D, m[0], m[1], a, s)) != cudaSuccess)
    return e;
  if (a.items > 0) {
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min<long long>(a.items, (long long)C::kCtas * std::max(sms, 1));
    kern<<<grid, kPThreads, C::kBytes, s>>>(m[0], m[1], m[2], m[3], a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return a.np + a.ns <= 8 ? launch_join<T, DV, 1, kDiff>(a, o, os, lse, s) : launch_join<T, DV, 4, kDiff>(a, o, os, lse, s);
}

}  // namespace

// Arguments have been checked (check_prefix in api.cu).
size_t prefix_workspace(const fa_prefix_params* p) {
  PArgs a{};
  plan(p, a);
  return playout(a, p->lam != nullptr ? 2 * p->d : p->d).total;
}

cudaError_t launch_prefix(const fa_prefix_params* p, const CUtensorMap (&m)[4], const void* q, Strides qs, void* o,
                          Strides os, float* lse, float scale_log2, uint8_t* ws, cudaStream_t s) {
  PArgs a{};
  plan(p, a);
  const PLayout L = playout(a, p->lam != nullptr ? 2 * p->d : p->d);
  a.q = q;
  a.qs = qs;
  a.lens = p->seqlens_k;
  a.scale_log2 = scale_log2;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.stat = reinterpret_cast<float4*>(ws + L.stat);
  a.part = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws + L.part) + kPartAlign - 1) & ~uintptr_t(kPartAlign - 1));
  a.sched = a.status + 1;
  cudaError_t e = cudaMemsetAsync(a.status, 0, 2 * sizeof(int), s);
  if (e != cudaSuccess) return e;
  using B16 = __nv_bfloat16;
  const bool bf = p->dtype == FA_DT_BF16;
  if (p->lam != nullptr)
    return bf ? launch_p<B16, 64, 128>(m, a, o, os, lse, s) : launch_p<__half, 64, 128>(m, a, o, os, lse, s);
  if (p->d == 128)
    return bf ? launch_p<B16, 128, 128>(m, a, o, os, lse, s) : launch_p<__half, 128, 128>(m, a, o, os, lse, s);
  return bf ? launch_p<B16, 64, 64>(m, a, o, os, lse, s) : launch_p<__half, 64, 64>(m, a, o, os, lse, s);
}

}  // namespace fa
