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
// memory tile would be seven eighths empty.
//
// Work items (one CTA each, two CTAs on an SM): (prefix, K/V head, row tile,
// key split) first, then (sequence, K/V head, row tile, key split).  Warp 4
// streams 64-key tiles of K and V with TMA; warps 0-3 compute:
//   * up to 16 rows: each warp takes 16 of a tile's 64 keys for all rows, with
//     its own running maximum, and the four join at the end: every key is read
//     from shared memory once;
//   * more rows: each warp takes 16 rows of a 64-row tile and all keys.
#include <algorithm>
#include <cmath>

#include "prefix.cuh"

namespace fa {
namespace {

constexpr int kPThreads = 160;   // warps 0-3 compute, 4 TMA
constexpr int kSlots = 304;      // CTAs resident at once: two on each of 152 SMs
constexpr float kLn2 = 0.6931471805599453f;

template <int D> struct PCfg {
  static constexpr int NB = D / 64;                  // 64-column boxes per row
  static constexpr int kTile = kKT * D * 2;          // one K or V stage
  static constexpr int NS = D == 64 ? 6 : 3;
  static constexpr int kK = 0;
  static constexpr int kV = NS * kTile;
  static constexpr int kBar = kV + NS * kTile;
  static constexpr int kBytes = kBar + 256;
};

struct PBars {
  uint64_t full[6], empty[6];
  int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (Cvt<T>::kAB == 1)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// State of 16 query rows in one warp: thread (lane / 4, lane % 4) holds rows
// lane / 4 and lane / 4 + 8, columns 2 (lane % 4) + {0, 1} of every 8.
template <typename T, int D> struct Rows {
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float m[2], lt[2], lr[2];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
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
  // NK keys (a multiple of 16) of a stage, from stage row `row0`; the key of
  // stage row x is key0 + x.  lim: keys at or past it are hidden, per row;
  // kend: V rows at or past it may hold anything.
  template <int NK>
  __device__ __forceinline__ void step(uint32_t sK, uint32_t sV, int row0, int key0, const int (&lim)[2], int kend,
                                       float sl2, int lane) {
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
        const uint32_t row = row0 + n * 16 + (lm >> 1) * 8 + lr_;
        const uint32_t col = (k & 3) * 16 + (lm & 1) * 8;
        uint32_t b[4];
        ldsm4(b, sK + (k >> 2) * (kKT * 128) + sw128_off(row, col));
        mma16816<T>(s[2 * n], q[k], b[0], b[1]);
        mma16816<T>(s[2 * n + 1], q[k], b[2], b[3]);
      }
    }
    const int kl = key0 + row0 + 2 * (lane & 3);      // key of s[0][0]
    if (key0 + row0 + NK > min(lim[0], lim[1])) {
#pragma unroll
      for (int n = 0; n < NK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kl + n * 8 + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NK / 8; ++n) {
      mx[0] = fmaxf(mx[0], fmaxf(s[n][0], s[n][1]));
      mx[1] = fmaxf(mx[1], fmaxf(s[n][2], s[n][3]));
    }
    float alpha[2], nm[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      const float m_new = fmaxf(m[x], mx[x] * sl2);
      alpha[x] = m[x] == -INFINITY ? 1.f : ex2(m[x] - m_new);
      m[x] = m_new;
      nm[x] = m_new == -INFINITY ? 0.f : -m_new;
      lt[x] *= alpha[x];
      lr[x] *= alpha[x];
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= alpha[0];
        o[n][1] *= alpha[0];
        o[n][2] *= alpha[1];
        o[n][3] *= alpha[1];
      }
    }
    // P in 16 bits, the product's operand type (half a step per weight); the
    // rounded sum normalises O, the unrounded one makes the logsumexp
    uint32_t p[NK / 16][4];
#pragma unroll
    for (int n = 0; n < NK / 8; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p0 = ex2(fmaf(s[n][2 * x], sl2, nm[x])), p1 = ex2(fmaf(s[n][2 * x + 1], sl2, nm[x]));
        lt[x] += p0 + p1;
        const uint32_t u = Cvt<T>::pack(p0, p1);
        lr[x] += Cvt<T>::lo(u) + Cvt<T>::hi(u);
        p[n >> 1][(n & 1) * 2 + x] = u;
      }
    }
    const bool tail = key0 + row0 + NK > kend;
#pragma unroll
    for (int k = 0; k < NK / 16; ++k) {
      // V rows past kend are replaced by zeros (0 x NaN would not be 0): register
      // pairs hold keys kp, kp + 1 and kp + 8, kp + 9
      uint32_t z0 = ~0u, z1 = ~0u;
      if (tail) {
        const int kp = key0 + row0 + k * 16 + 2 * (lane & 3);
        z0 = (kp < kend ? 0xFFFFu : 0u) | (kp + 1 < kend ? 0xFFFF0000u : 0u);
        z1 = (kp + 8 < kend ? 0xFFFFu : 0u) | (kp + 9 < kend ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        // matrices: keys 0-7 / 8-15 (lm & 1), columns 0-7 / 8-15 (lm >> 1)
        const uint32_t row = row0 + k * 16 + (lm & 1) * 8 + lr_;
        const uint32_t col = (n & 3) * 16 + (lm >> 1) * 8;
        uint32_t b[4];
        ldsm4t(b, sV + (n >> 2) * (kKT * 128) + sw128_off(row, col));
        mma16816<T>(o[2 * n], p[k], b[0] & z0, b[1] & z1);
        mma16816<T>(o[2 * n + 1], p[k], b[2] & z0, b[3] & z1);
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

template <typename T, int D>
__global__ void __launch_bounds__(kPThreads, 2)
prefix_kernel(const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PArgs a) {
  using C = PCfg<D>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {       // the 128-byte swizzle's tiles: see diff_fwd.cu
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  PBars* bars = reinterpret_cast<PBars*>(smem + C::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item
  int it = (int)blockIdx.x;
  const bool shared = it < a.pitems;
  int b = 0, hk, rt, sp, kend, chunk, rows, tile;
  if (shared) {
    rt = it % a.pt;            // row tiles of the same keys run together and share them in L2
    it /= a.pt;
    sp = it % a.np;
    hk = it / a.np;
    kend = a.P;
    chunk = a.pchunk; rows = a.R; tile = a.ptile;
  } else {
    it -= a.pitems;
    rt = it % a.st;
    it /= a.st;
    hk = it % a.Hkv;
    it /= a.Hkv;
    b = it % a.B;
    sp = it / a.B;
    kend = max(0, min(a.M, a.lens[b]));
    chunk = a.schunk; rows = a.r; tile = a.stile;
  }
  const int k0 = sp * chunk;
  if (k0 >= kend) return;                     // a split past this sequence's keys: the join does not read it
  const int len = kend;
  const int nt = (min(kend - k0, chunk) + kKT - 1) / kKT;

  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 4);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == 4) {
    if (lane == 0) {
      const CUtensorMap* mk = shared ? &tmKP : &tmK;
      const CUtensorMap* mv = shared ? &tmVP : &tmV;
      int t = 0;
      for (; t < nt; ++t) {
        const int st = t % NS;
        if (t >= NS && !mbar_wait(&bars->empty[st], (uint32_t)(t / NS - 1) & 1u, ctl)) break;
        mbar_expect_tx(&bars->full[st], 2 * C::kTile);
#pragma unroll
        for (int c = 0; c < C::NB; ++c) {
          tma_load_4d(smem + C::kK + st * C::kTile + c * (kKT * 128), mk, &bars->full[st], c * 64, k0 + t * kKT, hk, b);
          tma_load_4d(smem + C::kV + st * C::kTile + c * (kKT * 128), mv, &bars->full[st], c * 64, k0 + t * kKT, hk, b);
        }
      }
      // no load may still be writing shared memory when the CTA ends
      for (int j = max(0, t - NS); j < t; ++j) mbar_wait(&bars->full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
    }
    if (tile != 16) return;
  }

  Rows<T, D> w;
  const bool split_keys = tile == 16;
  const int rbase = rt * tile + (split_keys ? 0 : warp * 16) + (lane >> 2);
  int lim[2] = {0, 0};
  bool ok = true;
  if (warp < 4) {
    w.init();
    const T* qr[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rbase + 8 * x;
      qr[x] = nullptr;
      if (row < rows) {
        qr[x] = prefix_row<T>(a, hk, shared ? row : b * a.r + row);
        lim[x] = shared ? a.P : len - a.T + row % a.T + 1;
      }
    }
    w.load_q(qr[0], qr[1], lane);
    const bool idle = !split_keys && rt * tile + warp * 16 >= rows;
    for (int t = 0; t < nt; ++t) {
      const int st = t % NS;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[st], (uint32_t)(t / NS) & 1u, ctl));
      if (!ok) break;
      const uint32_t sK = smem_u32(smem + C::kK + st * C::kTile), sV = smem_u32(smem + C::kV + st * C::kTile);
      const int key0 = k0 + t * kKT;
      if (split_keys) {
        if (key0 + warp * 16 < kend) w.template step<16>(sK, sV, warp * 16, key0, lim, kend, a.scale_log2, lane);
      } else if (!idle) {
        w.template step<64>(sK, sV, 0, key0, lim, kend, a.scale_log2, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->empty[st]);
    }
    w.sum_lanes();
  }
  // row i of this item in the partial arrays
  const long long prow0 = shared ? ((long long)sp * a.Hkv + hk) * a.R
                                 : a.srow0 + (((long long)b * a.Hkv + hk) * a.ns + sp) * a.r;
  if (!split_keys) {
    if (!ok) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rbase + 8 * x;
      if (row >= rows) continue;
      float* dst = a.part + (prow0 + row) * D + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(w.o[n][2 * x], w.o[n][2 * x + 1]);
      if ((lane & 3) == 0) a.stat[prow0 + row] = make_float4(w.m[x], w.lt[x], w.lr[x], 0.f);
    }
    return;
  }
  // ---- join the four warps' key quarters (the stages are free: every load has landed and been read)
  float* so = reinterpret_cast<float*>(smem);                       // [4][16][D]
  float* ss = so + 4 * 16 * D;                                      // [4][16][3]
  const bool any_bad = __syncthreads_or(!ok || bars->abort);
  if (any_bad) return;
  if (warp < 4) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = (lane >> 2) + 8 * x;
      float* dst = so + (warp * 16 + row) * D + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(w.o[n][2 * x], w.o[n][2 * x + 1]);
      if ((lane & 3) == 0) {
        float* d = ss + (warp * 16 + row) * 3;
        d[0] = w.m[x]; d[1] = w.lt[x]; d[2] = w.lr[x];
      }
    }
  }
  __syncthreads();
  const int nrow = min(16, rows - rt * 16);
  for (int e = threadIdx.x; e < nrow * (D / 4); e += kPThreads) {
    const int row = e / (D / 4), c = (e % (D / 4)) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) m = fmaxf(m, ss[(g * 16 + row) * 3]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lt = 0.f, lr = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float mg = ss[(g * 16 + row) * 3];
      const float f = mg == -INFINITY ? 0.f : ex2(mg - m);
      const float4 v = *reinterpret_cast<const float4*>(so + (g * 16 + row) * D + c);
      acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
      lt += f * ss[(g * 16 + row) * 3 + 1];
      lr += f * ss[(g * 16 + row) * 3 + 2];
    }
    const long long pr = prow0 + rt * 16 + row;
    *reinterpret_cast<float4*>(a.part + pr * D + c) = acc;
    if (c == 0) a.stat[pr] = make_float4(m, lt, lr, 0.f);
  }
}

// Joins the splits of each query row: one warp per row, D / 32 columns a lane.
// Bound by the partial rows it reads (mostly from L2) and its launch.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PArgs a, T* __restrict__ o, Strides os,
                                                          float* __restrict__ lse) {
  constexpr int E = D / 32;
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.B * a.H * a.T) return;
  const int t = (int)(row % a.T);
  const long long bh = row / a.T;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H);
  const int hk = h / a.G, j = h - hk * a.G;
  const int len = max(0, min(a.M, a.lens[b]));
  const int ns = (len + a.schunk - 1) / a.schunk;
  const int n = a.np + ns;
  const long long prow = ((long long)b * a.G + j) * a.T + t;             // row of the prefix items
  const long long own = a.srow0 + (((long long)b * a.Hkv + hk) * a.ns) * a.r + (long long)j * a.T + t;
  auto at = [&](int s) -> long long {
    return s < a.np ? ((long long)s * a.Hkv + hk) * a.R + prow : own + (long long)(s - a.np) * a.r;
  };
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, a.stat[at(s)].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float acc[E] = {}, lt = 0.f, lr = 0.f;
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const long long p = at(s);
    const float4 st = a.stat[p];
    const float f = st.x == -INFINITY ? 0.f : ex2(st.x - m);
    lt += f * st.y;
    lr += f * st.z;
    float v[E];
    if constexpr (E == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(a.part + p * D + lane * E);
    else *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(a.part + p * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * v[e];
  }
  const float inv = lr > 0.f ? 1.f / lr : 0.f;
  T* dst = o + (int64_t)b * os.b + (int64_t)h * os.h + (int64_t)t * os.n + lane * E;
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) w[e] = Cvt<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
  else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  if (lane == 0) lse[row] = lt > 0.f ? (m + lg2(lt)) * kLn2 : -INFINITY;
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Row tiles and key splits.  Enough items to fill the resident CTAs about three
// times (ragged lengths even out), no split shorter than four key tiles, and
// prefix splits long against the 64 partial rows they leave where the grid
// allows it.
bool use_tc(const fa_prefix_params* p, int rows) {
  return rows > 128 && p->P >= 256;
}

void plan(const fa_prefix_params* p, PArgs& a) {
  a.B = p->B; a.H = p->H; a.Hkv = p->H_kv; a.T = p->T; a.G = p->H / p->H_kv;
  a.P = p->P; a.M = p->M;
  a.r = a.G * a.T;
  a.R = a.B * a.r;
  a.ptile = a.R <= 16 ? 16 : use_tc(p, a.R) ? 256 : 64;
  a.stile = a.r <= 16 ? 16 : 64;
  a.pt = (a.R + a.ptile - 1) / a.ptile;
  a.st = (a.r + a.stile - 1) / a.stile;
  const long long kp = (a.P + kKT - 1) / kKT, ks = (a.M + kKT - 1) / kKT;
  const long long wp = (long long)a.Hkv * a.pt * kp, wsuf = (long long)a.B * a.Hkv * a.st * ks;
  auto clampll = [](long long x, long long lo, long long hi) { return x < lo ? lo : x > hi ? hi : x; };
  const long long even = (wp + wsuf + 3 * kSlots - 1) / (3 * kSlots);
  long long pc = clampll(even, 4, 1 << 20), sc = clampll(even, 4, 64);
  if (a.ptile == 256) {
    // one CTA a SM: key splits such that one wave of 152 covers the heads and row tiles
    const long long groups = (long long)a.Hkv * a.pt, splits = std::max<long long>(1, 152 / groups);
    pc = 2 * std::max<long long>(1, ((kp + 1) / 2 + splits - 1) / splits);
    sc = clampll((wsuf + 3 * kSlots - 1) / (3 * kSlots), 4, 64);
  }
  if (a.ptile == 64) pc = std::max(pc, std::min<long long>(16, clampll(wp / kSlots, 4, 16)));
  a.pchunk = (int)(pc * kKT);
  a.schunk = (int)(sc * kKT);
  a.np = (int)((a.P + (long long)a.pchunk - 1) / a.pchunk);
  a.ns = (int)((a.M + (long long)a.schunk - 1) / a.schunk);
  a.pitems = a.ptile == 256 ? 0 : a.Hkv * a.pt * a.np;
  a.srow0 = (long long)a.np * a.Hkv * a.R;
}

struct PLayout { size_t status, stat, part, total; };
PLayout playout(const PArgs& a, int d) {
  PLayout L;
  const size_t rows = (size_t)a.srow0 + (size_t)a.B * a.Hkv * a.ns * a.r;
  L.status = 0;
  L.stat = 256;
  L.part = L.stat + al256(rows * sizeof(float4));
  L.total = L.part + al256(rows * d * sizeof(float));
  return L;
}

template <typename T, int D>
cudaError_t launch_p(const CUtensorMap (&m)[4], const PArgs& a, void* o, Strides os, float* lse, cudaStream_t s) {
  auto kern = prefix_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PCfg<D>::kBytes);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.pitems + (long long)a.B * a.Hkv * a.st * a.ns;
  if (a.ptile == 256 && (e = launch_prefix_tc(Cvt<T>::kAB ? FA_DT_BF16 : FA_DT_F16, D, m[0], m[1], a, s)) != cudaSuccess)
    return e;
  if (items > 0) {
    kern<<<(unsigned)items, kPThreads, PCfg<D>::kBytes, s>>>(m[0], m[1], m[2], m[3], a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const long long rows = (long long)a.B * a.H * a.T;
  prefix_join_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, static_cast<T*>(o), os, lse);
  return cudaGetLastError();
}

}  // namespace

// Arguments have been checked (check_prefix in api.cu).
size_t prefix_workspace(const fa_prefix_params* p) {
  PArgs a{};
  plan(p, a);
  return playout(a, p->d).total;
}

cudaError_t launch_prefix(const fa_prefix_params* p, const CUtensorMap (&m)[4], const void* q, Strides qs, void* o,
                          Strides os, float* lse, float scale_log2, uint8_t* ws, cudaStream_t s) {
  PArgs a{};
  plan(p, a);
  const PLayout L = playout(a, p->d);
  a.q = q;
  a.qs = qs;
  a.lens = p->seqlens_k;
  a.scale_log2 = scale_log2;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.stat = reinterpret_cast<float4*>(ws + L.stat);
  a.part = reinterpret_cast<float*>(ws + L.part);
  cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int), s);
  if (e != cudaSuccess) return e;
  if (p->dtype == FA_DT_BF16)
    return p->d == 128 ? launch_p<__nv_bfloat16, 128>(m, a, o, os, lse, s) : launch_p<__nv_bfloat16, 64>(m, a, o, os, lse, s);
  return p->d == 128 ? launch_p<__half, 128>(m, a, o, os, lse, s) : launch_p<__half, 64>(m, a, o, os, lse, s);
}

}  // namespace fa
