// cache8.cu -- attention of a few new tokens over a paged cache held in 8 bits.
//
// Mathematics.  Sequence b has L rows in pages of `page` tokens; a page of one
// K/V head holds E4M3 codes and one scale each for K and V, so that
// k_j = ks c_j, v_j = vs e_j.  Query t, at position p = L - T + t, sees the keys
// j <= p and, with a window, of those the ones with j > p - window or j < sinks:
//     O = sum_j w_j vs_j e_j / sum_j w_j,   w_j = exp(tau ks_j (q . c_j)).
// Codes are widened to 16 bits exactly and multiplied as such (m16n8k16 register
// products): q keeps 11 bits (scaled by a power of two of its own, so that the
// range of bf16 fits), the weights 11.  A page's K scale multiplies its scores; its
// V scale goes into the exponent of the weights, w_j vs_j = exp2(s_j + log2 vs_j),
// whose running maximum then keeps the 16-bit weights in range whatever the
// scales, and the sum of the w_j takes it out again per 16 keys.
//
// What bounds it: HBM, one byte for each coordinate of a visible key and value,
// read once for all G T query rows of a K/V head.
//
// Work.  The 64-key (d = 128: 32-key) units that the batch's rows see, sequence by
// sequence and K/V head by K/V head, form one line; every persistent CTA takes an
// equal piece of it, so that ragged lengths cost no balance.  Rows whose units all
// lie in one CTA leave O and the logsumexp; where they are cut, the CTAs leave
// partial rows in float32 and the last one to finish joins them in their order.
// The lengths stay on the device: each CTA sums the units itself (above kPreMax
// sequences a small kernel does).  In a CTA warp 4 looks up pages and scales a
// stage a lane, 32 stages ahead, and streams codes with TMA; warps 0-3 take 16
// rows each: a tile of 16 / 32 / 64 rows is split into 1 / 2 / 4 row groups, the
// stages among 4 / 2 / 1 key groups, which join at the end of their rows.
#include <algorithm>
#include <climits>
#include <cmath>

#include "cache8.cuh"
#include "register_mma.cuh"

namespace fa {
namespace {

constexpr int kCThreads = 160;   // warps 0-3 compute, 4 looks up and loads
constexpr float kLn2 = 0.6931471805599453f;

template <int D> struct CCfg {
  static constexpr int KS = D == 64 ? 64 : 32;   // keys of a stage
  static constexpr int NG = KS / 16;             // 16-key groups of a stage, each within one page
  static constexpr int kTile = KS * D;           // bytes of K (of V) of one stage
  static constexpr int NS = 8;                   // a multiple of 4: with split keys stage s is warp s % 4's
  static constexpr int kCtas = D == 64 ? 3 : 2;  // CTAs per SM
  static constexpr int kK = 0;
  static constexpr int kV = NS * kTile;
  static constexpr int kJoin = 2 * NS * kTile;   // [2][16][D] O and [2][16] statistics of two warps
  static constexpr int kInfo = kJoin + 2 * 16 * (D * 4 + 8);
  static constexpr int kPre = kInfo + NS * 64;
  static constexpr int kItem = kPre + (kPreMax + 4) * 4;
  static constexpr int kBar = kItem + 128;
  static constexpr int kBytes = kBar + 256;
};
template <int D> constexpr bool fits() { return CCfg<D>::kCtas * (CCfg<D>::kBytes + 1024) <= 233472; }
static_assert(fits<64>() && fits<128>(), "the CTAs of one SM exceed its shared memory");
static_assert(CCfg<64>::kCtas * 152 <= kCMax && CCfg<128>::kCtas * 152 <= kCMax, "more CTAs than partial rows");

struct CBars {
  uint64_t full[8], empty[8];
  uint64_t item_full[2], item_empty[2], join;
  int abort, last;
};
static_assert(sizeof(CBars) <= 256, "barrier block overflows its shared-memory slot");

// What the compute warps need of a stage: per 16 keys the K scale, log2 of the V
// scale and its inverse, and the first key.  A group whose page is absent has the
// factors 0, -inf and 0: its weights are zero.
struct __align__(16) CInfo { float kf[4], ve[4], vi[4]; int key0, pad[3]; };
static_assert(sizeof(CInfo) == 64, "a stage's record");

struct CItem {
  int b, hk, rt, L;        // rows of tile rt of K/V head hk of sequence b
  int nt;                  // stages in this CTA; -1: no more
  int c0, pieces;          // first CTA that works at these rows, and how many do
  int slot;                // partial rows' place
};
static_assert(sizeof(CItem) <= 64, "an item overflows its mailbox slot");

// Units of one sequence: [0, ns) and, behind a gap of `skip`, the others.
struct Units { int n, ns, skip; };
template <int KS> __device__ __forceinline__ Units units_of(const Cache8Args& a, int L) {
  Units u{0, 0, 0};
  if (L <= 0) return u;
  const int hi = (L + KS - 1) / KS;
  int lo = 0;
  if (a.window > 0) lo = max(0, L - a.T - a.window + 1) / KS;      // the first query's first key
  u.ns = min((min(a.sinks, L) + KS - 1) / KS, lo);
  u.skip = lo - u.ns;
  u.n = u.ns + hi - lo;
  return u;
}
__device__ __forceinline__ int length_of(const Cache8Args& a, int b) { return max(0, min(a.cap, a.lens[b])); }

// The CTAs' shares of the line of X units
struct Share {
  long long X;
  int C;
  __device__ __forceinline__ long long begin(int c) const { return X * c / C; }
  __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * C - 1) / X); }
};

__device__ __forceinline__ uint32_t widen(uint32_t two) {       // two E4M3 codes -> two halves, exact
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint4 lds4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

// Which of the 8 keys of a product's column tile is column n = 2 m + e: any order
// serves, as K's and V's agree.  These let the lanes that read K rows together
// (both e of an m) and those that read V rows together (all m of an e) meet
// different banks of the swizzled tiles.
template <int D> __device__ __forceinline__ int key_of(int m, int e) {
  return D == 64 ? ((m & 2) << 1 | e << 1 | ((m & 1) ^ e)) : (((m >> 1) ^ e) << 2 | (m & 1) << 1 | e);
}

// State of 16 query rows in one warp: thread (lane / 4, c = lane % 4) holds rows
// lane / 4 and lane / 4 + 8.  The products' column order is free as long as both
// operands agree: a thread's K columns are 16 c .. 16 c + 15 (and 64 on), its O
// columns c D/4 .. c D/4 + D/4 - 1.
template <int D> struct CRows {
  static constexpr int KS = CCfg<D>::KS;
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2], rf[2];     // rf: what a score of the scaled q has to be multiplied by

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
  // Row x from `src` (nullptr: zeros), as halves: scaled by the power of two that
  // brings its largest value to 2^14 .. 2^15, so that bf16 loses nothing that
  // float32 sums would keep.
  template <typename T> __device__ __forceinline__ void load_q(const T* src, int x, int lane, float sl2) {
    uint32_t raw[D / 8];
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (src != nullptr) v = *reinterpret_cast<const uint4*>(src + 64 * k + 16 * (lane & 3) + 8 * i);
        raw[8 * k + 4 * i] = v.x; raw[8 * k + 4 * i + 1] = v.y;
        raw[8 * k + 4 * i + 2] = v.z; raw[8 * k + 4 * i + 3] = v.w;
      }
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) mx = max3f(mx, fabsf(Cvt<T>::lo(raw[i])), fabsf(Cvt<T>::hi(raw[i])));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int k = 14 - ((int)(__float_as_uint(mx) >> 23) - 127);
    k = mx > 0.f ? min(k, 100) : 0;
    const float f = __uint_as_float((uint32_t)(127 + k) << 23);
    rf[x] = sl2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      q[i][x] = Cvt<__half>::pack(Cvt<T>::lo(raw[2 * i]) * f, Cvt<T>::hi(raw[2 * i]) * f);
      q[i][2 + x] = Cvt<__half>::pack(Cvt<T>::lo(raw[2 * i + 1]) * f, Cvt<T>::hi(raw[2 * i + 1]) * f);
    }
  }
  // The keys of one stage.  lim, low: keys at or past lim, and below low unless
  // below sinks, are hidden, per row; end: V rows at or past it may hold anything.
  // nx = 1: only rows 0-7 of the 16 exist.
  __device__ __forceinline__ void step(uint32_t sK, uint32_t sV, uint32_t info, const int (&lim)[2], const int (&low)[2],
                                       int sinks, int end, int lane, int nx) {
    const int n = lane >> 2, c = lane & 3;
    float s[KS / 8][4];
#pragma unroll
    for (int j = 0; j < KS / 8; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
      const int kr = key_of<D>(n >> 1, n & 1), row = 8 * j + kr;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 w = lds4(sK + row * D + (D == 64 ? (c ^ ((kr >> 1) & 3)) << 4 : ((c + 4 * h) ^ kr) << 4));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma16816<__half>(s[j], q[4 * h + k], widen(ww[k] & 0xFFFFu), widen(ww[k] >> 16));
      }
    }
    const uint4 kq = lds4(info), eq = lds4(info + 16), iq = lds4(info + 32);
    const float kf[4] = {__uint_as_float(kq.x), __uint_as_float(kq.y), __uint_as_float(kq.z), __uint_as_float(kq.w)};
    const float ve[4] = {__uint_as_float(eq.x), __uint_as_float(eq.y), __uint_as_float(eq.z), __uint_as_float(eq.w)};
    const float vi[4] = {__uint_as_float(iq.x), __uint_as_float(iq.y), __uint_as_float(iq.z), __uint_as_float(iq.w)};
    int key0;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(key0) : "r"(info + 48));
    const int kb[2] = {key_of<D>(c, 0), key_of<D>(c, 1)};
#pragma unroll
    for (int j = 0; j < KS / 8; ++j) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float f = rf[x] * kf[j >> 1];
        mul2(s[j][2 * x], s[j][2 * x + 1], s[j][2 * x], s[j][2 * x + 1], f, f);
      }
    }
    if (key0 + KS > min(lim[0], lim[1]) || key0 < max(low[0], low[1])) {
#pragma unroll
      for (int j = 0; j < KS / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 8 * j + kb[e & 1];
          if (key >= lim[e >> 1] || (key < low[e >> 1] && key >= sinks)) s[j][e] = -INFINITY;
        }
    }
    // the reference maximum, of the weights times their V scales
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int g = 0; g < KS / 16; ++g) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        mx[x] = fmaxf(mx[x], fmaxf(fmaxf(s[2 * g][2 * x], s[2 * g][2 * x + 1]),
                                   fmaxf(s[2 * g + 1][2 * x], s[2 * g + 1][2 * x + 1])) + ve[g]);
    }
    float alpha[2], nm[2];
    bool moved = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      // moved only when it is exceeded by 2^8: any reference gives the same
      // quotient, and most steps skip the rescale
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
        l[x] *= alpha[x];
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[t][2 * x] *= alpha[x];
          o[t][2 * x + 1] *= alpha[x];
        }
      }
    }
    // weights to 16 bits (half a step of 2^-11 each); their sum stays unrounded
    uint32_t p[KS / 16][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int g = 0; g < KS / 16; ++g) {
        if (x >= nx) {
          p[g][x] = p[g][2 + x] = 0u;
          continue;
        }
        const float nmg = nm[x] + ve[g];
        float a0 = s[2 * g][2 * x], a1 = s[2 * g][2 * x + 1], b0 = s[2 * g + 1][2 * x], b1 = s[2 * g + 1][2 * x + 1];
        add2(a0, a1, nmg, nmg);
        add2(b0, b1, nmg, nmg);
        a0 = ex2(a0); a1 = ex2(a1); b0 = ex2(b0); b1 = ex2(b1);
        p[g][x] = Cvt<__half>::pack(a0, a1);
        p[g][2 + x] = Cvt<__half>::pack(b0, b1);
        add2(a0, a1, b0, b1);
        l[x] += (a0 + a1) * vi[g];
      }
    }
    if (key0 + KS > end) pv<true>(sV, p, end - key0, lane);
    else pv<false>(sV, p, 0, lane);
  }
  // V rows from `live` on are replaced by zeros (0 x NaN would not be 0)
  template <bool kTail>
  __device__ __forceinline__ void pv(uint32_t sV, const uint32_t (&p)[KS / 16][4], int live, int lane) {
    const int n = lane >> 2, c = lane & 3;
    const int kb[2] = {key_of<D>(c, 0), key_of<D>(c, 1)};
    uint32_t at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      at[e] = sV + kb[e] * D + (D == 64 ? (((n >> 1) ^ ((kb[e] >> 1) & 3)) << 4) + ((n & 1) << 3) : (n ^ kb[e]) << 4);
    constexpr int W = D / 32;                      // words of a row that a lane reads
#pragma unroll
    for (int g = 0; g < KS / 16; ++g) {
      uint32_t v[2][2][W];                         // [key tile][e][word]
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (D == 64) {
            const uint2 w = lds2(at[e] + (2 * g + y) * 8 * D);
            v[y][e][0] = w.x; v[y][e][1] = w.y;
          } else {
            const uint4 w = lds4(at[e] + (2 * g + y) * 8 * D);
            v[y][e][0] = w.x; v[y][e][1] = w.y; v[y][e][2] = w.z; v[y][e][3] = w.w;
          }
        }
      uint32_t z[2] = {~0u, ~0u};
      if (kTail) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int k0 = 8 * (2 * g + y);
          z[y] = (k0 + kb[0] < live ? 0xFFFFu : 0u) | (k0 + kb[1] < live ? 0xFFFF0000u : 0u);
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {           // two columns at a time
          uint32_t b[2][2];                        // [column][key tile]
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t t = __byte_perm(v[y][0][w], v[y][1][w], hf ? 0x7362 : 0x5140);
            b[0][y] = widen(t & 0xFFFFu);
            b[1][y] = widen(t >> 16);
            if (kTail) {
              b[0][y] &= z[y];
              b[1][y] &= z[y];
            }
          }
          mma16816<__half>(o[4 * w + 2 * hf], p[g], b[0][0], b[0][1]);
          mma16816<__half>(o[4 * w + 2 * hf + 1], p[g], b[1][0], b[1][1]);
        }
      }
    }
  }
  __device__ __forceinline__ void put(float* so, float2* ss, int lane, int nx) const {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= nx) break;
      const int row = (lane >> 2) + 8 * x;
      // the rows' 16-byte pieces rotated by the row: eight rows a warp would meet the same banks
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
        *reinterpret_cast<float4*>(so + row * D + 4 * ((4 * t + (lane & 3) + row) & (D / 4 - 1))) =
            make_float4(o[2 * t][2 * x], o[2 * t][2 * x + 1], o[2 * t + 1][2 * x], o[2 * t + 1][2 * x + 1]);
      if ((lane & 3) == 0) ss[row] = make_float2(m[x], l[x]);
    }
  }
  __device__ __forceinline__ void join(const float* so, const float2* ss, int lane, int nx) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= nx) break;
      const int row = (lane >> 2) + 8 * x;
      const float2 st = ss[row];
      const float m_new = fmaxf(m[x], st.x);
      const float fa_ = m[x] == -INFINITY ? 0.f : ex2(m[x] - m_new), fb = st.x == -INFINITY ? 0.f : ex2(st.x - m_new);
      m[x] = m_new;
      l[x] = l[x] * fa_ + st.y * fb;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        const float4 v = *reinterpret_cast<const float4*>(so + row * D + 4 * ((4 * t + (lane & 3) + row) & (D / 4 - 1)));
        o[2 * t][2 * x] = o[2 * t][2 * x] * fa_ + v.x * fb;
        o[2 * t][2 * x + 1] = o[2 * t][2 * x + 1] * fa_ + v.y * fb;
        o[2 * t + 1][2 * x] = o[2 * t + 1][2 * x] * fa_ + v.z * fb;
        o[2 * t + 1][2 * x + 1] = o[2 * t + 1][2 * x + 1] * fa_ + v.w * fb;
      }
    }
  }
  __device__ __forceinline__ void sum_lanes() {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
  }
};

// logsumexp, and the factor of O: a row that saw no key has l = 0, one with a NaN in it l = NaN
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + lg2(l)) * kLn2 : l == 0.f ? -INFINITY : l; }
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : l; }

// Units before each sequence, by one CTA, for batches whose prefix sums do not fit the kernel's shared memory.
template <int KS> __global__ void __launch_bounds__(1024) cache8_plan_kernel(const Cache8Args a) {
  __shared__ int warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int n = b < a.B ? units_of<KS>(a, length_of(a, b)).n : 0;
    int s = n;
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, s, y);
      if (lane >= y) s += up;
    }
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warps[w];
      all += warps[w];
    }
    if (b < a.B) a.pre[b] = before + s - n;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.pre[a.B] = carry;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCThreads, (CCfg<D>::kCtas))
cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Cache8Args a) {
  using C = CCfg<D>;
  constexpr int NS = C::NS, KS = C::KS;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {       // the swizzled tiles: see diff_fwd.cu
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  CBars* bars = reinterpret_cast<CBars*>(smem + C::kBar);
  int* const own = reinterpret_cast<int*>(smem + C::kPre);
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
    bars->last = 0;
    fence_mbar_init();
  }
  // ---- units before each sequence
  const int* pre = a.B <= kPreMax ? own : a.pre;
  if (a.B <= kPreMax) {
    for (int b = threadIdx.x; b < a.B; b += kCThreads) own[b] = units_of<KS>(a, length_of(a, b)).n;
    __syncthreads();
    if (warp == 0) {
      int carry = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = b0 + lane < a.B ? own[b0 + lane] : 0;
        int s = n;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, s, y);
          if (lane >= y) s += up;
        }
        if (b0 + lane < a.B) own[b0 + lane] = carry + s - n;
        carry += __shfl_sync(0xffffffffu, s, 31);
      }
      if (lane == 0) own[a.B] = carry;
    }
  }
  __syncthreads();
  const int HS = a.Hkv * a.tiles;
  Share sh;
  sh.X = (long long)pre[a.B] * HS;
  // No more CTAs than units, and no more than 64 pieces of a row on average: the CTA that joins them reads them all.
  sh.C = (int)max(1ll, min(min((long long)gridDim.x, sh.X), (long long)a.B * HS * 64));
  const int me = blockIdx.x;
  const long long xb = me < sh.C ? sh.begin(me) : sh.X, xe = me < sh.C ? sh.begin(me + 1) : sh.X;

  if (warp == 4) {
    // ===================== pages, scales and TMA =====================
    if (xb >= xe && lane == 0) {
      reinterpret_cast<CItem*>(smem + C::kItem)->nt = -1;
      mbar_arrive(&bars->item_full[0]);
    }
    if (xb >= xe) return;
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    // one stage a lane
    struct Look {
      CItem it;
      bool first;            // of its rows in this CTA
      int key0, id[C::NG];
    };
    auto look = [&](long long x, Look& k) {
      k.key0 = 0;
      k.first = false;
#pragma unroll
      for (int g = 0; g < C::NG; ++g) k.id[g] = -1;
      if (x >= xe) return;
      const int y = (int)(x / HS);
      int lo = 0, hi = a.B;                  // pre[lo] <= y < pre[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= y) lo = mid; else hi = mid;
      }
      const int L = length_of(a, lo);
      const Units un = units_of<KS>(a, L);
      const long long x0 = (long long)pre[lo] * HS;
      const int seg = (int)((x - x0) / un.n), i = (int)((x - x0) - (long long)seg * un.n);
      const long long s0 = x0 + (long long)seg * un.n, s1 = s0 + un.n;
      k.it.b = lo;
      k.it.hk = seg / a.tiles;
      k.it.rt = seg - k.it.hk * a.tiles;
      k.it.L = L;
      k.it.nt = (int)(min(s1, xe) - x);
      k.it.c0 = sh.owner(s0);
      k.it.pieces = sh.owner(s1 - 1) - k.it.c0 + 1;
      k.it.slot = 2 * me + (s0 >= xb ? 1 : 0);       // begun here, or by a CTA before
      k.first = i == 0 || x == xb;
      k.key0 = (i < un.ns ? i : i + un.skip) * KS;
      const int32_t* row = a.table + (int64_t)lo * a.table_stride;
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        const int key = k.key0 + 16 * g;
        if (key < L) k.id[g] = row[key >> a.lg];
      }
    };
    const int rows = min(a.page, KS), boxes = KS / rows;
    const uint32_t box = (uint32_t)rows * D;
    Look cur, nxt;
    look(xb + lane, cur);
    int kf = 0;                              // items published
    bool ok = true;
    int g0 = 0;                              // stages loaded
    for (long long x = xb; x < xe && ok; x += 32) {
      CInfo inf;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        inf.kf[g] = 0.f;
        inf.ve[g] = -INFINITY;
        inf.vi[g] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        if ((unsigned)cur.id[g] < (unsigned)a.pages) {
          const size_t at = (size_t)cur.id[g] * a.Hkv + cur.it.hk;
          inf.kf[g] = a.ks[at];
          const float vs = a.vs[at];
          // a page of zeros may have the scale 0: its codes are zero too
          inf.ve[g] = vs > 0.f ? lg2(vs) : 0.f;
          inf.vi[g] = vs > 0.f ? 1.f / vs : 1.f;
        } else {
          cur.id[g] = a.pages;               // behind the last page: the copy fills in zeros
        }
      }
      inf.key0 = cur.key0;
      look(x + 32 + lane, nxt);
      const int cnt = (int)min(32ll, xe - x);
      for (int i = 0; i < cnt; ++i, ++g0) {
        const int st = g0 % NS;
        if (lane == i) {
          if (cur.first) {
            const int slot = kf & 1;
            ok = kf < 2 || mbar_wait(&bars->item_empty[slot], (uint32_t)((kf >> 1) - 1) & 1u, ctl);
            if (ok) {
              *reinterpret_cast<CItem*>(smem + C::kItem + slot * 64) = cur.it;
              mbar_arrive(&bars->item_full[slot]);
            }
          }
          if (ok && g0 >= NS) ok = mbar_wait(&bars->empty[st], (uint32_t)(g0 / NS - 1) & 1u, ctl);
          if (ok) {
            *reinterpret_cast<CInfo*>(smem + C::kInfo + st * 64) = inf;
            // boxes behind the last row are left out: what they would bring is hidden
            const int nb = min(boxes, (cur.it.L - cur.key0 + rows - 1) / rows);
            mbar_expect_tx(&bars->full[st], 2 * box * nb);
#pragma unroll
            for (int y = 0; y < C::NG; ++y) {
              if (y >= nb) break;
              const int key = cur.key0 + y * rows;
              const int id = boxes == 1 ? cur.id[0] : boxes == C::NG ? cur.id[y] : cur.id[(2 * y) & (C::NG - 1)];
              tma_load_4d(smem + C::kK + st * C::kTile + y * box, &tmK, &bars->full[st], 0, key & (a.page - 1), cur.it.hk, id);
              tma_load_4d(smem + C::kV + st * C::kTile + y * box, &tmV, &bars->full[st], 0, key & (a.page - 1), cur.it.hk, id);
            }
          }
        }
        kf += __shfl_sync(0xffffffffu, (int)cur.first, i);
        ok = __shfl_sync(0xffffffffu, (int)ok, i) != 0;
        if (!ok) break;
      }
      cur = nxt;
    }
    if (lane == 0) {
      if (ok && (kf < 2 || mbar_wait(&bars->item_empty[kf & 1], (uint32_t)((kf >> 1) - 1) & 1u, ctl))) {
        reinterpret_cast<CItem*>(smem + C::kItem + (kf & 1) * 64)->nt = -1;
        mbar_arrive(&bars->item_full[kf & 1]);
      }
      // no load may still be writing shared memory when the CTA ends
      for (int j = max(0, g0 - NS); j < g0; ++j) mbar_wait(&bars->full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
    }
    return;
  }

  // ===================== compute warps =====================
  // sequences without keys
  for (int b = me; b < a.B; b += gridDim.x) {
    if (pre[b + 1] > pre[b]) continue;
    for (int i = threadIdx.x; i < a.H * a.T * (D / 8); i += 128) {
      const int row = i / (D / 8), h = row / a.T, t = row - h * a.T;
      T* dst = static_cast<T*>(a.o) + (int64_t)b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + (i % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
      if (i % (D / 8) == 0) a.lse[(size_t)b * a.H * a.T + row] = -INFINITY;
    }
  }
  float* so = reinterpret_cast<float*>(smem + C::kJoin);              // [2][16][D]
  float2* ss = reinterpret_cast<float2*>(so + 2 * 16 * D);             // [2][16]
  // barrier of the four compute warps: bounded like every wait
  int nj = 0;
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->join);
    return __all_sync(0xffffffffu, mbar_wait(&bars->join, (uint32_t)nj++ & 1u, ctl));
  };
  // warp = (key group) * rgs + (row group)
  const int rgs = a.tile >> 4, kgs = 4 / rgs;
  const int rg = warp & (rgs - 1), kg = warp / rgs;
  int g = 0;
  for (int kc = 0;; ++kc) {
    const int slot = kc & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->item_full[slot], (uint32_t)(kc >> 1) & 1u, ctl))) return;
    const CItem it = *reinterpret_cast<const CItem*>(smem + C::kItem + slot * 64);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    if (it.nt < 0) return;
    // this warp's key group counted from the item's first stage: the joins go by it
    const int lk = (kg - g) & (kgs - 1), lw = lk * rgs + rg;
    const int rbase = it.rt * a.tile + rg * 16 + (lane >> 2);
    CRows<D> w;
    w.init();
    int lim[2] = {INT_MAX, INT_MAX}, low[2] = {0, 0};      // rows that do not exist mask nothing
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rbase + 8 * x;
      const T* src = nullptr;
      if (row < a.r) {
        const int j = row / a.T, t = row - j * a.T;
        src = static_cast<const T*>(a.q) + (int64_t)it.b * a.qs.b + (int64_t)(it.hk * a.G + j) * a.qs.h + (int64_t)t * a.qs.n;
        lim[x] = it.L - a.T + t + 1;
        low[x] = a.window > 0 ? lim[x] - a.window : 0;
      }
      w.load_q(src, x, lane, a.scale_log2);
    }
    const int left = a.r - it.rt * a.tile - rg * 16;                  // rows of this warp's 16
    const int nx = left <= 0 ? 0 : left <= 8 ? 1 : 2;                  // eights of rows that exist
    for (int t = 0; t < it.nt; ++t, ++g) {
      const int st = g % NS;
      if ((st & (kgs - 1)) != kg) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[st], (uint32_t)(g / NS) & 1u, ctl))) return;
      if (nx > 0)
        w.step(smem_u32(smem + C::kK + st * C::kTile), smem_u32(smem + C::kV + st * C::kTile),
               smem_u32(smem + C::kInfo + st * 64), lim, low, a.sinks, it.L, lane, nx);
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;"
                     :: "r"(smem_u32(&bars->empty[st])), "r"(kgs) : "memory");
    }
    w.sum_lanes();
    // ---- join the key groups: lw 2, 3 into 0, 1, then (one row group) 1 into 0
#pragma unroll 1
    for (int half = 2; half >= rgs; half >>= 1) {
      if (lw >= half && lw < 2 * half) w.put(so + (lw - half) * 16 * D, ss + (lw - half) * 16, lane, nx);
      if (!meet()) return;
      if (lw < half) w.join(so + lw * 16 * D, ss + lw * 16, lane, nx);
      if (!meet()) return;
    }
    const bool whole = it.pieces == 1;
    if (lk == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = rbase + 8 * x, c = lane & 3;
        if (row >= a.r) continue;
        if (whole) {
          const int j = row / a.T, t = row - j * a.T, h = it.hk * a.G + j;
          const float inv = inverse(w.l[x]);
          T* dst = static_cast<T*>(a.o) + (int64_t)it.b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + c * (D / 4);
          // columns t of the first and of the second half of this thread's D / 4
#pragma unroll
          for (int y = 0; y < D / 32; ++y) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = 8 * y + 2 * i, hf = col / (D / 8), tt = col % (D / 8);
              u[i] = Cvt<T>::pack(w.o[tt][2 * x + hf] * inv, w.o[tt + 1][2 * x + hf] * inv);
            }
            reinterpret_cast<uint4*>(dst)[y] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (c == 0) a.lse[((size_t)it.b * a.H + h) * a.T + t] = lse_of(w.m[x], w.l[x]);
        } else {
          const size_t at = (size_t)it.slot * a.tile + rg * 16 + (lane >> 2) + 8 * x;
          float4* dst = reinterpret_cast<float4*>(a.part + at * D + c * (D / 4));
#pragma unroll
          for (int y = 0; y < D / 16; ++y) {
            const int hf = 4 * y / (D / 8), tt = 4 * y % (D / 8);
            dst[y] = make_float4(w.o[tt][2 * x + hf], w.o[tt + 1][2 * x + hf], w.o[tt + 2][2 * x + hf], w.o[tt + 3][2 * x + hf]);
          }
          if (c == 0) a.stat[at] = make_float2(w.m[x], w.l[x]);
        }
      }
    }
    if (whole) continue;
    // ---- rows that were cut: the last CTA to leave its part joins them, in the CTAs' order
    __threadfence();
    if (!meet()) return;
    if (threadIdx.x == 0) bars->last = atomicAdd(a.count + it.c0, 1) == it.pieces - 1;
    if (!meet()) return;
    if (!*(volatile int*)&bars->last) continue;
    __threadfence();
    constexpr int E = D / 32;                     // columns of a lane
    const int have = min(a.tile, a.r - it.rt * a.tile);
    for (int row = warp; row < have; row += 4) {
      float m = -INFINITY, l = 0.f, acc[E] = {};
      for (int s0 = 0; s0 < it.pieces; s0 += 32) {
        // piece s is in CTA c0 + s: the first one's rows begin there, the others' before
        const int cnt = min(32, it.pieces - s0);
        auto at = [&](int s) { return (size_t)(2 * (it.c0 + s0 + s) + (s0 + s == 0 ? 1 : 0)) * a.tile + row; };
        const float2 st = lane < cnt ? __ldcg(a.stat + at(lane)) : make_float2(-INFINITY, 0.f);
        float mx = st.x;
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float m_new = fmaxf(m, mx), old = m == -INFINITY ? 0.f : ex2(m - m_new);
        const float f = st.x == -INFINITY ? 0.f : ex2(st.x - m_new);
        m = m_new;
        float fl = f * st.y;
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, y);
        l = l * old + fl;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
        for (int s1 = 0; s1 < cnt; s1 += 8) {
          float v[8][E];
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const float* src = a.part + at(min(s1 + s, cnt - 1)) * D + lane * E;
            if constexpr (E == 2) {
              const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
              v[s][0] = u.x; v[s][1] = u.y;
            } else {
              const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
              v[s][0] = u.x; v[s][1] = u.y; v[s][2] = u.z; v[s][3] = u.w;
            }
          }
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
      const int rr = it.rt * a.tile + row, j = rr / a.T, t = rr - j * a.T, h = it.hk * a.G + j;
      const float inv = inverse(l);
      uint32_t u[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) u[e] = Cvt<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      T* dst = static_cast<T*>(a.o) + (int64_t)it.b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + lane * E;
      if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = u[0];
      else *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
      if (lane == 0) a.lse[((size_t)it.b * a.H + h) * a.T + t] = lse_of(m, l);
    }
  }
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
int tile_of(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct CLayout { size_t count, stat, part, pre, total; };
CLayout clayout(int rows, int d, int B) {
  CLayout L;
  const size_t n = 2 * (size_t)kCMax * tile_of(rows);
  L.count = 256;                                 // behind the status word, cleared with it
  L.stat = al256(L.count + kCMax * sizeof(int));
  L.part = L.stat + al256(n * sizeof(float2));
  L.pre = L.part + al256(n * d * sizeof(float));
  L.total = L.pre + (B > kPreMax ? al256(((size_t)B + 1) * sizeof(int)) : 0);
  return L;
}

template <typename T, int D>
cudaError_t launch_c(const CUtensorMap& mk, const CUtensorMap& mv, const Cache8Args& a, cudaStream_t s) {
  using C = CCfg<D>;
  auto kern = cache8_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if (a.B > kPreMax) {
    cache8_plan_kernel<C::KS><<<1, 1024, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const long long most = (long long)a.B * a.Hkv * a.tiles * ((a.cap + C::KS - 1) / C::KS);
  const unsigned grid = (unsigned)std::min<long long>(std::max<long long>(most, 1), std::min(kCMax, C::kCtas * std::max(sms, 1)));
  kern<<<grid, kCThreads, C::kBytes, s>>>(mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

size_t cache8_workspace(const fa_cache8_params* p) { return clayout(p->H / p->H_kv * p->T, p->d, p->B).total; }

cudaError_t launch_cache8_fwd(int dtype, int d, const CUtensorMap& mk, const CUtensorMap& mv, Cache8Args a, uint8_t* ws,
                              cudaStream_t s) {
  a.r = a.G * a.T;
  a.tile = tile_of(a.r);
  a.tiles = (a.r + a.tile - 1) / a.tile;
  const CLayout L = clayout(a.r, d, a.B);
  a.status = reinterpret_cast<int*>(ws);
  a.count = reinterpret_cast<int*>(ws + L.count);
  a.stat = reinterpret_cast<float2*>(ws + L.stat);
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.pre = reinterpret_cast<int*>(ws + L.pre);
  cudaError_t e = cudaMemsetAsync(ws, 0, L.count + kCMax * sizeof(int), s);
  if (e != cudaSuccess) return e;
  using B16 = __nv_bfloat16;
  const bool bf = dtype == FA_DT_BF16;
  if (d == 128) return bf ? launch_c<B16, 128>(mk, mv, a, s) : launch_c<__half, 128>(mk, mv, a, s);
  return bf ? launch_c<B16, 64>(mk, mv, a, s) : launch_c<__half, 64>(mk, mv, a, s);
}

}  // namespace fa
