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
// read once for all G T query rows of a K/V head.  Measured: 64 sequences of 1 to
// 8,191 keys, 16 heads of 64 (537 MB) 97 us, 5.5 TB/s (0.81 of the copy rate); 8 heads
// of 128, 99 us; 8 query heads a K/V head 101 and 105 us; 6 sequences of 5 tokens and 12
// heads, window 4,096 of up to 23,400 keys (32 MB) 16 us with the counters' clearing: 4
// are the lengths', pages' and scales' latencies before the first keys, 5 the joins.
//
// Work.  The 64-key (d = 128: 32-key) units that the batch's rows see, sequence by
// sequence and K/V head by K/V head, form one line; every persistent CTA takes an
// equal piece of it, so that ragged lengths cost no balance.  Rows whose units all
// lie in one CTA leave O and the logsumexp; where they are cut, the CTAs leave
// partial rows in float32 and the last one to finish joins them in their order.
// The lengths stay on the device: each CTA sums the units itself (above kPreMax
// sequences the small kernel that clears the counters does).  In a CTA warp 4 looks up pages and scales a
// stage a lane, 32 stages ahead, and streams codes with TMA; warps 0-3 take 8 or 16
// rows each: a tile of 8 or 16 / 32 / 64 rows is split into 1 / 2 / 4 row groups, the
// stages among 4 / 2 / 1 key groups, which join at the end of their rows.
#include <algorithm>
#include <climits>
#include <cmath>

#include "cache8_plan.cuh"

namespace fa {
namespace {

constexpr int kCThreads = 160;   // warps 0-3 compute, 4 looks up and loads
constexpr float kLn2 = 0.6931471805599453f;
// The weights' sums, weights over V scales, are held times 2^-28, so that scales down to 2^-126, the smallest that
// rows are written with, leave them finite; scales up to 2^98 leave them normal.
constexpr float kSum = 0x1p-28f, kSumLog2 = -28.f;
// A page of zeros may have the scale 0: it counts as 2^-64, so that it does not set the reference that other pages'
// weights are rounded against, and its weights still reach the sums.
constexpr float kZeroPage = 0x1p-64f, kZeroPageLog2 = -64.f;

// x = 2^e f with f in [1, 2), x > 0 normal.  lg2 is off by up to 2^-22 of its result: for a sum, or a scale, far from 1
// that is more than the logsumexp may be off by; e + lg2(f) is exact for powers of two.
struct Power {
  float e, f;
  __device__ __forceinline__ explicit Power(float x) {
    const uint32_t u = __float_as_uint(x);
    e = (float)((int)(u >> 23) - 127);
    f = __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u);
  }
  __device__ __forceinline__ float log2() const { return e + lg2(f); }
};

template <int D, int NX> struct CCfg {
  static constexpr int RW = 8 * NX;              // query rows of a warp
  static constexpr int KS = D == 64 ? 64 : 32;   // keys of a stage
  static constexpr int NG = KS / 16;             // 16-key groups of a stage, each within one page
  static constexpr int kTile = KS * D;           // bytes of K (of V) of one stage
  static constexpr int NS = 8;                   // a multiple of 4: with split keys stage s is warp s % 4's
  static constexpr int kCtas = D == 64 ? 3 : NX == 1 ? 3 : 2;   // CTAs per SM
  static constexpr int kK = 0;
  static constexpr int kV = NS * kTile;
  static constexpr int kJoin = 2 * NS * kTile;   // [2][RW][D] O and [2][RW] statistics of two warps
  static constexpr int kInfo = kJoin + 2 * RW * (D * 4 + 8);
  static constexpr int kPre = kInfo + NS * 64;
  static constexpr int kItem = kPre + (kPreMax + 4) * 8;
  static constexpr int kBar = kItem + 256;
  static constexpr int kBytes = kBar + 288;
};
template <int D, int NX> constexpr bool fits() { return CCfg<D, NX>::kCtas * (CCfg<D, NX>::kBytes + 1024) <= 233472; }
static_assert(fits<64, 1>() && fits<64, 2>() && fits<128, 1>() && fits<128, 2>(), "the CTAs of one SM exceed its shared memory");
static_assert(CCfg<64, 1>::kCtas * 152 <= kCMax && CCfg<128, 1>::kCtas * 152 <= kCMax, "more CTAs than partial rows");
static_assert(kCMax <= 32 * kGroup, "more groups of pieces than a warp joins");

struct CBars {
  uint64_t full[8], empty[8];
  uint64_t item_full[8], item_empty[8], join;
  int abort, last;
};
static_assert(sizeof(CBars) <= 288, "barrier block overflows its shared-memory slot");

// What the compute warps need of a stage: per 16 keys the K scale, log2 of the V
// scale and its inverse (times kSum), and the first key.  A group whose page is absent has the
// factors 0, -inf and 0: its weights are zero.
struct __align__(16) CInfo { float kf[4], ve[4], vi[4]; int key0, pad[3]; };
static_assert(sizeof(CInfo) == 64, "a stage's record");

struct CItem {
  int b, hk, rt, tokens;   // rows of tile rt of K/V head hk of sequence b
  int nt;                  // stages in this CTA; -1: no more
  int n;                   // units of these rows, the first at s0 of the line
  long long s0;
};
static_assert(sizeof(CItem) == 32, "a mailbox slot");

__device__ __forceinline__ int tokens_of(const Cache8Args& a, int b) { return max(0, a.lens[b]); }
__device__ __forceinline__ void widen(uint32_t four, uint32_t& lo, uint32_t& hi) {   // E4M3 codes -> halves, exact
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(four));
}
// Plain loads and products that are not volatile: the compiler may move them past one another.
__device__ __forceinline__ uint4 lds4(const uint8_t* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ uint2 lds2(const uint8_t* at) { return *reinterpret_cast<const uint2*>(at); }
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes the 8 x 8 matrix of halves whose row l / 4 lane l holds two columns of.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// State of 8 NX query rows in one warp.  The products are the transposed ones, S^T = K q^T and O^T = V^T P^T: the 16
// rows of their first operand are keys, then value columns, of which there are always enough, and the 8 columns of
// the second the query rows, of which decoding has 1 to 8.  (With the query rows first half of a product or more was
// empty, and the accumulators and q took twice the registers.)  Thread (n = lane / 4, c = lane % 4) has, of the scores,
// rows 2 c and 2 c + 1 against key n of every eight, and of O their columns n D/8 .. n D/8 + D/8 - 1; the weights turn
// from the first layout to the second operand's by movmatrix.  The products' inner order is free as long as both
// operands agree: a thread's K columns are 16 c .. 16 c + 15 (and 64 on).
template <int D, int NX> struct CRows {
  static constexpr int KS = CCfg<D, NX>::KS;
  uint32_t q[NX][D / 16][2];
  float o[NX][D / 16][4];        // [.][t][2 y + x]: column 2 t + y of the thread's, row 2 c + x
  float m[NX][2], l[NX][2];
  float rf[NX][2];               // what a score of the scaled q has to be multiplied by

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int z = 0; z < NX; ++z) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[z][t][e] = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[z][x] = -INFINITY;
        l[z][x] = 0.f;
      }
    }
  }
  // Row n of the z-th eight from `src` (nullptr: zeros), as halves: scaled by the power of two that brings its largest
  // value to 2^14 .. 2^15, so that bf16 loses nothing that float32 sums would keep.
  template <typename T> __device__ __forceinline__ void load_q(const T* src, int z, int lane, float sl2) {
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
    const float mine = sl2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
    for (int x = 0; x < 2; ++x) rf[z][x] = __shfl_sync(0xffffffffu, mine, (2 * (lane & 3) + x) * 4);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        q[z][i][e] = Cvt<__half>::pack(Cvt<T>::lo(raw[2 * i + e]) * f, Cvt<T>::hi(raw[2 * i + e]) * f);
  }
  // The keys of one stage.  lim, low: keys at or past lim, and below low unless below sinks, are hidden, per row; end: V
  // rows at or past it may hold anything.
  __device__ __forceinline__ void step(const uint8_t* sK, const uint8_t* sV, const uint8_t* info, const int (&lim)[NX][2],
                                       const int (&low)[NX][2], int sinks, int end, int lane) {
    const int n = lane >> 2, c = lane & 3, kr = key_of<D>(n >> 1, n & 1);
    float s[NX][KS / 16][4];
#pragma unroll
    for (int g = 0; g < KS / 16; ++g) {
#pragma unroll
      for (int z = 0; z < NX; ++z)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[z][g][e] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint8_t* at = sK + (16 * g + kr) * D + (D == 64 ? (c ^ ((kr >> 1) & 3)) << 4 : ((c + 4 * h) ^ kr) << 4);
        const uint4 w0 = lds4(at), w1 = lds4(at + 8 * D);
        const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t a[4];
          widen(a0[k], a[0], a[2]);
          widen(a1[k], a[1], a[3]);
#pragma unroll
          for (int z = 0; z < NX; ++z) mma(s[z][g], a, q[z][4 * h + k][0], q[z][4 * h + k][1]);
        }
      }
    }
    const uint4 kq = lds4(info), eq = lds4(info + 16), iq = lds4(info + 32);
    const float kf[4] = {__uint_as_float(kq.x), __uint_as_float(kq.y), __uint_as_float(kq.z), __uint_as_float(kq.w)};
    const float ve[4] = {__uint_as_float(eq.x), __uint_as_float(eq.y), __uint_as_float(eq.z), __uint_as_float(eq.w)};
    const float vi[4] = {__uint_as_float(iq.x), __uint_as_float(iq.y), __uint_as_float(iq.z), __uint_as_float(iq.w)};
    const int key0 = *reinterpret_cast<const int*>(info + 48);
    uint32_t p[NX][KS / 16][2];
    bool moved = false;
    float alpha[NX][2];
#pragma unroll
    for (int z = 0; z < NX; ++z) {
#pragma unroll
      for (int g = 0; g < KS / 16; ++g) {
        const float f0 = rf[z][0] * kf[g], f1 = rf[z][1] * kf[g];
        mul2(s[z][g][0], s[z][g][1], s[z][g][0], s[z][g][1], f0, f1);
        mul2(s[z][g][2], s[z][g][3], s[z][g][2], s[z][g][3], f0, f1);
      }
      if (key0 + KS > min(lim[z][0], lim[z][1]) || key0 < max(low[z][0], low[z][1])) {
#pragma unroll
        for (int g = 0; g < KS / 16; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 16 * g + 8 * (e >> 1) + kr;
            if (key >= lim[z][e & 1] || (key < low[z][e & 1] && key >= sinks)) s[z][g][e] = -INFINITY;
          }
      }
      // the reference maximum, of the weights times their V scales
      float nm[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < KS / 16; ++g) mx = fmaxf(mx, fmaxf(s[z][g][x], s[z][g][2 + x]) + ve[g]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        // moved only when it is exceeded by 2^8: any reference gives the same
        // quotient, and most steps skip the rescale
        const float m_new = mx > m[z][x] + 8.f ? mx : m[z][x];
        alpha[z][x] = 1.f;
        if (m_new != m[z][x]) {
          alpha[z][x] = m[z][x] == -INFINITY ? 0.f : ex2(m[z][x] - m_new);
          moved = true;
        }
        m[z][x] = m_new;
        nm[x] = m_new == -INFINITY ? 0.f : -m_new;
        l[z][x] *= alpha[z][x];
      }
      // weights to 16 bits (half a step of 2^-11 each); their sum stays unrounded
#pragma unroll
      for (int g = 0; g < KS / 16; ++g) {
        const float n0 = nm[0] + ve[g], n1 = nm[1] + ve[g];
        float a0 = s[z][g][0], a1 = s[z][g][1], b0 = s[z][g][2], b1 = s[z][g][3];
        add2(a0, a1, n0, n1);
        add2(b0, b1, n0, n1);
        a0 = ex2(a0); a1 = ex2(a1); b0 = ex2(b0); b1 = ex2(b1);
        p[z][g][0] = transposed(Cvt<__half>::pack(a0, a1));
        p[z][g][1] = transposed(Cvt<__half>::pack(b0, b1));
        add2(a0, a1, b0, b1);
        fma2(l[z][0], l[z][1], a0, a1, vi[g], vi[g], l[z][0], l[z][1]);
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int z = 0; z < NX; ++z)
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[z][t][e] *= alpha[z][e & 1];
    }
    if (key0 + KS > end) pv<true>(sV, p, end - key0, lane);
    else pv<false>(sV, p, 0, lane);
  }
  // V rows from `live` on are replaced by zeros (0 x NaN would not be 0)
  template <bool kTail>
  __device__ __forceinline__ void pv(const uint8_t* sV, const uint32_t (&p)[NX][KS / 16][2], int live, int lane) {
    const int n = lane >> 2, c = lane & 3;
    const int kb[2] = {key_of<D>(c, 0), key_of<D>(c, 1)};
    const uint8_t* at[2];
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
      uint32_t m[2] = {~0u, ~0u};
      if (kTail) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int k0 = 8 * (2 * g + y);
          m[y] = (k0 + kb[0] < live ? 0xFFFFu : 0u) | (k0 + kb[1] < live ? 0xFFFF0000u : 0u);
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {           // two columns at a time
          uint32_t a[4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            widen(__byte_perm(v[y][0][w], v[y][1][w], hf ? 0x7362 : 0x5140), a[2 * y], a[2 * y + 1]);
            if (kTail) {
              a[2 * y] &= m[y];
              a[2 * y + 1] &= m[y];
            }
          }
#pragma unroll
          for (int z = 0; z < NX; ++z) mma(o[z][2 * w + hf], a, p[z][g][0], p[z][g][1]);
        }
      }
    }
  }
  // float4 i of this thread's columns of row 8 z + 2 c + x, turned by the row so that eight lanes meet eight banks
  static __device__ __forceinline__ int place(int z, int x, int i, int lane) {
    constexpr int P = D / 32;
    const int n = lane >> 2, c = lane & 3;
    const int turn = D == 64 ? (c & 1) | (c & 2) << 1 : c;
    return (8 * z + 2 * c + x) * D + 4 * ((n * P + i + turn) & (D / 4 - 1));
  }
  __device__ __forceinline__ float4 columns(int z, int x, int i) const {
    return make_float4(o[z][2 * i][x], o[z][2 * i][2 + x], o[z][2 * i + 1][x], o[z][2 * i + 1][2 + x]);
  }
  __device__ __forceinline__ void put(float* so, float2* ss, int lane) const {
#pragma unroll
    for (int z = 0; z < NX; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) *reinterpret_cast<float4*>(so + place(z, x, i, lane)) = columns(z, x, i);
        if (lane < 4) ss[8 * z + 2 * lane + x] = make_float2(m[z][x], l[z][x]);
      }
  }
  __device__ __forceinline__ void join(const float* so, const float2* ss, int lane) {
#pragma unroll
    for (int z = 0; z < NX; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 st = ss[8 * z + 2 * (lane & 3) + x];
        const float m_new = fmaxf(m[z][x], st.x);
        // a row that is NaN has the maximum -inf; its sum stays NaN
        const float fa_ = m[z][x] == -INFINITY ? (l[z][x] != l[z][x] ? 1.f : 0.f) : ex2(m[z][x] - m_new);
        const float fb = st.x == -INFINITY ? (st.y != st.y ? 1.f : 0.f) : ex2(st.x - m_new);
        m[z][x] = m_new;
        l[z][x] = l[z][x] * fa_ + st.y * fb;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(so + place(z, x, i, lane));
          o[z][2 * i][x] = o[z][2 * i][x] * fa_ + v.x * fb;
          o[z][2 * i][2 + x] = o[z][2 * i][2 + x] * fa_ + v.y * fb;
          o[z][2 * i + 1][x] = o[z][2 * i + 1][x] * fa_ + v.z * fb;
          o[z][2 * i + 1][2 + x] = o[z][2 * i + 1][2 + x] * fa_ + v.w * fb;
        }
      }
  }
  __device__ __forceinline__ void sum_lanes() {
#pragma unroll
    for (int z = 0; z < NX; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[z][x] += __shfl_xor_sync(0xffffffffu, l[z][x], y);
  }
};

// logsumexp, and the factor of kSum O: a row that saw no key has l = 0, one with a NaN in it l = NaN
__device__ __forceinline__ float lse_of(float m, float l) {
  if (!(l > 0.f && l < INFINITY)) return l == 0.f ? -INFINITY : l;
  const Power p(l);
  // m, which the V scales move as they move the power, is rounded next to neither 28 nor the power
  return ((m + (p.e - kSumLog2)) + lg2(p.f)) * kLn2;
}
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : l; }

// Clears the status word and the counters, and, for batches whose prefix sums do not fit the kernel's shared memory,
// sums the units of the line, and the sequences with keys, before each sequence.  One CTA.
template <int KS> __global__ void __launch_bounds__(1024) cache8_plan_kernel(const Cache8Args a) {
  __shared__ int2 warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 carry = make_int2(0, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) *a.status = 0;
  for (int i = threadIdx.x; i < 3 * kCMax; i += blockDim.x) a.count[i] = 0;
  if (a.B <= kPreMax) return;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int n = b < a.B ? units_of<KS>(a, tokens_of(a, b)).line() : 0;
    int s = n;
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, s, y);
      if (lane >= y) s += up;
    }
    const unsigned some = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 31) warps[warp] = make_int2(s, __popc(some));
    __syncthreads();
    int2 before = carry;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) { before.x += warps[w].x; before.y += warps[w].y; }
      carry.x += warps[w].x;
      carry.y += warps[w].y;
    }
    if (b < a.B) a.pre[b] = make_int2(before.x + s - n, before.y + __popc(some & ((1u << lane) - 1u)));
    __syncthreads();
  }
  if (threadIdx.x == 0) a.pre[a.B] = carry;
}

template <typename T, int D, int NX>
__global__ void __launch_bounds__(kCThreads, (CCfg<D, NX>::kCtas))
cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ Cache8Args a) {
  using C = CCfg<D, NX>;
  constexpr int NS = C::NS, KS = C::KS, RW = C::RW;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {       // the swizzled tiles: see diff_fwd.cu
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) atomicExch(a.status, (int)FA_ERR_CUDA);
    return;
  }
  CBars* bars = reinterpret_cast<CBars*>(smem + C::kBar);
  int2* const own = reinterpret_cast<int2*>(smem + C::kPre);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WaitCtl ctl{a.status, &bars->abort, kWaitSleepNs};
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->full[s], 2);            // the copies announced, the record written
      mbar_init(&bars->empty[s], 4);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 4);
    }
    mbar_init(&bars->join, 4);
    bars->abort = 0;
    bars->last = 0;
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- units before each sequence: warp 4, whose copies wait for them, sums them; the others meet it behind that
  const int2* pre = a.B <= kPreMax ? own : a.pre;
  if (warp == 4 && a.B <= kPreMax) {
    int2 carry = make_int2(0, 0);
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int n = b0 + lane < a.B ? units_of<KS>(a, tokens_of(a, b0 + lane)).line() : 0;
      int s = n;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, s, y);
        if (lane >= y) s += up;
      }
      const unsigned some = __ballot_sync(0xffffffffu, n > 0);
      if (b0 + lane < a.B) own[b0 + lane] = make_int2(carry.x + s - n, carry.y + __popc(some & ((1u << lane) - 1u)));
      carry.x += __shfl_sync(0xffffffffu, s, 31);
      carry.y += __popc(some);
    }
    if (lane == 0) own[a.B] = carry;
    __syncwarp();
  }
  if (warp == 4) named_bar_arrive(1, kCThreads);
  else named_bar_sync(1, kCThreads);
  const int HS = a.Hkv * a.tiles;
  Share sh;
  const long long X = (long long)pre[a.B].x * HS;
  sh.cut(X, (int)max(1ll, min((long long)gridDim.x, X)));
  const int me = blockIdx.x;
  const long long xb = me < sh.C ? sh.begin(me) : sh.X, xe = me < sh.C ? sh.begin(me + 1) : sh.X;

  if (warp == 4) {
    // ===================== pages, scales and TMA =====================
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    // the keys' units (without the kItemUnits in front of each sequence's rows) before sequence b
    auto real = [&](int b) -> long long { return (long long)(pre[b].x - kItemUnits * pre[b].y) * HS; };
    // ... and before unit x of the line; the last sequence that begins at or before it has keys.  The CTA's key units
    // are rb .. re - 1, of sequences bb .. be.
    long long rb = real(a.B), re = rb;
    int bb = 0, be = a.B - 1;
    if (xb < sh.X) {
      const long long x = lane & 1 ? xe : xb;        // lanes side by side, for both ends
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)pre[mid].x * HS <= x) lo = mid; else hi = mid;
      }
      const int line = pre[lo + 1].x - pre[lo].x;
      const unsigned y = (unsigned)(x - (long long)pre[lo].x * HS), seg = line > 0 ? y / (unsigned)line : 0u;    // < 2^31 (api.cu)
      const long long r = real(lo) + (line > 0 ? (long long)seg * (line - kItemUnits) +
                                                     max(0, (int)(y - seg * (unsigned)line) - kItemUnits) : 0);
      rb = __shfl_sync(0xffffffffu, r, 0);
      bb = __shfl_sync(0xffffffffu, lo, 0);
      re = __shfl_sync(0xffffffffu, r, 1);
      be = __shfl_sync(0xffffffffu, lo, 1);
      if (xe == sh.X) {
        re = real(a.B);
        be = a.B - 1;
      }
    }
    if (rb >= re) {
      if (lane == 0) {
        reinterpret_cast<CItem*>(smem + C::kItem)->nt = -1;
        mbar_arrive(&bars->item_full[0]);
      }
      return;
    }
    // one stage a lane
    struct Look {
      CItem it;
      bool real, first;      // a stage; the first one of its rows in this CTA
      int key0, id[C::NG];
    };
    auto look = [&](long long x, Look& k) {          // key unit x
      k.key0 = 0;
      k.real = k.first = false;
#pragma unroll
      for (int g = 0; g < C::NG; ++g) k.id[g] = -1;
      if (x >= re) return;
      int lo = bb, hi = be + 1;              // the sequence of unit x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (real(mid) <= x) lo = mid; else hi = mid;
      }
      const int tokens = tokens_of(a, lo), L = min(tokens, a.cap);
      const Units un = units_of<KS>(a, tokens);
      const unsigned y = (unsigned)(x - real(lo)), seg = y / (unsigned)un.n;
      const int i = (int)(y - seg * (unsigned)un.n);
      const long long s0 = (long long)pre[lo].x * HS + (long long)seg * un.line() + kItemUnits;
      k.it.b = lo;
      k.it.hk = (int)seg / a.tiles;
      k.it.rt = (int)seg - k.it.hk * a.tiles;
      k.it.tokens = tokens;
      k.it.nt = (int)min((long long)(un.n - i), re - x);
      k.it.n = un.n;
      k.it.s0 = s0;
      k.real = true;
      k.first = i == 0 || x == rb;
      k.key0 = (i < un.ns ? i : i + un.skip) * KS;
      const int32_t* row = a.table + (int64_t)lo * a.table_stride;
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        const int key = k.key0 + 16 * g;
        if (key < L) k.id[g] = row[key >> a.lg];
      }
    };
    float ks[C::NG], vs[C::NG];              // scales on their way
    auto scales = [&](const Look& k) {
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        ks[g] = vs[g] = -1.f;
        if ((unsigned)k.id[g] < (unsigned)a.pages) {
          const size_t at = (size_t)k.id[g] * a.Hkv + k.it.hk;
          ks[g] = a.ks[at];
          vs[g] = a.vs[at];
        }
      }
    };
    const int rows = min(a.page, KS), boxes = KS / rows;
    const uint32_t box = (uint32_t)rows * D;
    Look cur, nxt;
    look(rb + lane, cur);
    scales(cur);
    int kf = 0;                              // items published
    bool ok = true;
    int g0 = 0;                              // stages loaded
    for (long long x = rb; x < re && ok; x += 32) {
      // the next 32 stages' pages are looked up while these are on their way
      const int cnt = (int)min(32ll, re - x);
      // Four lanes issue their stages side by side: a stage is a chain of some 600 cycles in its lane.  Their items
      // find room in the mailbox, whose eight slots outlast what two batches can publish: the oldest of the eight
      // was published two batches ago, and all stages before it are loaded.
      for (int i0 = 0; i0 < cnt; i0 += 4) {
        const bool mine = (lane >> 2) == (i0 >> 2) && cur.real;
        const unsigned reals = __ballot_sync(0xffffffffu, mine), below = (1u << lane) - 1u;
        const int n = __popc(reals);
        const unsigned firsts = __ballot_sync(0xffffffffu, mine && cur.first);
        // all lanes wait for all four stages: lanes that waited apart would go on apart
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (g0 + y >= NS && y < n) ok = ok && mbar_wait(&bars->empty[(g0 + y) % NS], (uint32_t)((g0 + y) / NS - 1) & 1u, ctl);
        if (mine) {
          const int gi = g0 + __popc(reals & below), st = gi % NS;
          if (cur.first) {
            const int kk = kf + __popc(firsts & below), slot = kk & 7;
            ok = kk < 8 || mbar_wait(&bars->item_empty[slot], (uint32_t)((kk >> 3) - 1) & 1u, ctl);
            if (ok) {
              *reinterpret_cast<CItem*>(smem + C::kItem + slot * sizeof(CItem)) = cur.it;
              mbar_arrive(&bars->item_full[slot]);
            }
          }
          if (ok) {
            // boxes behind the last row are left out: what they would bring is hidden
            const int nb = min(boxes, (min(cur.it.tokens, a.cap) - cur.key0 + rows - 1) / rows);
            mbar_expect_tx(&bars->full[st], 2 * box * nb);
#pragma unroll
            for (int y = 0; y < C::NG; ++y) {
              if (y >= nb) break;
              const int key = cur.key0 + y * rows;
              int id = boxes == 1 ? cur.id[0] : boxes == C::NG ? cur.id[y] : cur.id[(2 * y) & (C::NG - 1)];
              if ((unsigned)id >= (unsigned)a.pages) id = a.pages;      // behind the last page: the copy fills in zeros
              tma_load_4d(smem + C::kK + st * C::kTile + y * box, &tmK, &bars->full[st], 0, key & (a.page - 1), cur.it.hk, id);
              tma_load_4d(smem + C::kV + st * C::kTile + y * box, &tmV, &bars->full[st], 0, key & (a.page - 1), cur.it.hk, id);
            }
            CInfo inf;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float k = g < C::NG ? ks[g < C::NG ? g : 0] : -1.f, v = g < C::NG ? vs[g < C::NG ? g : 0] : -1.f;
              const bool there = g < C::NG && (unsigned)cur.id[g < C::NG ? g : 0] < (unsigned)a.pages;
              inf.kf[g] = there ? k : 0.f;
              inf.ve[g] = there ? (v == 0.f ? kZeroPageLog2 : Power(v).log2()) : -INFINITY;
              inf.vi[g] = there ? kSum / (v == 0.f ? kZeroPage : v) : 0.f;
            }
            inf.key0 = cur.key0;
            *reinterpret_cast<CInfo*>(smem + C::kInfo + st * 64) = inf;
            mbar_arrive(&bars->full[st]);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        kf += __popc(firsts);
        g0 += n;
        if (i0 == 0) look(x + 32 + lane, nxt);
      }
      cur = nxt;
      scales(cur);
    }
    if (lane == 0) {
      if (ok && (kf < 8 || mbar_wait(&bars->item_empty[kf & 7], (uint32_t)((kf >> 3) - 1) & 1u, ctl))) {
        reinterpret_cast<CItem*>(smem + C::kItem + (kf & 7) * sizeof(CItem))->nt = -1;
        mbar_arrive(&bars->item_full[kf & 7]);
      }
      // no load may still be writing shared memory when the CTA ends
      for (int j = max(0, g0 - NS); j < g0; ++j) mbar_wait(&bars->full[j % NS], (uint32_t)(j / NS) & 1u, ctl);
    }
    return;
  }

  // ===================== compute warps =====================
  // sequences without keys
  for (int b = me; b < a.B; b += gridDim.x) {
    if (pre[b + 1].x > pre[b].x) continue;
    for (int i = threadIdx.x; i < a.H * a.T * (D / 8); i += 128) {
      const int row = i / (D / 8), h = row / a.T, t = row - h * a.T;
      T* dst = static_cast<T*>(a.o) + (int64_t)b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + (i % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
      if (i % (D / 8) == 0) a.lse[(size_t)b * a.H * a.T + row] = -INFINITY;
    }
  }
  float* so = reinterpret_cast<float*>(smem + C::kJoin);              // [2][RW][D]
  float2* ss = reinterpret_cast<float2*>(so + 2 * RW * D);             // [2][RW]
  // barrier of the four compute warps: bounded like every wait
  int nj = 0;
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->join);
    return __all_sync(0xffffffffu, mbar_wait(&bars->join, (uint32_t)nj++ & 1u, ctl));
  };
  // warp = (key group) * rgs + (row group)
  const int rgs = a.tile / RW, kgs = 4 / rgs;
  const int rg = warp & (rgs - 1), kg = warp / rgs;
  int g = 0;
  for (int kc = 0;; ++kc) {
    const int slot = kc & 7;
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->item_full[slot], (uint32_t)(kc >> 3) & 1u, ctl))) return;
    const CItem it = *reinterpret_cast<const CItem*>(smem + C::kItem + slot * sizeof(CItem));
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    if (it.nt < 0) return;
    // this warp's key group counted from the item's first stage: the joins go by it
    const int lk = (kg - g) & (kgs - 1), lw = lk * rgs + rg;
    const int r0 = it.rt * a.tile + rg * RW;                          // first row of this warp's
    // Stage t of the item is key group t % kgs's: of an item with fewer stages than key groups some have none, of a
    // tile with fewer rows some warps.  They fetch no q and go on to the next item; the joins leave them out.
    const bool busy = lk < it.nt && r0 < a.r;
    const int L = min(it.tokens, a.cap);                              // rows; the positions go by the tokens
    CRows<D, NX> w;
    w.init();
    int lim[NX][2], low[NX][2];
#pragma unroll
    for (int z = 0; z < NX; ++z) {
      const int row = r0 + 8 * z + (lane >> 2);
      const T* src = nullptr;
      if (busy && row < a.r) {
        const int j = row / a.T, t = row - j * a.T;
        src = static_cast<const T*>(a.q) + (int64_t)it.b * a.qs.b + (int64_t)(it.hk * a.G + j) * a.qs.h + (int64_t)t * a.qs.n;
      }
      if (busy) w.load_q(src, z, lane, a.scale_log2);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rx = r0 + 8 * z + 2 * (lane & 3) + x;
        const int p = it.tokens - a.T + rx % a.T;
        lim[z][x] = rx < a.r ? min(L, p + 1) : INT_MAX;               // rows that do not exist mask nothing
        low[z][x] = rx < a.r && a.window > 0 ? first_seen(a, p) : 0;
      }
    }
    for (int t = 0; t < it.nt; ++t, ++g) {
      const int st = g % NS;
      if ((st & (kgs - 1)) != kg) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[st], (uint32_t)(g / NS) & 1u, ctl))) return;
      if (busy)
        w.step(smem + C::kK + st * C::kTile, smem + C::kV + st * C::kTile, smem + C::kInfo + st * 64, lim, low, a.sinks, L, lane);
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;"
                     :: "r"(smem_u32(&bars->empty[st])), "r"(kgs) : "memory");
    }
    if (busy) w.sum_lanes();
    // ---- join the key groups: lw 2, 3 into 0, 1, then (one row group) 1 into 0; not the rounds in which no group
    //      that would be joined has stages
#pragma unroll 1
    for (int half = 2; half >= rgs; half >>= 1) {
      const int groups = half / rgs;
      if (it.nt <= groups) continue;
      if (busy && lw >= half && lw < 2 * half) w.put(so + (lw - half) * RW * D, ss + (lw - half) * RW, lane);
      if (!meet()) return;
      if (busy && lw < half && lk + groups < it.nt) w.join(so + lw * RW * D, ss + lw * RW, lane);
      if (!meet()) return;
    }
    const bool whole = it.s0 >= xb && it.s0 + it.n <= xe;
    if (busy && lk == 0) {
#pragma unroll
      for (int z = 0; z < NX; ++z)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = r0 + 8 * z + 2 * (lane & 3) + x, n = lane >> 2;
          if (row >= a.r) continue;
          if (whole) {
            const int j = row / a.T, t = row - j * a.T, h = it.hk * a.G + j;
            const float inv = inverse(w.l[z][x]);
            T* dst = static_cast<T*>(a.o) + (int64_t)it.b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + n * (D / 8);
#pragma unroll
            for (int y = 0; y < D / 64; ++y) {
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) u[i] = Cvt<T>::pack(w.o[z][4 * y + i][x] * kSum * inv, w.o[z][4 * y + i][2 + x] * kSum * inv);
              reinterpret_cast<uint4*>(dst)[y] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            if (n == 0) a.lse[((size_t)it.b * a.H + h) * a.T + t] = lse_of(w.m[z][x], w.l[z][x]);
          } else {
            // begun here, or by a CTA before
            const size_t at = (size_t)(2 * me + (it.s0 >= xb ? 1 : 0)) * a.tile + (row - it.rt * a.tile);
            float4* dst = reinterpret_cast<float4*>(a.part + at * D + n * (D / 8));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) dst[i] = w.columns(z, x, i);
            if (n == 0) a.stat[at] = make_float2(w.m[z][x], w.l[z][x]);
          }
        }
    }
    if (whole) continue;
    // ---- rows that were cut: of every kGroup pieces the last CTA to leave its own joins them, of all groups the last
    //      one those; in the CTAs' order, whoever is last
    const int c0 = sh.owner(it.s0), pieces = sh.owner(it.s0 + it.n - 1) - c0 + 1;
    auto slot_of = [&](int piece) { return piece_slot(c0, piece); };
    auto arrive_last = [&](int* count, int of, bool& ok) -> bool {
      __threadfence();
      if (!(ok = meet())) return false;
      if (threadIdx.x == 0) bars->last = atomicAdd(count, 1) == of - 1;
      if (!(ok = meet())) return false;
      const bool last = *(volatile int*)&bars->last != 0;
      __threadfence();
      return last;
    };
    // rows of `cnt` <= 32 pieces, one every `step` from piece `from` on, into the first one's place or (final) O
    auto join_pieces = [&](int from, int step, int cnt, bool final) {
      // A warp a row, D / 32 columns a lane; the pieces' statistics side by side, then kGroup pieces' rows at a time.
      // Two rows at a time join faster and take registers that slow the loop above by 13 %, as a function of its own
      // does, by 20 %.
      constexpr int E = D / 32;
      const int have = min(a.tile, a.r - it.rt * a.tile);
      for (int row = warp; row < have; row += 4) {
        auto at = [&](int s) { return (size_t)slot_of(from + s * step) * a.tile + row; };
        float v[kGroup][E];
        auto fetch = [&](int s1) {
#pragma unroll
          for (int s = 0; s < kGroup; ++s) {
            const float* src = a.part + at(min(s1 + s, cnt - 1)) * D + lane * E;
            if constexpr (E == 2) {
              const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
              v[s][0] = u.x; v[s][1] = u.y;
            } else {
              const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
              v[s][0] = u.x; v[s][1] = u.y; v[s][2] = u.z; v[s][3] = u.w;
            }
          }
        };
        fetch(0);
        const float2 st = lane < cnt ? __ldcg(a.stat + at(lane)) : make_float2(-INFINITY, 0.f);
        float m = st.x;
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
        // a row that is NaN in a piece has the maximum -inf there and a NaN for its sum, which stays
        const float f = st.x == -INFINITY ? (st.y != st.y ? 1.f : 0.f) : ex2(st.x - m);
        float l = f * st.y, acc[E] = {};
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
#pragma unroll 1
        for (int s1 = 0; s1 < cnt; s1 += kGroup) {
          if (s1 > 0) fetch(s1);
#pragma unroll
          for (int s = 0; s < kGroup; ++s) {
            const float fs = __shfl_sync(0xffffffffu, f, (s1 + s) & 31);
            if (s1 + s < cnt) {
#pragma unroll
              for (int e = 0; e < E; ++e) acc[e] += fs * v[s][e];
            }
          }
        }
        if (!final) {
          float* dst = a.part + at(0) * D + lane * E;
          if constexpr (E == 2) *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
          else *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (lane == 0) a.stat[at(0)] = make_float2(m, l);
          continue;
        }
        const int rr = it.rt * a.tile + row, j = rr / a.T, t = rr - j * a.T, h = it.hk * a.G + j;
        const float inv = inverse(l);
        uint32_t u[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) u[e] = Cvt<T>::pack(acc[2 * e] * kSum * inv, acc[2 * e + 1] * kSum * inv);
        T* dst = static_cast<T*>(a.o) + (int64_t)it.b * a.os.b + (int64_t)h * a.os.h + (int64_t)t * a.os.n + lane * E;
        if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = u[0];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
        if (lane == 0) a.lse[((size_t)it.b * a.H + h) * a.T + t] = lse_of(m, l);
      }
    };
    bool ok = true;
    const int mine = me - c0, first = mine / kGroup * kGroup, cnt = min(kGroup, pieces - first);
    // counters: of the group that begins at a CTA, by which of its two places that is, and of all groups
    if (!arrive_last(a.count + slot_of(first), cnt, ok)) {
      if (!ok) return;
      continue;
    }
    join_pieces(first, 1, cnt, pieces <= kGroup);
    if (pieces <= kGroup) continue;
    const int groups = (pieces + kGroup - 1) / kGroup;
    if (!arrive_last(a.count + 2 * kCMax + c0, groups, ok)) {
      if (!ok) return;
      continue;
    }
    join_pieces(0, kGroup, groups, true);
  }
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
int tile_of(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct CLayout { size_t count, stat, part, pre, total; };
CLayout clayout(int rows, int d, int B) {
  CLayout L;
  const size_t n = 2 * (size_t)kCMax * tile_of(rows);
  L.count = 256;                                 // behind the status word, cleared with it
  L.stat = al256(L.count + 3 * kCMax * sizeof(int));
  L.part = L.stat + al256(n * sizeof(float2));
  L.pre = L.part + al256(n * d * sizeof(float));
  L.total = L.pre + (B > kPreMax ? al256(((size_t)B + 1) * sizeof(int2)) : 0);
  return L;
}

template <typename T, int D, int NX>
cudaError_t launch_n(const CUtensorMap& mk, const CUtensorMap& mv, const Cache8Args& a, cudaStream_t s) {
  using C = CCfg<D, NX>;
  auto kern = cache8_kernel<T, D, NX>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // Both launches begin over the end of the kernel before them (griddepcontrol.wait): about 1 us less than a clear and
  // a plain launch.
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(1);
  c.blockDim = dim3(a.B > kPreMax ? 1024 : 256);
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&c, cache8_plan_kernel<C::KS>, a)) != cudaSuccess) return e;
  const long long most = (long long)a.B * a.Hkv * a.tiles * ((a.cap + C::KS - 1) / C::KS);
  const unsigned grid = (unsigned)std::min<long long>(std::max<long long>(most, 1), std::min(kCMax, C::kCtas * std::max(sms, 1)));
  c.gridDim = dim3(grid);
  c.blockDim = dim3(kCThreads);
  c.dynamicSmemBytes = C::kBytes;
  return cudaLaunchKernelEx(&c, kern, mk, mv, a);
}

template <typename T, int D>
cudaError_t launch_c(const CUtensorMap& mk, const CUtensorMap& mv, const Cache8Args& a, cudaStream_t s) {
  return a.tile == 8 ? launch_n<T, D, 1>(mk, mv, a, s) : launch_n<T, D, 2>(mk, mv, a, s);
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
  a.pre = reinterpret_cast<int2*>(ws + L.pre);
  using B16 = __nv_bfloat16;
  const bool bf = dtype == FA_DT_BF16;
  if (d == 128) return bf ? launch_c<B16, 128>(mk, mv, a, s) : launch_c<__half, 128>(mk, mv, a, s);
  return bf ? launch_c<B16, 64>(mk, mv, a, s) : launch_c<__half, 64>(mk, mv, a, s);
}

}  // namespace fa
