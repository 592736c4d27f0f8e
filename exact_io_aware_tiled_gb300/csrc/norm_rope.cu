// norm_rope.cu -- q and k normalised for each head and rotated by their
// positions in one pass, and the gradients of that.
//
// Mathematics.  A row x of d columns (one token of one head) becomes
//     h = x r,  r = 1 / sqrt(mean(x^2) + eps),   y = R_p (w o h),
// with w the d weights that all heads of q (of k) share and R_p the rotation of
// rope.cu.  For the gradient dy of y:
//     dz = R_p^T dy,  g = w o dz,
//     dx = r g - x r^3 (g . x) / d,   dw = sum over rows of dz o h.
// x^2 and g . x do not need each other, so one round of shuffles sums both.  r
// is made again from x instead of being kept: x has to be read anyway.
//
// What bounds it: HBM.  The forward pass reads and writes each element once, the
// backward reads x and dy and writes dx.  As in rope.cu a thread owns 16 (8)
// columns of one token and walks over the heads, so that a sine and cosine
// serve them all; a row is the columns of a group of 2^n lanes, which shuffles
// sum.  dw is summed by a thread over its rows in registers (kFold), by a CTA through
// shared memory and over the CTAs by a second kernel, each in a fixed order.
// Measured: GPT-2-medium q and k, 537 MB forward 87 us (6.1 TB/s, 0.90 of the copy
// rate), 805 MB backward 131 us (6.2 TB/s); 32 + 4 heads of 128, 581 MB backward 117 us
// (5.0 TB/s), whichever type, pairs or part of the columns turn: latency, with 12 warps
// on an SM.
#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace fa {
namespace {

constexpr int kNThreads = 128;
// Rows whose dw a thread adds up plainly.  A warp's sums of so many go to sums in shared memory that carry what their
// additions lose (Kahan's summation), so that no chain of additions grows with the number of rows: 3,000 equal terms a
// thread, the worst case, were off by 2^-14.5 of their sum.  Backward, without and so: GPT-2-medium q and k 148 and 144
// us, 46 of 64 columns 92 and 94; each thread's sums apart take 16 KB of what float32 rows need as L1, 141 -> 170 us.
constexpr int kFold = 64;

// Where the pairs of a thread's columns lie.
enum Pairs {
  kHalves = 0,   // (i, i + rot/2), rot/2 a multiple of 8: a thread owns 8 columns of each half, or 8 that do not turn
  kAdjacent,     // (2i, 2i + 1): 16 columns
  kShared        // (i, i + rot/2), any rot: 8 columns, the partners through shared memory
};

// The kernel's CTAs on an SM, of which the whole grid is one round, and its rows in flight.  kShared, whose threads have
// half the columns, takes more: 46 of 64 columns turned, 268 MB forward 96 / 79 / 69 / 112 us with 3 / 4 / 5 / 6, 403 MB
// backward 109 / 91 / 138 with 3 / 4 / 5 (94 with 4 and dw's sums by warp).  The others are slower so: forward 100 us
// against 87 with 4 or 5.
__host__ __device__ constexpr int ctas_of(int pairs, bool back) { return pairs != kShared ? 3 : back ? 4 : 5; }
// [warps][sum, lost][d] float32, see kFold
__host__ __device__ constexpr int sums_bytes(int d) { return kNThreads / 32 * 2 * d * (int)sizeof(float); }
template <typename T, int kPairs, bool kBack> struct NormCfg {
  static constexpr int kPer = 16 / (int)sizeof(T);                       // elements of a 16-byte piece
  static constexpr int kRow = (kPairs == kShared ? 8 : 16) / kPer;       // pieces of a row in a thread
  static constexpr int kPieces = kBack ? 2 * kRow : kRow;
  // four CTAs of kShared in float32 have room for 5; 16 heads of 46 of 64 columns 87 -> 71 us with 5 instead of 6
  static constexpr int kStages = kPieces == 8 ? 3 : kPieces == 4 ? (kBack && kPairs == kShared ? 5 : 6) : 8;
  static constexpr int kAhead = kStages * kPieces * kNThreads * 16;
  static constexpr int kStatic = 128 * 12 + (kPairs == kShared ? kNThreads * 32 : 32);
  static constexpr int kMost = kAhead + (kBack ? sums_bytes(256) : 0);
  static_assert(ctas_of(kPairs, kBack) * (kMost + kStatic + 1024) <= 233472, "the CTAs of one SM exceed its shared memory");
};

struct NormArgs {
  const void* x[2];        // q, k
  const void* dy[2];       // backward only
  void* y[2];              // y, or dx
  const float* w[2];       // [d] or nullptr (ones)
  Strides xs[2], ds[2], ys[2];
  int heads[2];
  int N, d, rot, units, lg;   // units: threads that own columns of a row; 2^lg lanes a row
  uint32_t tokens;         // B * N
  const void* pos;
  int pos64;
  int64_t pos_b, pos_n, start;
  const double* inv_freq;
  float mscale, eps, inv_d;
  int ctas[2];             // CTAs of q, then of k
  // backward: each CTA leaves one row of sums
  float* part;             // [ctas[0] + ctas[1]][d]
  float* dw[2];            // [d] or nullptr
};

// 8 consecutive elements
template <typename T> struct V8;
template <> struct V8<float> {
  float4 a, b;
  __device__ __forceinline__ void pieces(const uint8_t* p, int step) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + step);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <typename T> struct V8 {
  uint4 a;
  __device__ __forceinline__ void pieces(const uint8_t* p, int) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Cvt<T>::lo(w[i]);
      f[2 * i + 1] = Cvt<T>::hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
    *reinterpret_cast<uint4*>(p) = make_uint4(Cvt<T>::pack(f[0], f[1]), Cvt<T>::pack(f[2], f[3]),
                                              Cvt<T>::pack(f[4], f[5]), Cvt<T>::pack(f[6], f[7]));
  }
};

// The sines, cosines and weights of one thread's columns.  Columns of the
// thread: c0 .. c0 + 7 and, in kHalves where they turn and in kAdjacent where the row
// has them, c1 .. c1 + 7 half a row further (the lanes of a load lie side by side).
template <int kPairs> struct Turn {
  static constexpr int NC = kPairs == kShared ? 8 : 16;
  static constexpr int NP = 8;
  bool live, rotates, two;         // owns columns; some of them turn; owns the second eight
  int c0, c1, half;
  float cs[NP], sn[NP], w[NC];

  __device__ __forceinline__ void place(int u, int rot, int units, int d) {
    half = rot >> 1;
    live = u < units;
    if constexpr (kPairs == kHalves) {
      const int nrot = half >> 3;
      two = rotates = u < nrot;
      c0 = rotates ? u * 8 : rot + (u - nrot) * 8;
      c1 = two ? c0 + half : c0;
    } else {
      c0 = u * 8;
      c1 = (units + u) * 8;
      two = NC > 8 && c1 < d;
      if (!two) c1 = c0;
      rotates = c0 < rot;
    }
    if (!live) rotates = two = false;
  }
  __device__ __forceinline__ int pair_of(int e) const { return e < 4 ? (c0 >> 1) + e : two ? (c1 >> 1) + e - 4 : half; }   // kAdjacent
  __device__ __forceinline__ void angles(long long p, const unsigned long long* sF, const float* sM, float sgn) {
    if (!rotates) return;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      int i = kPairs == kAdjacent ? pair_of(e) : c0 + e;
      if (kPairs == kShared && i >= half) i -= half;
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (kPairs == kHalves || i < half) turn(p, sF[i], sM[i], sgn * sM[i], cs[e], sn[e]);
      if (kPairs == kShared && c0 + e < half) sn[e] = -sn[e];
    }
  }
  __device__ __forceinline__ void weights(const float* g) {
#pragma unroll
    for (int e = 0; e < NC; ++e) {
      const int c = e < 8 ? c0 + e : c1 + e - 8;
      w[e] = g != nullptr && live && (e < 8 || two) ? g[c] : 1.f;
    }
  }
  // v turned (kShared: through `rows`, where column 8 u + e of a row lies at [e][u] behind the row's first lane, so that
  // neither the lanes' own columns nor their partners, half a rotation away, share a bank)
  __device__ __forceinline__ void apply(float (&v)[NC], float* rows, int first) const {
    if constexpr (kPairs == kShared) {
      __syncwarp();
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rows[e * kNThreads + threadIdx.x] = v[e];
      }
      __syncwarp();
      if (rotates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + e, pc = c < half ? c + half : c - half;
          if (c < 2 * half) v[e] = v[e] * cs[e] + rows[(pc & 7) * kNThreads + first + (pc >> 3)] * sn[e];
        }
      }
    } else if (rotates) {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const int a = kPairs == kHalves ? e : 2 * e, b = kPairs == kHalves ? 8 + e : 2 * e + 1;
        if (kPairs == kAdjacent && pair_of(e) >= half) continue;
        const float x0 = v[a], x1 = v[b];
        v[a] = x0 * cs[e] - x1 * sn[e];
        v[b] = x1 * cs[e] + x0 * sn[e];
      }
    }
  }
};

// kL1: through L1, where a thread's two pieces share a 32-byte sector
template <bool kL1> __device__ __forceinline__ void cp_async16(uint32_t smem, const void* g) {
  if constexpr (kL1) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" :: "r"(smem), "l"(g) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// sum over the 2^lg lanes of a row (every lane of the warp takes part)
__device__ __forceinline__ float row_sum(float s, int lg) {
  for (int o = 1 << lg >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ void load_turns(const NormArgs& a, unsigned long long* sF, float* sM) {
  // float64 is slow on this GPU: the turns are made once per CTA, not once per thread
  for (int i = threadIdx.x; i < a.rot >> 1; i += kNThreads) {
    const double f = a.inv_freq[i];
    sF[i] = turns_of(f);
    sM[i] = isfinite(f) ? a.mscale : nanf("");
  }
  __syncthreads();
}

__device__ __forceinline__ long long position(const NormArgs& a, uint32_t b, uint32_t n) {
  if (a.pos == nullptr) return a.start + (long long)n;
  const int64_t at = (int64_t)b * a.pos_b + (int64_t)n * a.pos_n;
  return a.pos64 ? static_cast<const long long*>(a.pos)[at] : (long long)static_cast<const int*>(a.pos)[at];
}

// Both directions.  The rows of q (of k), tile by tile of kNThreads >> lg tokens and
// in a tile head by head, are shared out evenly over its CTAs.  A thread copies its
// rows ahead into shared memory that it has to itself (no barriers), so that what is
// in flight takes no registers.  GPT-2-medium q and k: backward 155 us with two rows in
// registers, 137 so (131 with dw's sums by warp, kFold); forward 93 with four, 87 so (537
// MB, 0.90 of the copy rate).
template <typename T, int kPairs, bool kBack>
__global__ void __launch_bounds__(kNThreads, ctas_of(kPairs, kBack)) norm_rope_kernel(const NormArgs a) {
  using R = Turn<kPairs>;
  using C = NormCfg<T, kPairs, kBack>;
  __shared__ unsigned long long sF[128];
  __shared__ float sM[128];
  __shared__ float rows[kPairs == kShared ? kNThreads * 8 : 8];
  extern __shared__ __align__(16) uint8_t ahead[];   // [kStages][kPieces][kNThreads] 16-byte pieces, of x, then of dy
  asm volatile("griddepcontrol.wait;" ::: "memory");
  load_turns(a, sF, sM);
  const int v = (int)blockIdx.x < a.ctas[0] ? 0 : 1;
  const int c = (int)blockIdx.x - (v ? a.ctas[0] : 0);
  const int per = kNThreads >> a.lg, heads = a.heads[v];      // tokens of a tile
  const unsigned long long total = (unsigned long long)((a.tokens + per - 1) / per) * heads;
  const unsigned long long from = total * c / a.ctas[v];
  const int count = (int)(total * (c + 1) / a.ctas[v] - from);   // rows of this CTA's groups
  const uint32_t tile0 = (uint32_t)(from / heads);
  const int head0 = (int)(from - (unsigned long long)tile0 * heads);
  R r;
  r.place((int)threadIdx.x & ((1 << a.lg) - 1), a.rot, a.units, a.d);
  r.weights(a.w[v]);
  const R all = r;
  const int first = (int)threadIdx.x >> a.lg << a.lg;      // the row's first lane
  const Strides xs = a.xs[v], ds = a.ds[v], ys = a.ys[v];
  struct Token { uint32_t b, n; bool there; };
  auto token_of = [&](uint32_t tile) -> Token {
    const uint32_t token = tile * per + (threadIdx.x >> a.lg), tk = min(token, a.tokens - 1);
    Token t;
    t.b = tk / (uint32_t)a.N;
    t.n = tk - t.b * (uint32_t)a.N;
    t.there = token < a.tokens;
    return t;
  };
  // ---- the copies' place in the sequence
  const uint32_t slot0 = smem_u32(ahead) + threadIdx.x * 16;
  uint32_t ltile = tile0;
  int lh = head0, ls = 0, left = count;
  bool lt = false;
  const T *lx = nullptr, *lg = nullptr;
  auto enter = [&]() {
    const Token t = token_of(ltile);
    lt = t.there;
    lx = static_cast<const T*>(a.x[v]) + (int64_t)t.b * xs.b + (int64_t)lh * xs.h + (int64_t)t.n * xs.n;
    if (kBack) lg = static_cast<const T*>(a.dy[v]) + (int64_t)t.b * ds.b + (int64_t)lh * ds.h + (int64_t)t.n * ds.n;
  };
  auto copy = [&]() {                                // the next row, into stage ls
    if (left > 0) {
      if (lt) {
        const uint32_t at = slot0 + ls * (C::kPieces * kNThreads * 16);
#pragma unroll
        for (int i = 0; i < C::kRow; ++i) {
          // of the first eight columns, then of the second
          const int e = i * C::kPer, col = (e < 8 ? all.c0 + e : all.c1 + e - 8);
          if (e < 8 ? all.live : all.two) {
            cp_async16<sizeof(T) == 4>(at + i * (kNThreads * 16), lx + col);
            if (kBack) cp_async16<sizeof(T) == 4>(at + (C::kRow + i) * (kNThreads * 16), lg + col);
          }
        }
      }
      lx += xs.h;
      if (kBack) lg += ds.h;
      if (++lh == heads) {
        lh = 0;
        ++ltile;
        enter();
      }
      --left;
    }
    cp_async_commit();
    ls = ls + 1 == C::kStages ? 0 : ls + 1;
  };
  enter();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) copy();
  int st = 0;
  float acc[kBack ? R::NC : 1] = {};
  // dw of kFold rows: over the warp's groups, then into its sums
  float* const sums = reinterpret_cast<float*>(ahead + C::kAhead) + (threadIdx.x >> 5) * 2 * a.d;
  if constexpr (kBack) {
    for (int i = threadIdx.x & 31; i < 2 * a.d; i += 32) sums[i] = 0.f;
    __syncwarp();
  }
  auto fold = [&]() {
    if constexpr (kBack) {
      for (int o = 16; o >= 1 << a.lg; o >>= 1) {
#pragma unroll
        for (int e = 0; e < R::NC; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      }
#pragma unroll
      for (int e = 0; e < R::NC; ++e) {
        if ((int)(threadIdx.x & 31) < 1 << a.lg && (e < 8 ? all.live : all.two)) {
          float* const at = sums + (e < 8 ? all.c0 + e : all.c1 + e - 8);
          const float old = at[0], t = acc[e] - at[a.d], sum = old + t;
          at[a.d] = (sum - old) - t;
          at[0] = sum;
        }
        acc[e] = 0.f;
      }
    }
  };
  int since = 0;
  uint32_t tile = tile0;
  for (int done = 0, h0 = head0; done < count; ++tile, h0 = 0) {
    const Token it = token_of(tile);
    const int h1 = min(heads, h0 + count - done);
    done += h1 - h0;
    r.live = all.live && it.there;
    r.two = all.two && it.there;
    r.rotates = all.rotates && it.there;
    r.angles(position(a, it.b, it.n), sF, sM, kBack ? -1.f : 1.f);       // the transposed rotation, or the rotation
    T* dst = static_cast<T*>(a.y[v]) + (int64_t)it.b * ys.b + (int64_t)h0 * ys.h + (int64_t)it.n * ys.n;
#pragma unroll 1
    for (int h = h0; h < h1; ++h, dst += ys.h) {
      copy();                                        // over the stage of the row before this one
      cp_async_wait<C::kStages - 1>();
      float x[R::NC] = {}, g[kBack ? R::NC : 1] = {};
      const uint8_t* at = ahead + (st * C::kPieces * kNThreads + threadIdx.x) * 16;
      st = st + 1 == C::kStages ? 0 : st + 1;
#pragma unroll
      for (int e = 0; e < R::NC; e += 8) {
        if (!(e < 8 ? r.live : r.two)) continue;
        V8<T> p;
        p.pieces(at + (e / C::kPer) * (kNThreads * 16), kNThreads * 16);
        p.get(x + e);
        if constexpr (kBack) {
          p.pieces(at + (C::kRow + e / C::kPer) * (kNThreads * 16), kNThreads * 16);
          p.get(g + e);
        }
      }
      if constexpr (kBack) {
        r.apply(g, rows, first);                             // dz
        float sx = 0.f, sg = 0.f, sx1 = 0.f, sg1 = 0.f;
#pragma unroll
        for (int e = 0; e < R::NC; e += 2) {
          float y0, y1;                              // w dz
          mul2(y0, y1, g[e], g[e + 1], r.w[e], r.w[e + 1]);
          fma2(sg, sg1, y0, y1, x[e], x[e + 1], sg, sg1);
          fma2(sx, sx1, x[e], x[e + 1], x[e], x[e + 1], sx, sx1);
        }
        sx += sx1;
        sg += sg1;
        for (int o = 1 << a.lg >> 1; o > 0; o >>= 1) {
          sx += __shfl_xor_sync(0xffffffffu, sx, o);
          sg += __shfl_xor_sync(0xffffffffu, sg, o);
        }
        const float rs = rsqrtf(sx * a.inv_d + a.eps);
        const float k = -rs * (rs * (rs * (sg * a.inv_d)));  // dx = rs w dz - x rs^3 (g . x) / d; rs^2 alone may overflow
#pragma unroll
        for (int e = 0; e < R::NC; e += 2) {
          float y0, y1;
          mul2(y0, y1, g[e], g[e + 1], rs, rs);
          fma2(acc[e], acc[e + 1], y0, y1, x[e], x[e + 1], acc[e], acc[e + 1]);
          mul2(y0, y1, y0, y1, r.w[e], r.w[e + 1]);
          fma2(x[e], x[e + 1], x[e], x[e + 1], k, k, y0, y1);
        }
        if (++since == kFold) {
          since = 0;
          fold();
        }
      } else {
        float sx = 0.f, sx1 = 0.f;
#pragma unroll
        for (int e = 0; e < R::NC; e += 2) fma2(sx, sx1, x[e], x[e + 1], x[e], x[e + 1], sx, sx1);
        const float rs = rsqrtf(row_sum(sx + sx1, a.lg) * a.inv_d + a.eps);
#pragma unroll
        for (int e = 0; e < R::NC; e += 2) {
          mul2(x[e], x[e + 1], x[e], x[e + 1], rs, rs);
          mul2(x[e], x[e + 1], x[e], x[e + 1], r.w[e], r.w[e + 1]);
        }
        r.apply(x, rows, first);
      }
      if (r.live) V8<T>::store(dst + r.c0, x);
      if (R::NC > 8 && r.two) V8<T>::store(dst + r.c1, x + (R::NC - 8));
    }
  }
  if (!kBack || a.dw[v] == nullptr) return;
  // the CTA's sums: the warps', in their order
  cp_async_wait<0>();
  fold();
  __syncthreads();
  const float* const from0 = reinterpret_cast<const float*>(ahead + C::kAhead);
  for (int c = threadIdx.x; c < a.d; c += kNThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNThreads / 32; ++w) s += from0[w * 2 * a.d + c] - from0[(w * 2 + 1) * a.d + c];
    a.part[(size_t)blockIdx.x * a.d + c] = s;
  }
}

// dw of q (blockIdx.y = 0) and k: eight columns a block, 128 threads a column, each with
// every 128th CTA's sums, joined in their order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int d, int n0, int n1, float* dq,
                                                       float* dk) {
  __shared__ float sh[128][9];
  float* out = blockIdx.y ? dk : dq;
  if (out == nullptr) return;
  const int n = blockIdx.y ? n1 : n0;
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  part += (blockIdx.y ? (size_t)n0 * d : 0) + blockIdx.x * 8 + c;
  float s = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 8
  for (int i = g; i < n; i += 128) s += part[(size_t)i * d];
  sh[g][c] = s;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;      // a warp a column
  s = (sh[lane][w] + sh[lane + 32][w]) + (sh[lane + 64][w] + sh[lane + 96][w]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) out[blockIdx.x * 8 + w] = s;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
bool n16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fa_status norm_strides(Strides& s, int B, int heads, int N, int d, int unit, bool output) {
  if (N == 1) s.n = d;
  if (heads == 1) s.h = (int64_t)N * s.n;
  if (B == 1) s.b = (int64_t)heads * s.h;
  const int64_t least = output ? 1 : 0;          // an input may be broadcast (stride 0)
  if (s.n < (output ? d : 0) || s.h < least || s.b < least) return FA_ERR_INVALID_ARG;
  if (s.n % unit || s.h % unit || s.b % unit) return FA_ERR_MISALIGNED;
  return FA_OK;
}

Pairs pairs_of(const fa_norm_rope_params* p) {
  if (p->interleaved) return kAdjacent;
  return p->rot % 16 == 0 ? kHalves : kShared;
}

int units_of(const fa_norm_rope_params* p) {
  const Pairs m = pairs_of(p);
  return m == kHalves ? (p->d - p->rot / 2) / 8 : m == kAdjacent ? (p->d + 8) / 16 : p->d / 8;
}

int lg_of(int units) {
  int lg = 0;
  while ((1 << lg) < units) ++lg;
  return lg;
}

// the shape alone
fa_status check_norm(const fa_norm_rope_params* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 1 || p->H < 1 || p->H_kv < 0 || p->N < 1 || p->d < 1) return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_DT_F32 && p->dtype != FA_DT_F16 && p->dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  if (p->rot < 0 || p->rot > p->d || (p->rot & 1)) return FA_ERR_INVALID_ARG;
  if (p->d % 8 != 0 || p->d > 256) return FA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->mscale) || !std::isfinite(p->eps) || !(p->eps > 0.f)) return FA_ERR_INVALID_ARG;
  if (p->rot > 0 && p->inv_freq == nullptr) return FA_ERR_INVALID_ARG;
  // 32-bit thread and token indexes
  if ((unsigned long long)p->B * p->N * p->d >= (1ull << 32) - 4096) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// CTAs of q and of k: by their heads, no more than there are tokens' tiles x heads (152 SMs: a workspace's size does
// not depend on the device)
void norm_ctas(const fa_norm_rope_params* p, bool back, int (&n)[2]) {
  const int heads[2] = {p->H, p->H_kv};
  const int per = kNThreads >> lg_of(units_of(p));
  const long long tiles = ((long long)p->B * p->N + per - 1) / per;
  for (int v = 0; v < 2; ++v) {
    const long long share = std::max<long long>(1, 152ll * ctas_of(pairs_of(p), back) * heads[v] / (p->H + p->H_kv));
    n[v] = heads[v] == 0 ? 0 : (int)std::min(share, tiles * heads[v]);
  }
}

// What both directions check and fill in.  t: x, dy (backward), y
fa_status fill(const fa_norm_rope_params* p, const void* const (&x)[2], const void* const (&dy)[2], void* const (&y)[2],
               const float* const (&w)[2], bool bwd, NormArgs& a) {
  fa_status s = check_norm(p);
  if (s != FA_OK) return s;
  const int nt = p->H_kv > 0 ? 2 : 1;
  for (int v = 0; v < nt; ++v)
    if (x[v] == nullptr || y[v] == nullptr || (bwd && dy[v] == nullptr)) return FA_ERR_INVALID_ARG;
  for (int v = 0; v < nt; ++v) {
    if (!n16(x[v]) || !n16(y[v]) || (bwd && !n16(dy[v]))) return FA_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(w[v]) & 3u) return FA_ERR_MISALIGNED;
  }
  if (reinterpret_cast<uintptr_t>(p->inv_freq) & 7u) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->positions) & (p->positions_i64 ? 7u : 3u)) return FA_ERR_MISALIGNED;
  const int unit = p->dtype == FA_DT_F32 ? 4 : 8;
  a.xs[0] = {p->q_stride_b, p->q_stride_h, p->q_stride_n};
  a.ys[0] = {p->q_out_stride_b, p->q_out_stride_h, p->q_out_stride_n};
  a.ds[0] = {p->dq_stride_b, p->dq_stride_h, p->dq_stride_n};
  a.xs[1] = {p->k_stride_b, p->k_stride_h, p->k_stride_n};
  a.ys[1] = {p->k_out_stride_b, p->k_out_stride_h, p->k_out_stride_n};
  a.ds[1] = {p->dk_stride_b, p->dk_stride_h, p->dk_stride_n};
  a.heads[0] = p->H; a.heads[1] = p->H_kv;
  for (int v = 0; v < nt; ++v) {
    s = norm_strides(a.xs[v], p->B, a.heads[v], p->N, p->d, unit, false);
    if (s == FA_OK) s = norm_strides(a.ys[v], p->B, a.heads[v], p->N, p->d, unit, true);
    if (s == FA_OK && bwd) s = norm_strides(a.ds[v], p->B, a.heads[v], p->N, p->d, unit, false);
    if (s != FA_OK) return s;
    // an output in an input's place needs the input's strides: rows would overwrite one another
    const void* in[2] = {x[v], bwd ? dy[v] : nullptr};
    const Strides st[2] = {a.xs[v], a.ds[v]};
    for (int i = 0; i < 2; ++i)
      if (in[i] == y[v] && (st[i].b != a.ys[v].b || st[i].h != a.ys[v].h || st[i].n != a.ys[v].n))
        return FA_ERR_INVALID_ARG;
    a.x[v] = x[v]; a.dy[v] = dy[v]; a.y[v] = y[v]; a.w[v] = w[v];
  }
  a.N = p->N; a.d = p->d; a.rot = p->rot;
  a.units = units_of(p);
  a.lg = lg_of(a.units);
  a.tokens = (uint32_t)((long long)p->B * p->N);
  a.pos = p->positions; a.pos64 = p->positions_i64;
  a.pos_b = p->pos_stride_b; a.pos_n = p->pos_stride_n; a.start = p->start;
  a.inv_freq = p->inv_freq;
  a.mscale = p->mscale; a.eps = p->eps; a.inv_d = 1.f / (float)p->d;
  return FA_OK;
}

template <typename T, int kPairs, bool kBack> cudaError_t launch_n(const NormArgs& a, cudaStream_t s) {
  auto kern = norm_rope_kernel<T, kPairs, kBack>;
  using C = NormCfg<T, kPairs, kBack>;
  const int bytes = C::kAhead + (kBack ? sums_bytes(a.d) : 0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(a.ctas[0] + a.ctas[1]));
  c.blockDim = dim3(kNThreads);
  c.dynamicSmemBytes = bytes;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, kern, a);
  if (e != cudaSuccess || !kBack || (a.dw[0] == nullptr && a.dw[1] == nullptr)) return e;
  c.gridDim = dim3((unsigned)(a.d / 8), 2);
  c.blockDim = dim3(1024);
  c.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&c, norm_dw_kernel, (const float*)a.part, a.d, a.ctas[0], a.ctas[1], a.dw[0], a.dw[1]);
}

template <typename T, bool kBack> cudaError_t launch_t(const NormArgs& a, Pairs m, cudaStream_t s) {
  switch (m) {
    case kHalves: return launch_n<T, kHalves, kBack>(a, s);
    case kAdjacent: return launch_n<T, kAdjacent, kBack>(a, s);
    default: return launch_n<T, kShared, kBack>(a, s);
  }
}

template <bool kBack> fa_status launch(const fa_norm_rope_params* p, NormArgs& a, void* stream) {
  norm_ctas(p, kBack, a.ctas);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Pairs m = pairs_of(p);
  const cudaError_t e = p->dtype == FA_DT_F32   ? launch_t<float, kBack>(a, m, s)
                        : p->dtype == FA_DT_F16 ? launch_t<__half, kBack>(a, m, s)
                                                : launch_t<__nv_bfloat16, kBack>(a, m, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_norm_rope(const fa_norm_rope_params* p, const void* q, const void* k, const float* q_weight,
                       const float* k_weight, void* q_out, void* k_out, void* stream) {
  NormArgs a{};
  const fa_status s = fill(p, {q, k}, {nullptr, nullptr}, {q_out, k_out}, {q_weight, k_weight}, false, a);
  return s == FA_OK ? launch<false>(p, a, stream) : s;
}

size_t fa_norm_rope_bwd_workspace_size(const fa_norm_rope_params* p) {
  if (check_norm(p) != FA_OK) return 256;
  int n[2];
  norm_ctas(p, true, n);
  return 256 + (size_t)(n[0] + n[1]) * p->d * sizeof(float);
}

fa_status fa_norm_rope_bwd(const fa_norm_rope_params* p, const void* q, const void* k, const void* dq_out,
                           const void* dk_out, const float* q_weight, const float* k_weight, void* dq, void* dk,
                           float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes, void* stream) {
  NormArgs a{};
  fa_status s = fill(p, {q, k}, {dq_out, dk_out}, {dq, dk}, {q_weight, k_weight}, true, a);
  if (s != FA_OK) return s;
  if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u) return FA_ERR_MISALIGNED;
  if (ws == nullptr || ws_bytes < fa_norm_rope_bwd_workspace_size(p) || !n16(ws)) return FA_ERR_WORKSPACE;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
  a.dw[0] = dq_weight;
  a.dw[1] = p->H_kv > 0 ? dk_weight : nullptr;
  return launch<true>(p, a, stream);
}

}  // extern "C"
