// sink_few.cu -- the backward pass of a few first keys that stay visible under a
// sliding window, with the prepass of the backward kernels in the same pass.
//
// Mathematics.  For the pairs of a query i with the first keys j that its window
// has left behind (j <= i - window, j < few <= 8):
//     p_ij = exp(tau q_i . k_j - LSE_i),  ds_ij = p_ij (z_ij dO_i . v_j - D_i),
//     dQ_i += tau ds_ij k_j,  dK_j += tau ds_ij q_i,  dV_j += z_ij p_ij dO_i
// (z: the dropout mask over 1 - p).  All other pairs are those of the window alone.
//
// What bounds it: HBM.  The backward kernel visits a first key tile with 128 x 128
// products for each query tile, of which 8 columns or fewer are used.  Here one pass reads
// Q, dO, O and LSE, which the prepass (D_i, LSE in log2 units) reads in part anyway,
// and writes the float32 dQ accumulator, which the prepass clears anyway.  A warp
// takes 16 rows, copied ahead into shared memory that a thread has to itself, and
// forms the products in registers (m16n8k16), the first keys as the 8 columns of
// the scores and, transposed, of dK and dV; p and ds are rounded to 16 bits for
// them as in the backward kernels, all sums are float32.  dK and dV of a CTA's rows go
// to few_part, which few_finish adds up in a fixed order.  Measured: 64 heads of 64 x
// 4,096, window 512, 4 first keys 31 us (168 MB, 5.4 TB/s; the prepass alone 24), the
// whole backward pass 211 us, with the first key tiles in the backward kernel 240,
// without first keys 200; window 64, 128 heads of 2,048, 8 first keys 155, 9 (the other
// way) 174.  On CUDA cores, 8 columns a thread, this pass takes 400 instructions for
// 4 rows and 67 us.
#include <type_traits>

#include "bwd_items.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFThreads = 128;

template <int D> struct FCfg {
  static constexpr int NP = D / 32;                    // 16-byte pieces of a row in a thread: columns 32 p + 8 c ..
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kCtas = D == 64 ? 3 : 2;        // CTAs on an SM
  static constexpr int kStage = kFThreads * (3 * 2 * NP * 16 + 2 * 4);   // O, dO, Q of two rows, their LSE
  static constexpr int kLse = kFThreads * 3 * 2 * NP * 16;
  static constexpr int kBytes = kStages * kStage;
  static_assert(kCtas * (kBytes + 1024) <= 233472, "the CTAs of one SM exceed its shared memory");
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {   // an 8 x 8 matrix whose row l / 4 lane l has two columns of
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <typename T> __device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                            uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T> __device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(b0));
  else
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(b0));
}

// Thread (g = lane / 4, c = lane % 4) of a warp has rows g and g + 8 of its 16.  Its element e of a row is column
// 32 (e / 8) + 8 c + e % 8: the lanes of a copy lie side by side.  The products' inner order is free as long as both
// operands agree: step t of the scores takes elements 4 t .. 4 t + 3.  Columns of dQ's product u, and rows of dK's and
// dV's, are elements 2 u and 2 u + 1 of the four c.
template <typename T, int D>
__global__ void __launch_bounds__(kFThreads, FCfg<D>::kCtas)
sink_few_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ o,
                const T* __restrict__ dout, Strides st, const float* __restrict__ lse, float* __restrict__ lse2,
                float* __restrict__ dvec, float* __restrict__ dqacc, float dscale, int rows, const BwdArgs a) {
  using C = FCfg<D>;
  constexpr int NP = C::NP, NU = D / 8;                // pieces, pairs of elements of a row in a thread
  constexpr bool kFold = std::is_same<T, __nv_bfloat16>::value;   // tau in ds before it is rounded, as in bwd_tc.cu
  extern __shared__ __align__(16) uint8_t ahead[];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.sched = 0;      // backward work counter
  const int bh = (int)blockIdx.x / a.few_chunks, chunk = (int)blockIdx.x - bh * a.few_chunks;
  const int b = bh / a.H, h = bh - b * a.H, hk = h / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  int few = a.few;
  if (a.mask.seqlens_k != nullptr) few = max(0, min(few, a.mask.seqlens_k[b]));
  const size_t off = (size_t)b * st.b + (size_t)h * st.h + c * 8;
  const int i1 = min((chunk + 1) * rows, a.npad);      // a multiple of 64, like the chunk's first row
  const uint32_t mine = smem_u32(ahead) + threadIdx.x * 16, minel = smem_u32(ahead) + C::kLse + threadIdx.x * 4;
  int li = chunk * rows + warp * 16 + gq, ls = 0;
  auto copy = [&]() {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int i = li + 8 * y;
      if (i < min(i1, a.N)) {
        const size_t at = off + (size_t)i * st.n;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint32_t to = mine + ls * C::kStage + (y * NP + p) * kFThreads * 16;
          copy16(to, o + at + 32 * p);
          copy16(to + 2 * NP * kFThreads * 16, dout + at + 32 * p);
          if (few > 0 && i >= a.mask.window) copy16(to + 4 * NP * kFThreads * 16, q + at + 32 * p);
        }
        copy4(minel + ls * C::kStage + y * kFThreads * 4, lse + (size_t)bh * a.N + i);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    li += 64;
    ls = ls + 1 == C::kStages ? 0 : ls + 1;
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) copy();
  // K and V of key gq as the scores' second operand, K of keys 2 c and 2 c + 1 as dQ's
  uint32_t kb[NU], vb[NU], kd[NU];
  {
    const T* kp = k + (size_t)b * a.kst.b + (size_t)hk * a.kst.h;
    const T* vp = v + (size_t)b * a.kst.b + (size_t)hk * a.kst.h;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      if (gq < few) {
        x = *reinterpret_cast<const uint4*>(kp + (size_t)gq * a.kst.n + 32 * p + 8 * c);
        y = *reinterpret_cast<const uint4*>(vp + (size_t)gq * a.kst.n + 32 * p + 8 * c);
      }
      kb[4 * p] = x.x; kb[4 * p + 1] = x.y; kb[4 * p + 2] = x.z; kb[4 * p + 3] = x.w;
      vb[4 * p] = y.x; vb[4 * p + 1] = y.y; vb[4 * p + 2] = y.z; vb[4 * p + 3] = y.w;
    }
    // the pair u of key gq: columns of the four c; transposed, column gq of keys 2 c and 2 c + 1
#pragma unroll
    for (int u = 0; u < NU; ++u) kd[u] = transposed(kb[u]);
  }
  float ak[NU / 2][4] = {}, av[NU / 2][4] = {};
  int cs = 0;
  for (int iw = chunk * rows + warp * 16; iw < i1; iw += 64) {
    copy();
    asm volatile("cp.async.wait_group %0;" :: "n"(C::kStages - 1) : "memory");
    const uint8_t* at = ahead + cs * C::kStage + threadIdx.x * 16;
    const uint8_t* atl = ahead + cs * C::kStage + C::kLse + threadIdx.x * 4;
    cs = cs + 1 == C::kStages ? 0 : cs + 1;
    uint32_t x[2][NU], g[2][NU];                       // q, dO
    float d[2], l2[2];
    bool pairs[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int i = iw + gq + 8 * y;
      const bool there = i < a.N;
      d[y] = 0.f;
      l2[y] = INFINITY;
      float d1 = 0.f;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u), z = w;
        if (there) {
          w = *reinterpret_cast<const uint4*>(at + (y * NP + p) * kFThreads * 16);
          z = *reinterpret_cast<const uint4*>(at + ((2 + y) * NP + p) * kFThreads * 16);
        }
        const uint32_t ow[4] = {w.x, w.y, w.z, w.w}, gw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[y][4 * p + e] = gw[e];
          fma2(d[y], d1, Cvt<T>::lo(ow[e]), Cvt<T>::hi(ow[e]), Cvt<T>::lo(gw[e]), Cvt<T>::hi(gw[e]), d[y], d1);
        }
      }
      d[y] += d1;
      if (there) {
        const float l = *reinterpret_cast<const float*>(atl + y * kFThreads * 4);
        if (l != -INFINITY) l2[y] = l * kLog2e;
      }
      pairs[y] = there && few > 0 && i >= a.mask.window;
      if (pairs[y] && a.mask.row_list != nullptr) {
        const int qt = i / kTile;
        pairs[y] = a.mask.row_cnt[qt] > 0 && a.mask.row_list[(size_t)qt * a.mask.nb] == 0;
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      d[y] += __shfl_xor_sync(0xffffffffu, d[y], 1);
      d[y] += __shfl_xor_sync(0xffffffffu, d[y], 2);
      const int i = iw + gq + 8 * y;
      if (c == 0) {
        lse2[(size_t)bh * a.npad + i] = l2[y];
        dvec[(size_t)bh * a.npad + i] = i < a.N ? d[y] * dscale : 0.f;
      }
    }
    const bool work = __any_sync(0xffffffffu, pairs[0] || pairs[1]);
    uint32_t da[2] = {0u, 0u};
    if (work) {
      // rows without pairs (of a sequence without keys, all of them) are zeros: 0 times a row that is not finite would
      // not be 0
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (pairs[y]) w = *reinterpret_cast<const uint4*>(at + ((4 + y) * NP + p) * kFThreads * 16);
          x[y][4 * p] = w.x; x[y][4 * p + 1] = w.y; x[y][4 * p + 2] = w.z; x[y][4 * p + 3] = w.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) g[y][4 * p + e] = pairs[y] ? g[y][4 * p + e] : 0u;
        }
      float s[4] = {}, t[4] = {};                      // rows g (0, 1) and g + 8 (2, 3), keys 2 c and 2 c + 1
#pragma unroll
      for (int u = 0; u < NU; u += 2) {
        mma16<T>(s, x[0][u], x[1][u], x[0][u + 1], x[1][u + 1], kb[u], kb[u + 1]);
        mma16<T>(t, g[0][u], g[1][u], g[0][u + 1], g[1][u + 1], vb[u], vb[u + 1]);
      }
      const float rp = a.drop.enabled ? a.drop.rp : 1.f;
      uint32_t pt[2], dt[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = iw + gq + 8 * y;
        uint32_t keep = ~0u;
        if (a.drop.enabled && pairs[y]) keep = dropout_keep8(0u, (uint32_t)bh * (uint32_t)a.N + (uint32_t)i, a.drop);
        float p[2], ds[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * c + e;
          const bool see = pairs[y] && j < few && i - a.mask.window >= j;
          const float z = (keep >> j) & 1u ? rp : 0.f;
          p[e] = see ? ex2(s[2 * y + e] * a.scale_log2 - l2[y]) : 0.f;
          ds[e] = see ? p[e] * (z * t[2 * y + e] - d[y]) * (kFold ? a.scale : 1.f) : 0.f;
          p[e] *= z;
        }
        da[y] = Cvt<T>::pack(ds[0], ds[1]);
        pt[y] = transposed(Cvt<T>::pack(p[0], p[1]));
        dt[y] = transposed(da[y]);
      }
#pragma unroll
      for (int m = 0; m < NU / 2; ++m) {
        mma16<T>(ak[m], transposed(x[0][2 * m]), transposed(x[0][2 * m + 1]), transposed(x[1][2 * m]),
                 transposed(x[1][2 * m + 1]), dt[0], dt[1]);
        mma16<T>(av[m], transposed(g[0][2 * m]), transposed(g[0][2 * m + 1]), transposed(g[1][2 * m]),
                 transposed(g[1][2 * m + 1]), pt[0], pt[1]);
      }
    }
    float* const dst = dqacc + ((size_t)bh * a.N + iw + gq) * D + 8 * c;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float r[4][4] = {};
      if (work) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mma8<T>(r[e], da[0], da[1], kd[4 * p + e]);
      }
      const float f = kFold ? 1.f : a.scale;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (iw + gq + 8 * y >= a.N) continue;
        float4* z = reinterpret_cast<float4*>(dst + 8 * y * D + 32 * p);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          z[e] = make_float4(r[2 * e][2 * y] * f, r[2 * e][2 * y + 1] * f, r[2 * e + 1][2 * y] * f, r[2 * e + 1][2 * y + 1] * f);
      }
    }
  }
  // ---- dK and dV: over the warps
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ahead);       // [4][kFewSinks][2][D]
  static_assert(kFewSinks == 8, "the products' 8 columns");
#pragma unroll
  for (int m = 0; m < NU / 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // product row gq (+ 8: e / 2) of m is element 2 u + gq % 2, u = 2 m + e / 2, of the c that is gq / 2
      const int u = 2 * m + (e >> 1), at = 2 * u + (gq & 1);
      float* to = sums + ((size_t)warp * kFewSinks + 2 * c + (e & 1)) * 2 * D + 32 * (at >> 3) + 8 * (gq >> 1) + (at & 7);
      to[0] = ak[m][e] * (kFold ? 1.f : a.scale);
      to[D] = av[m][e];
    }
  __syncthreads();
  constexpr int n = kFewSinks * 2 * D;
  for (int i = threadIdx.x; i < n; i += kFThreads)
    a.few_part[(size_t)blockIdx.x * n + i] = (sums[i] + sums[n + i]) + (sums[2 * n + i] + sums[3 * n + i]);
}

template <typename T, int D>
cudaError_t launch_t(const void* q, const void* k, const void* v, const void* o, const void* dout, Strides st,
                     const float* lse, float* lse2, float* dvec, float* dqacc, float dscale, const BwdArgs& a, cudaStream_t s) {
  auto kern = sink_few_kernel<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg<D>::kBytes);
  if (e != cudaSuccess) return e;
  const int rows = ((a.npad + a.few_chunks - 1) / a.few_chunks + 63) / 64 * 64;
  kern<<<(unsigned)(a.B * a.H * a.few_chunks), kFThreads, FCfg<D>::kBytes, s>>>(
      static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), static_cast<const T*>(o),
      static_cast<const T*>(dout), st, lse, lse2, dvec, dqacc, dscale, rows, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sink_few(int dtype, int d, const void* q, const void* k, const void* v, const void* o, const void* dout,
                            Strides st, const float* lse, float* lse2, float* dvec, float* dqacc, float dscale,
                            const BwdArgs& a, cudaStream_t s) {
  using B16 = __nv_bfloat16;
  if (dtype == FA_DT_BF16)
    return d == 128 ? launch_t<B16, 128>(q, k, v, o, dout, st, lse, lse2, dvec, dqacc, dscale, a, s)
                    : launch_t<B16, 64>(q, k, v, o, dout, st, lse, lse2, dvec, dqacc, dscale, a, s);
  return d == 128 ? launch_t<__half, 128>(q, k, v, o, dout, st, lse, lse2, dvec, dqacc, dscale, a, s)
                  : launch_t<__half, 64>(q, k, v, o, dout, st, lse, lse2, dvec, dqacc, dscale, a, s);
}

}  // namespace fa
