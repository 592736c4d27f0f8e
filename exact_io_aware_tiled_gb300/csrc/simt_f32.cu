// simt_f32.cu -- float32 attention forward / backward on CUDA cores.
//
// The float32 path must agree with the float64 definition to ~1e-5, which
// tensor-core float32 formats (tf32, 10-bit mantissa) cannot reach, so these
// kernels use plain FFMA.  They implement the same method as the tensor-core
// kernels: forward = Q-outer tiles with the online-softmax recurrence
// (lynx-cortex, "El algoritmo Flash (forward)"); backward = recomputation of
// P from the saved logsumexp, D = rowsum(dO o O) (tonho.wtf, "como
// funciona"), with the same masks, block lists and Philox dropout mapping.
// Head dimension 64; one thread per query row (forward, dQ) or key row
// (dK, dV); K/V or Q/dO sub-tiles of 32 rows staged in shared memory.
// Grouped-query heads read K/V head h / g, and a dK/dV block sums over the g
// query heads of its K/V head; the sliding window bounds both tile lists and
// masks inside the boundary tiles.
#include "simt_lists.cuh"

namespace fa {
namespace {

constexpr int kRows = 128;   // rows per block
constexpr int kD = 64;
// Rows whose products with a thread's own row (backward) are formed side by side: each is a chain of 64 sums.  32 heads
// x 2,048, window 128: one at a time 891 us, 4 696, 8 657, dQ and dK, dV in one launch 618.
constexpr int kAtOnce = 8;
constexpr float kLn2 = 0.6931471805599453f;

// kWin: a WindowKind.  Tests for first keys or a window that are not there cost the unrolled products 5 to 20 %: 32 heads
// x 2,048 causal 1,225 us with them and 1,065 so, all keys 1,510 and 1,357, window 128 213 and 192.
template <int kWin>
__global__ void __launch_bounds__(kRows)
fwd_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                float* __restrict__ o, Strides st, Strides kst, const FwdArgs a) {
  __shared__ float Ks[kSub][kD];
  __shared__ float Vs[kSub][kD];
  const int qt = blockIdx.x;
  const int bh = blockIdx.y;
  const int b = bh / a.H, h = bh % a.H;
  const int r = threadIdx.x;
  const int i = qt * kRows + r;
  int Lk = a.N;
  if (a.mask.seqlens_k) Lk = max(0, min(a.N, a.mask.seqlens_k[b]));
  const size_t base = (size_t)b * st.b + (size_t)h * st.h;
  const size_t kbase = (size_t)b * kst.b + (size_t)(h / a.group) * kst.h;
  float qr[kD], acc[kD];
#pragma unroll
  for (int c = 0; c < kD; ++c) {
    qr[c] = i < a.N ? q[base + (size_t)i * st.n + c] : 0.f;
    acc[c] = 0.f;
  }
  const int jmax = a.mask.causal ? min(Lk - 1, i) : Lk - 1;
  const int jmin = a.mask.window > 0 ? i - a.mask.window + 1 : 0;
  const float sl2 = a.scale_log2;
  const uint32_t row_g = (uint32_t)bh * (uint32_t)a.N + (uint32_t)i;
  float m = -INFINITY, l = 0.f;
  const TileList tl = fwd_list(a.mask, qt, Lk);
  for (int s = 0; s < tl.n; ++s) {
    const int kvt = tl.at(s);
    for (int sub = 0; sub < kTile / kSub; ++sub) {
      const int j0 = kvt * kTile + sub * kSub;
      if (kWin != kAllKeys && hidden(a.mask, j0, qt * kRows, kRows)) continue;
      __syncthreads();
      for (int e = r; e < kSub * kD; e += kRows) {
        const int jj = j0 + e / kD, c = e % kD;
        Ks[e / kD][c] = jj < a.N ? k[kbase + (size_t)jj * kst.n + c] : 0.f;
        Vs[e / kD][c] = jj < a.N ? v[kbase + (size_t)jj * kst.n + c] : 0.f;
      }
      __syncthreads();
      if (kWin != kAllKeys && hidden(a.mask, j0, i & ~31, 32)) continue;
      float sc[kSub];
      float mx = -INFINITY;
#pragma unroll
      for (int jj = 0; jj < kSub; ++jj) {
        float d = 0.f;
#pragma unroll
        for (int c = 0; c < kD; ++c) d = fmaf(qr[c], Ks[jj][c], d);
        sc[jj] = j0 + jj <= jmax && (kWin == kAllKeys || j0 + jj >= jmin || (kWin == kWindowSinks && j0 + jj < a.mask.sinks))
                     ? d * sl2 : -INFINITY;
        mx = fmaxf(mx, sc[jj]);
      }
      const float mn = fmaxf(m, mx);
      const float mref = mn == -INFINITY ? 0.f : mn;
      const float alpha = m == -INFINITY ? 0.f : ex2(m - mref);
      l *= alpha;
#pragma unroll
      for (int c = 0; c < kD; ++c) acc[c] *= alpha;
      uint32_t keep = ~0u;
      if (a.drop.enabled) {
        keep = 0;
#pragma unroll
        for (int g = 0; g < kSub / 8; ++g)
          keep |= dropout_keep8((uint32_t)((j0 >> 3) + g), row_g, a.drop) << (8 * g);
      }
#pragma unroll
      for (int jj = 0; jj < kSub; ++jj) {
        const float p = ex2(sc[jj] - mref);
        l += p;
        const float pt = ((keep >> jj) & 1u) ? p * (a.drop.enabled ? a.drop.rp : 1.f) : 0.f;
#pragma unroll
        for (int c = 0; c < kD; ++c) acc[c] = fmaf(pt, Vs[jj][c], acc[c]);
      }
      m = mn;
    }
  }
  if (i < a.N) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int c = 0; c < kD; ++c) o[base + (size_t)i * st.n + c] = acc[c] * inv;
    a.lse[(size_t)bh * a.N + i] = l > 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
  }
}

// dK, dV: one thread per key row.  Blocks past the nq key tiles take the parts of
// the first ones (BwdArgs::part).
__device__ __forceinline__ void
dkdv_rows(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
          const float* __restrict__ dout, float* __restrict__ dk, float* __restrict__ dv, const Strides& st,
          const Strides& kst, const BwdArgs& a, int jt, int bk) {
  extern __shared__ float dyn_smem[];
  auto KVs = reinterpret_cast<float (*)[kRows][kD + 1]>(dyn_smem);   // [2][kRows][kD + 1]
  __shared__ float Qs[kSub][kD];
  __shared__ float Ds[kSub][kD];
  __shared__ float Ls[kSub], Dv[kSub];
  int chunk = 0;
  const bool cut = a.sink_tiles > 0 && a.sink_chunks > 1;
  if (jt >= a.nq) {
    chunk = (jt - a.nq) % a.sink_chunks;
    jt = (jt - a.nq) / a.sink_chunks;
  } else if (cut && jt < a.sink_tiles) {
    return;
  }
  const int b = bk / a.H_kv, hk = bk % a.H_kv;
  const int r = threadIdx.x;
  const int j = jt * kRows + r;
  int Lk = a.N;
  if (a.mask.seqlens_k) Lk = max(0, min(a.N, a.mask.seqlens_k[b]));
  const size_t kbase = (size_t)b * kst.b + (size_t)hk * kst.h;
  for (int c = 0; c < kD; ++c) {
    KVs[0][r][c] = j < a.N ? k[kbase + (size_t)j * kst.n + c] : 0.f;
    KVs[1][r][c] = j < a.N ? v[kbase + (size_t)j * kst.n + c] : 0.f;
  }
  float gk[kD], gv[kD];
#pragma unroll
  for (int c = 0; c < kD; ++c) { gk[c] = 0.f; gv[c] = 0.f; }
  const bool key_ok = j < Lk;
  const TileList tl = bwd_list(a.mask, jt, a.nq, Lk);
  const float rp = a.drop.enabled ? a.drop.rp : 1.f;
  const bool part = cut && jt < a.sink_tiles;
  const int send = part ? min(tl.n * a.group, (chunk + 1) * a.sink_steps) : tl.n * a.group;
  for (int s = part ? chunk * a.sink_steps : 0; s < send; ++s) {
    const int qti = tl.at(s % tl.n);
    const int h = hk * a.group + s / tl.n;     // query head of this step
    const int bh = b * a.H + h;
    const size_t base = (size_t)b * st.b + (size_t)h * st.h;
    for (int sub = 0; sub < kTile / kSub; ++sub) {
      const int i0 = qti * kTile + sub * kSub;
      __syncthreads();
      for (int e = r; e < kSub * kD; e += kRows) {
        const int ii = i0 + e / kD, c = e % kD;
        Qs[e / kD][c] = ii < a.N ? q[base + (size_t)ii * st.n + c] : 0.f;
        Ds[e / kD][c] = ii < a.N ? dout[base + (size_t)ii * st.n + c] : 0.f;
      }
      if (r < kSub) {
        Ls[r] = a.lse2[(size_t)bh * a.npad + i0 + r];
        Dv[r] = a.dvec[(size_t)bh * a.npad + i0 + r];
      }
      __syncthreads();
      if (!key_ok) continue;
      for (int i4 = 0; i4 < kSub; i4 += kAtOnce) {
        bool see[kAtOnce], some = false;
#pragma unroll
        for (int t = 0; t < kAtOnce; ++t) {
          const int i = i0 + i4 + t;
          see[t] = !(a.mask.causal && j > i) && !(a.mask.window > 0 && j >= a.mask.sinks && i >= j + a.mask.window);
          some |= see[t];
        }
        if (!some) continue;
        float sdot[kAtOnce] = {}, ddot[kAtOnce] = {};
#pragma unroll 8
        for (int c = 0; c < kD; ++c) {
          const float kc = KVs[0][r][c], vc = KVs[1][r][c];
#pragma unroll
          for (int t = 0; t < kAtOnce; ++t) {
            sdot[t] = fmaf(Qs[i4 + t][c], kc, sdot[t]);
            ddot[t] = fmaf(Ds[i4 + t][c], vc, ddot[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < kAtOnce; ++t) {
          if (!see[t]) continue;
          const int ii = i4 + t;
          const float p = ex2(fmaf(sdot[t], a.scale_log2, -Ls[ii]));
          bool kept = true;
          if (a.drop.enabled)
            kept = (dropout_keep8((uint32_t)j >> 3, (uint32_t)bh * (uint32_t)a.N + (uint32_t)(i0 + ii), a.drop) >> (j & 7)) & 1u;
          const float pt = kept ? p * rp : 0.f;
          const float ds = p * ((kept ? ddot[t] * rp : 0.f) - Dv[ii]);
#pragma unroll
          for (int c = 0; c < kD; ++c) {
            gv[c] = fmaf(pt, Ds[ii][c], gv[c]);
            gk[c] = fmaf(ds, Qs[ii][c], gk[c]);
          }
        }
      }
    }
  }
  if (part) {
    float* dst = a.part + ((((size_t)bk * a.sink_tiles + jt) * a.sink_chunks + chunk) * kTile + r) * 2 * kD;
#pragma unroll
    for (int c = 0; c < kD; ++c) {
      dst[c] = gk[c];
      dst[kD + c] = gv[c];
    }
  } else if (j < a.N) {
#pragma unroll
    for (int c = 0; c < kD; ++c) {
      dk[kbase + (size_t)j * kst.n + c] = gk[c] * a.scale;
      dv[kbase + (size_t)j * kst.n + c] = gv[c];
    }
  }
}

// dQ: one thread per query row.
__device__ __forceinline__ void
dq_rows(const float* q, const float* __restrict__ k, const float* __restrict__ v, const float* dout, float* dq,
        const Strides& st, const Strides& kst, const BwdArgs& a, int qt, int bh) {
  extern __shared__ float dyn_smem[];
  auto QDs = reinterpret_cast<float (*)[kRows][kD + 1]>(dyn_smem);   // [2][kRows][kD + 1]
  __shared__ float Ks[kSub][kD];
  __shared__ float Vs[kSub][kD];
  const int b = bh / a.H, h = bh % a.H;
  const int r = threadIdx.x;
  const int i = qt * kRows + r;
  int Lk = a.N;
  if (a.mask.seqlens_k) Lk = max(0, min(a.N, a.mask.seqlens_k[b]));
  const size_t base = (size_t)b * st.b + (size_t)h * st.h;
  for (int c = 0; c < kD; ++c) {
    QDs[0][r][c] = i < a.N ? q[base + (size_t)i * st.n + c] : 0.f;
    QDs[1][r][c] = i < a.N ? dout[base + (size_t)i * st.n + c] : 0.f;
  }
  float g[kD];
#pragma unroll
  for (int c = 0; c < kD; ++c) g[c] = 0.f;
  const size_t kbase = (size_t)b * kst.b + (size_t)(h / a.group) * kst.h;
  const float lse2 = a.lse2[(size_t)bh * a.npad + i];
  const float Di = a.dvec[(size_t)bh * a.npad + i];
  const int jmax = a.mask.causal ? min(Lk - 1, i) : Lk - 1;
  const int jmin = a.mask.window > 0 ? i - a.mask.window + 1 : 0;
  const float rp = a.drop.enabled ? a.drop.rp : 1.f;
  const uint32_t row_g = (uint32_t)bh * (uint32_t)a.N + (uint32_t)i;
  const TileList tl = fwd_list(a.mask, qt, Lk);
  for (int s = 0; s < tl.n; ++s) {
    const int kvt = tl.at(s);
    for (int sub = 0; sub < kTile / kSub; ++sub) {
      const int j0 = kvt * kTile + sub * kSub;
      if (hidden(a.mask, j0, qt * kRows, kRows)) continue;
      __syncthreads();
      for (int e = r; e < kSub * kD; e += kRows) {
        const int jj = j0 + e / kD, c = e % kD;
        Ks[e / kD][c] = jj < a.N ? k[kbase + (size_t)jj * kst.n + c] : 0.f;
        Vs[e / kD][c] = jj < a.N ? v[kbase + (size_t)jj * kst.n + c] : 0.f;
      }
      __syncthreads();
      uint32_t keep = ~0u;
      if (a.drop.enabled) {
        keep = 0;
#pragma unroll
        for (int gg = 0; gg < kSub / 8; ++gg)
          keep |= dropout_keep8((uint32_t)((j0 >> 3) + gg), row_g, a.drop) << (8 * gg);
      }
      for (int j4 = 0; j4 < kSub; j4 += kAtOnce) {
        bool see[kAtOnce], some = false;
#pragma unroll
        for (int t = 0; t < kAtOnce; ++t) {
          const int j = j0 + j4 + t;
          see[t] = j <= jmax && (j >= jmin || j < a.mask.sinks);
          some |= see[t];
        }
        if (!some) continue;
        float sdot[kAtOnce] = {}, ddot[kAtOnce] = {};
#pragma unroll 8
        for (int c = 0; c < kD; ++c) {
          const float qc = QDs[0][r][c], dc = QDs[1][r][c];
#pragma unroll
          for (int t = 0; t < kAtOnce; ++t) {
            sdot[t] = fmaf(qc, Ks[j4 + t][c], sdot[t]);
            ddot[t] = fmaf(dc, Vs[j4 + t][c], ddot[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < kAtOnce; ++t) {
          if (!see[t]) continue;
          const float p = ex2(fmaf(sdot[t], a.scale_log2, -lse2));
          const bool kept = (keep >> (j4 + t)) & 1u;
          const float ds = p * ((kept ? ddot[t] * rp : 0.f) - Di);
#pragma unroll
          for (int c = 0; c < kD; ++c) g[c] = fmaf(ds, Ks[j4 + t][c], g[c]);
        }
      }
    }
  }
  if (i < a.N) {
#pragma unroll
    for (int c = 0; c < kD; ++c) dq[base + (size_t)i * st.n + c] = g[c] * a.scale;
  }
}

// Block u = blockIdx.x + u0: the first `keys` dK and dV, then dQ.  In one launch, as neither fills the GPU when there
// are few heads.
__global__ void __launch_bounds__(kRows, 2)
bwd_simt_kernel(const float* q, const float* __restrict__ k, const float* __restrict__ v, const float* dout, float* dq,
                float* __restrict__ dk, float* __restrict__ dv, Strides st, Strides kst, const BwdArgs a, int keys,
                int u0) {
  const int u = (int)blockIdx.x + u0, per = keys / (a.B * a.H_kv);
  if (u < keys) dkdv_rows(q, k, v, dout, dk, dv, st, kst, a, u % per, u / per);
  else dq_rows(q, k, v, dout, dq, st, kst, a, (u - keys) % a.nq, (u - keys) / a.nq);
}

}  // namespace

cudaError_t launch_fwd_simt(const float* q, const float* k, const float* v, float* o, Strides st,
                            Strides kst, const FwdArgs& a, cudaStream_t s) {
  dim3 grid(a.nq, a.B * a.H);
  if (a.mask.sinks > 0) fwd_simt_kernel<kWindowSinks><<<grid, kRows, 0, s>>>(q, k, v, o, st, kst, a);
  else if (a.mask.window > 0) fwd_simt_kernel<kWindow><<<grid, kRows, 0, s>>>(q, k, v, o, st, kst, a);
  else fwd_simt_kernel<kAllKeys><<<grid, kRows, 0, s>>>(q, k, v, o, st, kst, a);
  return cudaGetLastError();
}

cudaError_t launch_bwd_simt(const float* q, const float* k, const float* v, const float* dout, float* dq,
                            float* dk, float* dv, Strides st, Strides kst, const BwdArgs& a, cudaStream_t s) {
  const int cut = a.sink_tiles > 0 && a.sink_chunks > 1 ? a.sink_tiles * a.sink_chunks : 0;
  const long long keys = (long long)(a.nq + cut) * a.B * a.H_kv, all = keys + (long long)a.nq * a.B * a.H;
  if (all > 0x7fffffff) return cudaErrorInvalidConfiguration;
  constexpr int dyn = 2 * kRows * (kD + 1) * (int)sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(bwd_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  // dQ in the place of Q or dO: dK and dV have to have read them
  const unsigned first = dq == q || dq == dout ? (unsigned)keys : (unsigned)all;
  bwd_simt_kernel<<<first, kRows, dyn, s>>>(q, k, v, dout, dq, dk, dv, st, kst, a, (int)keys, 0);
  if (first < all)
    bwd_simt_kernel<<<(unsigned)all - first, kRows, dyn, s>>>(q, k, v, dout, dq, dk, dv, st, kst, a, (int)keys, (int)first);
  return cudaGetLastError();
}

}  // namespace fa
