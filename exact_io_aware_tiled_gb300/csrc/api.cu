// api.cu -- host side of the C ABI declared in include/fa.h.
//
// Validates arguments, lays out the caller's workspace, encodes the TMA
// tensor maps (cuTensorMapEncodeTiled, fetched through the runtime's
// driver-entry-point query so the library needs no -lcuda), and enqueues the
// kernels on the caller's stream.  It never allocates, frees or synchronises
// device memory (fa_check_status excepted) and keeps no mutable global state.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "cache8.cuh"
#include "fa_internal.h"
#include "sink_plan.h"

namespace fa {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t status = 0, rlist = 0, rcnt = 0, clist = 0, ccnt = 0, lse2 = 0, dvec = 0, dqacc = 0, sched = 0, part = 0, few = 0,
         total = 0;
  bool sparse = false;
  int nb = 0, nq = 0, npad = 0;
};

Layout layout(const fa_params* p, bool bwd, const SinkPlan& sk = SinkPlan()) {
  Layout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  L.nq = (p->N + kTile - 1) / kTile;
  L.npad = L.nq * kTile;
  L.status = take(256);
  if (p->block_mask != nullptr) {
    L.sparse = true;
    L.nb = L.nq;
    L.rlist = take((size_t)L.nb * L.nb * sizeof(int16_t));
    L.rcnt = take((size_t)L.nb * sizeof(int32_t));
    L.clist = take((size_t)L.nb * L.nb * sizeof(int16_t));
    L.ccnt = take((size_t)L.nb * sizeof(int32_t));
  }
  if (bwd) {
    const size_t rows = (size_t)p->B * p->H * L.npad;
    L.lse2 = take(rows * sizeof(float));
    L.dvec = take(rows * sizeof(float));
    if (p->dtype != FA_DT_F32) L.dqacc = take((size_t)p->B * p->H * p->N * p->d * sizeof(float));
    L.sched = take(sizeof(int));
    const size_t heads = (size_t)p->B * (p->H_kv == 0 ? p->H : p->H_kv), row = 2 * p->d * sizeof(float);
    if (sk.chunks > 1) L.part = take(heads * sk.tiles * sk.chunks * kTile * row);
    if (sk.few > 0) {
      L.part = take(heads * kFewSinks * row);
      L.few = take((size_t)p->B * p->H * sk.few_chunks * kFewSinks * row);
    }
  }
  L.total = off;
  return L;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

int elem_bytes(int dt) { return dt == FA_DT_F32 ? 4 : 2; }

int hkv_of(const fa_params* p) { return p->H_kv == 0 ? p->H : p->H_kv; }

bool kv_strides_given(const fa_params* p) { return p->kv_stride_b || p->kv_stride_h || p->kv_stride_n; }

// Shape / dtype / stride / alignment checks shared by fa_fwd and fa_bwd.
fa_status check_params(const fa_params* p) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 1 || p->H < 1 || p->N < 1 || p->d < 1) return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_DT_F32 && p->dtype != FA_DT_F16 && p->dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  // d = 64 on every path; d = 128 on the 16-bit tensor-core forward
  if (p->d != 64 && !(p->d == 128 && p->dtype != FA_DT_F32)) return FA_ERR_UNSUPPORTED;
  if (p->stride_n < p->d || p->stride_h < 1 || p->stride_b < 1) return FA_ERR_INVALID_ARG;
  if (!(p->dropout_p >= 0.f && p->dropout_p < 1.f)) return FA_ERR_INVALID_ARG;
  if ((long long)p->B * p->H * p->N >= (1ll << 32)) return FA_ERR_UNSUPPORTED;
  if (p->block_mask != nullptr && p->block_size != kTile) return FA_ERR_UNSUPPORTED;
  if (p->block_mask != nullptr && (p->N + kTile - 1) / kTile > 32767) return FA_ERR_UNSUPPORTED;
  const int64_t unit = 16 / elem_bytes(p->dtype);   // elements per 16 bytes
  if (p->stride_n % unit || p->stride_h % unit || p->stride_b % unit) return FA_ERR_MISALIGNED;
  if (p->o_f32 != nullptr && !aligned16(p->o_f32)) return FA_ERR_MISALIGNED;
  const int hkv = hkv_of(p);
  if (hkv < 1 || p->H % hkv != 0) return FA_ERR_INVALID_ARG;
  if (kv_strides_given(p)) {
    if (p->kv_stride_n < p->d || p->kv_stride_h < 1 || p->kv_stride_b < 1) return FA_ERR_INVALID_ARG;
    if (p->kv_stride_n % unit || p->kv_stride_h % unit || p->kv_stride_b % unit) return FA_ERR_MISALIGNED;
  } else if (hkv != p->H) {
    return FA_ERR_INVALID_ARG;   // K/V with fewer heads need their own strides
  }
  if (p->window < 0) return FA_ERR_INVALID_ARG;
  if (p->window > 0 && !p->causal) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Singleton dimensions carry whatever stride the caller had; normalise them
// so every stride handed to TMA is a valid, representable byte stride.
Strides normalised(Strides s, const fa_params* p, int heads) {
  if (heads == 1) s.h = (int64_t)p->N * s.n;
  if (p->B == 1) s.b = (int64_t)heads * s.h;
  return s;
}

// Strides of Q, O, dO, dQ ([B,H,N,d]).
Strides strides_of(const fa_params* p) { return normalised({p->stride_b, p->stride_h, p->stride_n}, p, p->H); }

// Strides of K, V, dK, dV ([B,H_kv,N,d]).
Strides kv_strides_of(const fa_params* p) {
  if (!kv_strides_given(p)) return strides_of(p);
  return normalised({p->kv_stride_b, p->kv_stride_h, p->kv_stride_n}, p, hkv_of(p));
}

float scale_of(const fa_params* p) {
  return (p->scale > 0.f && std::isfinite(p->scale)) ? p->scale : 1.f / std::sqrt((float)p->d);
}

DropoutArgs dropout_of(const fa_params* p) {
  DropoutArgs d{};
  d.k0 = (uint32_t)(p->seed & 0xFFFFFFFFu);
  d.k1 = (uint32_t)(p->seed >> 32);
  // Philox4x32 key schedule (Salmon et al., SC'11): the key is bumped by the
  // Weyl constants before every round after the first.  It depends on the
  // seed only, so it is computed once here and the kernels read each round's
  // key as a constant.
  for (int r = 0; r < 10; ++r) {
    d.rk0[r] = d.k0 + (uint32_t)r * 0x9E3779B9u;
    d.rk1[r] = d.k1 + (uint32_t)r * 0xBB67AE85u;
  }
  d.off_lo = (uint32_t)(p->offset & 0xFFFFFFFFu);
  d.off_hi = (uint32_t)(p->offset >> 32);
  const double t = std::floor((double)p->dropout_p * 65536.0 + 0.5);
  d.threshold = (uint32_t)t;
  d.rp = 1.f / (1.f - p->dropout_p);
  d.enabled = p->dropout_p > 0.f ? 1 : 0;
  return d;
}

// 4-D map over a [B,heads,N,cols] tensor: dims (cols, N, heads, B), box (box_c, box_r, 1, 1), 128-byte swizzle.
fa_status make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, int cols, int box_c,
                   const fa_params* p, int heads, Strides s, int box_r = kTile) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return FA_ERR_CUDA;
  cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)p->N, (cuuint64_t)heads, (cuuint64_t)p->B};
  cuuint64_t strides[3] = {(cuuint64_t)(s.n * esize), (cuuint64_t)(s.h * esize), (cuuint64_t)(s.b * esize)};
  cuuint32_t box[4] = {(cuuint32_t)box_c, (cuuint32_t)box_r, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, dt, 4, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

fa_status map16(CUtensorMap* m, const void* base, const fa_params* p, int heads, Strides s, int rows = kTile) {
  const CUtensorMapDataType dt =
      p->dtype == FA_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return make_map(m, base, dt, 2, p->d, 64, p, heads, s, rows);   // 64-column (128-byte) boxes
}

MaskArgs mask_of(const fa_params* p, const Layout& L, uint8_t* ws, const SinkPlan& sk) {
  MaskArgs m{};
  m.causal = p->causal ? 1 : 0;
  m.window = sk.window;
  m.sinks = sk.sinks;
  m.seqlens_k = p->seqlens_k;
  if (L.sparse) {
    m.row_list = reinterpret_cast<const int16_t*>(ws + L.rlist);
    m.row_cnt = reinterpret_cast<const int32_t*>(ws + L.rcnt);
    m.col_list = reinterpret_cast<const int16_t*>(ws + L.clist);
    m.col_cnt = reinterpret_cast<const int32_t*>(ws + L.ccnt);
    m.nb = L.nb;
  }
  return m;
}

fa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

fa_status prepare_common(const fa_params* p, const Layout& L, uint8_t* ws, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws + L.status, 0, sizeof(int), st);
  if (e == cudaSuccess && L.sparse)
    e = launch_block_lists(p->block_mask, L.nb, reinterpret_cast<int16_t*>(ws + L.rlist),
                           reinterpret_cast<int32_t*>(ws + L.rcnt), reinterpret_cast<int16_t*>(ws + L.clist),
                           reinterpret_cast<int32_t*>(ws + L.ccnt), st);
  return cuda_status(e);
}

// Records the caller's optional profiling events around the main kernel.
struct ProfScope {
  cudaEvent_t a, b;
  cudaStream_t s;
  ProfScope(const fa_params* p, cudaStream_t st)
      : a((cudaEvent_t)p->prof_start), b((cudaEvent_t)p->prof_stop), s(st) {
    if (a && b) cudaEventRecord(a, s);
  }
  ~ProfScope() {
    if (a && b) cudaEventRecord(b, s);
  }
};

// ---- FP8 forward -------------------------------------------------------------
struct Fp8Layout {
  size_t q8 = 0, k8 = 0, v8t = 0, sq = 0, sk = 0, sv = 0, amax = 0, total = 0;
  int nt = 0, npad = 0;
};

Fp8Layout fp8_layout(const fa_params* p) {
  Fp8Layout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  const int hkv = hkv_of(p);
  L.nt = (p->N + kTile - 1) / kTile;
  L.npad = L.nt * kTile;
  const size_t rq = (size_t)p->B * p->H, rk = (size_t)p->B * hkv;
  L.q8 = take(rq * p->N * p->d);
  L.k8 = take(rk * p->N * p->d);
  L.v8t = take(rk * p->d * L.npad);
  L.sq = take(rq * L.nt * sizeof(float));
  L.sk = take(rk * L.nt * sizeof(float));
  L.sv = take(rk * L.nt * sizeof(float));
  L.amax = take(4 * sizeof(float));
  L.total = off;
  return L;
}

// What the FP8 path supports on top of check_params.
fa_status check_fp8(const fa_params* p, const fa_fp8_params* f) {
  fa_status s = check_params(p);
  if (s != FA_OK) return s;
  if (f == nullptr) return FA_ERR_INVALID_ARG;
  if (p->dtype == FA_DT_F32 || (p->d != 64 && p->d != 128) || p->dropout_p > 0.f) return FA_ERR_UNSUPPORTED;
  if (f->per_tensor != 0 && f->per_tensor != 1) return FA_ERR_INVALID_ARG;
  if (f->signs != nullptr && !aligned16(f->signs)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// 4-D byte map: dims (d0, d1, d2, d3), byte strides of dims 1-3, box (b0, b1, 1, 1).
fa_status map_u8(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                 cuuint32_t b0, cuuint32_t b1, CUtensorMapSwizzle sw) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return FA_ERR_CUDA;
  cuuint32_t box[4] = {b0, b1, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// ---- differential attention ---------------------------------------------------
struct DiffLayout {
  size_t status = 0, rows = 0, dqacc = 0, part = 0, sched = 0, total = 0;
  int nq = 0, npad = 0;
};

int diff_hkv(const fa_diff_params* p) { return p->H_kv == 0 ? p->H : p->H_kv; }

DiffLayout diff_layout(const fa_diff_params* p, bool bwd) {
  DiffLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  L.nq = (p->N + kTile - 1) / kTile;
  L.npad = L.nq * kTile;
  L.status = take(256);
  if (bwd) {
    L.rows = take((size_t)p->B * p->H * L.npad * 4 * sizeof(float));
    L.dqacc = take((size_t)p->B * p->H * 2 * p->N * p->d * sizeof(float));
    L.part = take((size_t)p->B * p->H * L.nq * 16 * sizeof(float));
    L.sched = take(sizeof(int));
  }
  L.total = off;
  return L;
}

// One [B,heads,N,cols] tensor's strides: the dimensions of one element are
// normalised, the others follow the 16-byte rule.
fa_status diff_strides(Strides& s, const fa_diff_params* p, int heads, int cols) {
  if (p->N == 1) s.n = cols;
  if (heads == 1) s.h = (int64_t)p->N * s.n;
  if (p->B == 1) s.b = (int64_t)heads * s.h;
  if (s.n < cols || s.h < 1 || s.b < 1) return FA_ERR_INVALID_ARG;
  if (s.n % 8 || s.h % 8 || s.b % 8) return FA_ERR_MISALIGNED;
  return FA_OK;
}

struct DiffStrides { Strides q, k, v, o, dout; };

fa_status check_diff(const fa_diff_params* p, DiffStrides& s, bool bwd) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 1 || p->H < 1 || p->N < 1 || p->d < 1 || p->H_kv < 0) return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_DT_F32 && p->dtype != FA_DT_F16 && p->dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  if (p->d != 64 || p->dtype == FA_DT_F32) return FA_ERR_UNSUPPORTED;
  const int hkv = diff_hkv(p);
  if (p->H % hkv != 0) return FA_ERR_INVALID_ARG;
  if (p->window < 0) return FA_ERR_INVALID_ARG;
  if (p->window > 0 && !p->causal) return FA_ERR_UNSUPPORTED;
  if (2ll * p->B * p->H * p->N >= (1ll << 32)) return FA_ERR_UNSUPPORTED;
  if (p->lam == nullptr) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->lam) | reinterpret_cast<uintptr_t>(p->seqlens_k)) & 3u) return FA_ERR_MISALIGNED;
  s.q = {p->q_stride_b, p->q_stride_h, p->q_stride_n};
  s.k = {p->k_stride_b, p->k_stride_h, p->k_stride_n};
  s.v = {p->v_stride_b, p->v_stride_h, p->v_stride_n};
  s.o = {p->o_stride_b, p->o_stride_h, p->o_stride_n};
  s.dout = {p->do_stride_b, p->do_stride_h, p->do_stride_n};
  fa_status e;
  if ((e = diff_strides(s.q, p, 2 * p->H, 64)) != FA_OK || (e = diff_strides(s.k, p, 2 * hkv, 64)) != FA_OK ||
      (e = diff_strides(s.v, p, hkv, 128)) != FA_OK || (e = diff_strides(s.o, p, p->H, 128)) != FA_OK)
    return e;
  return bwd ? diff_strides(s.dout, p, p->H, 128) : FA_OK;
}

float diff_scale(const fa_diff_params* p) {
  return (p->scale > 0.f && std::isfinite(p->scale)) ? p->scale : 1.f / std::sqrt((float)p->d);
}

// A 16-bit [B,heads,N,cols] map with boxes of 64 columns and `rows` rows.
fa_status diff_map(CUtensorMap* m, const void* base, const fa_diff_params* p, int heads, int cols, Strides s, int rows) {
  fa_params q{};
  q.B = p->B;
  q.N = p->N;
  return make_map(m, base, p->dtype == FA_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  2, cols, 64, &q, heads, s, rows);
}

// ---- attention over a shared prefix -------------------------------------------
struct PrefixStrides { Strides q, o, kp, vp, k, v; };

// One tensor of nb x nh x n rows of d columns (see diff_strides).
fa_status row_strides(Strides& s, int nb, int nh, int n, int d) {
  if (n <= 1) s.n = d;
  if (nh <= 1) s.h = (int64_t)std::max(n, 1) * s.n;
  if (nb <= 1) s.b = (int64_t)std::max(nh, 1) * s.h;
  if (s.n < d || s.h < 1 || s.b < 1) return FA_ERR_INVALID_ARG;
  if (s.n % 8 || s.h % 8 || s.b % 8) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// The problem with H_kv filled in, its strides normalised.
fa_status check_prefix(const fa_prefix_params* in, fa_prefix_params& p, PrefixStrides& s) {
  if (in == nullptr) return FA_ERR_INVALID_ARG;
  p = *in;
  if (p.B < 1 || p.H < 1 || p.T < 1 || p.d < 1 || p.H_kv < 0 || p.P < 0 || p.M < 0) return FA_ERR_INVALID_ARG;
  if (p.dtype != FA_DT_F32 && p.dtype != FA_DT_F16 && p.dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  if ((p.d != 64 && p.d != 128) || p.dtype == FA_DT_F32) return FA_ERR_UNSUPPORTED;
  if (p.lam != nullptr && p.d != 64) return FA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(p.lam) & 3u) return FA_ERR_MISALIGNED;
  const int maps = p.lam != nullptr ? 2 : 1, dv = maps * p.d;      // score heads per head, value columns
  if (p.H_kv == 0) p.H_kv = p.H;
  if (p.H % p.H_kv != 0) return FA_ERR_INVALID_ARG;
  if ((double)maps * p.B * p.H * p.T >= (double)(1 << 26) || p.P > (1 << 28) || p.M > (1 << 28)) return FA_ERR_UNSUPPORTED;
  s.q = {p.q_stride_b, p.q_stride_h, p.q_stride_n};
  s.o = {p.o_stride_b, p.o_stride_h, p.o_stride_n};
  s.k = {p.k_stride_b, p.k_stride_h, p.k_stride_n};
  s.v = {p.v_stride_b, p.v_stride_h, p.v_stride_n};
  s.kp = {0, p.kp_stride_h, p.kp_stride_n};
  s.vp = {0, p.vp_stride_h, p.vp_stride_n};
  fa_status e;
  if ((e = row_strides(s.q, p.B, maps * p.H, p.T, p.d)) != FA_OK || (e = row_strides(s.o, p.B, p.H, p.T, dv)) != FA_OK)
    return e;
  if (p.M > 0 && ((e = row_strides(s.k, p.B, maps * p.H_kv, p.M, p.d)) != FA_OK ||
                  (e = row_strides(s.v, p.B, p.H_kv, p.M, dv)) != FA_OK))
    return e;
  if (p.P > 0 && ((e = row_strides(s.kp, 1, maps * p.H_kv, p.P, p.d)) != FA_OK ||
                  (e = row_strides(s.vp, 1, p.H_kv, p.P, dv)) != FA_OK))
    return e;
  return FA_OK;
}

// ---- paged cache in 8 bits ------------------------------------------------------
struct Cache8Strides { Strides q, o, k, v, kc, vc; };

// strides in bytes of a [pages,H_kv,page,d] code array
fa_status code_strides(Strides& s, const fa_cache8_params& p) {
  if (p.H_kv == 1) s.h = (int64_t)p.page * s.n;
  if (p.pages == 1) s.b = (int64_t)p.H_kv * s.h;
  if (s.n < p.d || s.h < 1 || s.b < 1) return FA_ERR_INVALID_ARG;
  if (s.n % 16 || s.h % 16 || s.b % 16) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// The problem with H_kv filled in, its strides normalised.  rows: append and read (k, v), else the attention (q, o)
fa_status check_cache8(const fa_cache8_params* in, fa_cache8_params& p, Cache8Strides& s, bool rows) {
  if (in == nullptr) return FA_ERR_INVALID_ARG;
  p = *in;
  if (p.B < 1 || p.H < 1 || p.T < 1 || p.d < 1 || p.H_kv < 0 || p.pages < 1 || p.width < 1) return FA_ERR_INVALID_ARG;
  if (p.dtype != FA_DT_F32 && p.dtype != FA_DT_F16 && p.dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  if ((p.d != 64 && p.d != 128) || p.dtype == FA_DT_F32) return FA_ERR_UNSUPPORTED;
  if (p.page != 16 && p.page != 32 && p.page != 64 && p.page != 128) return FA_ERR_UNSUPPORTED;
  if (p.H_kv == 0) p.H_kv = p.H;
  if (p.H % p.H_kv != 0 || p.window < 0 || p.sinks < 0) return FA_ERR_INVALID_ARG;
  if (p.B > 1 && p.table_stride < p.width) return FA_ERR_INVALID_ARG;
  if (p.seqlens_k == nullptr || p.table == nullptr) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p.seqlens_k) | reinterpret_cast<uintptr_t>(p.table)) & 3u) return FA_ERR_MISALIGNED;
  const double most = 2147483648.0;
  if ((long long)p.width * p.page > (1 << 28) || (double)p.pages * p.H_kv >= most) return FA_ERR_UNSUPPORTED;
  if (rows) {
    if ((double)p.B * p.H_kv * (p.T / 16 + 2.0) * 2 >= most || p.T > (1 << 30)) return FA_ERR_UNSUPPORTED;   // CTAs, rows
  } else {
    if ((double)p.B * p.H * p.T >= (double)(1 << 26)) return FA_ERR_UNSUPPORTED;
    // 32-bit units (32 keys and up, 16 more for each sequence): of all sequences, and of one over heads and row tiles
    const double units = p.width * p.page / 32 + 16.0;
    if (p.B * units >= most || units * p.H_kv * ((double)(p.H / p.H_kv) * p.T / 8 + 1) >= most) return FA_ERR_UNSUPPORTED;
  }
  s.kc = {p.kc_stride_p, p.kc_stride_h, p.kc_stride_n};
  s.vc = {p.vc_stride_p, p.vc_stride_h, p.vc_stride_n};
  fa_status e;
  if ((e = code_strides(s.kc, p)) != FA_OK || (e = code_strides(s.vc, p)) != FA_OK) return e;
  if (rows) {
    s.k = {p.k_stride_b, p.k_stride_h, p.k_stride_n};
    s.v = {p.v_stride_b, p.v_stride_h, p.v_stride_n};
    if ((e = row_strides(s.k, p.B, p.H_kv, p.T, p.d)) != FA_OK) return e;
    return row_strides(s.v, p.B, p.H_kv, p.T, p.d);
  }
  s.q = {p.q_stride_b, p.q_stride_h, p.q_stride_n};
  s.o = {p.o_stride_b, p.o_stride_h, p.o_stride_n};
  if ((e = row_strides(s.q, p.B, p.H, p.T, p.d)) != FA_OK) return e;
  return row_strides(s.o, p.B, p.H, p.T, p.d);
}

fa_status cache8_pointers(const void* kc, const void* vc, const float* ks, const float* vs) {
  if (!kc || !vc || !ks || !vs) return FA_ERR_INVALID_ARG;
  if (!aligned16(kc) || !aligned16(vc) || ((reinterpret_cast<uintptr_t>(ks) | reinterpret_cast<uintptr_t>(vs)) & 3u))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

Cache8Rows cache8_rows(const fa_cache8_params& p, const Cache8Strides& s, const void* kc, const void* vc,
                       const float* ks, const float* vs, const void* k, const void* v) {
  Cache8Rows a{};
  a.B = p.B; a.Hkv = p.H_kv; a.T = p.T; a.d = p.d;
  a.page = p.page; a.pages = p.pages; a.width = p.width;
  while ((1 << a.lg) < p.page) ++a.lg;
  a.lens = p.seqlens_k;
  a.table = p.table;
  a.table_stride = p.table_stride;
  a.x[0] = const_cast<void*>(k); a.x[1] = const_cast<void*>(v);
  a.xs[0] = s.k; a.xs[1] = s.v;
  a.code[0] = static_cast<uint8_t*>(const_cast<void*>(kc));
  a.code[1] = static_cast<uint8_t*>(const_cast<void*>(vc));
  a.cs[0] = s.kc; a.cs[1] = s.vc;
  a.scale[0] = const_cast<float*>(ks); a.scale[1] = const_cast<float*>(vs);
  return a;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_workspace_size(const fa_params* p) {
  if (p == nullptr || p->N < 1) return 256;
  return layout(p, false).total;
}

size_t fa_bwd_workspace_size(const fa_params* p) {
  if (p == nullptr || p->N < 1 || p->B < 1 || p->H < 1) return 256;
  return layout(p, true).total;
}

fa_status fa_fwd(const fa_params* p, const void* q, const void* k, const void* v, void* o, float* lse, void* ws,
                 size_t ws_bytes, void* stream) {
  return fa_fwd_sinks(p, 0, q, k, v, o, lse, ws, ws_bytes, stream);
}

fa_status fa_fwd_sinks(const fa_params* p, int32_t sinks, const void* q, const void* k, const void* v, void* o,
                       float* lse, void* ws, size_t ws_bytes, void* stream) {
  fa_status s = check_params(p);
  if (s != FA_OK) return s;
  if (sinks < 0) return FA_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const SinkPlan sk = sink_plan(p, sinks);
  const Layout L = layout(p, false);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const Strides sd = strides_of(p), skv = kv_strides_of(p);
  const int hkv = hkv_of(p);

  FwdArgs a{};
  a.B = p->B; a.H = p->H; a.N = p->N;
  a.group = p->H / hkv;
  a.nq = L.nq;
  a.npairs = (L.nq + 1) / 2;
  a.scale_log2 = scale_of(p) * 1.4426950408889634f;
  a.mask = mask_of(p, L, w, sk);
  a.drop = dropout_of(p);
  a.fwd_kernel = p->fwd_kernel;
  a.lse = lse;
  a.o_f32 = p->o_f32;
  a.status = reinterpret_cast<int*>(w + L.status);

  if ((s = prepare_common(p, L, w, st)) != FA_OK) return s;
  if (p->dtype == FA_DT_F32) {
    if (p->o_f32 != nullptr) return FA_ERR_UNSUPPORTED;   // O is already float32
    ProfScope prof(p, st);
    return cuda_status(
        launch_fwd_simt((const float*)q, (const float*)k, (const float*)v, (float*)o, sd, skv, a, st));
  }
  CUtensorMap mq, mk, mv, mo;
  if ((s = map16(&mq, q, p, p->H, sd)) != FA_OK || (s = map16(&mk, k, p, hkv, skv)) != FA_OK ||
      (s = map16(&mv, v, p, hkv, skv)) != FA_OK || (s = map16(&mo, o, p, p->H, sd)) != FA_OK)
    return s;
  ProfScope prof(p, st);
  return cuda_status(launch_fwd_tc(p->dtype, p->d, mq, mk, mv, mo, a, st));
}

fa_status fa_bwd(const fa_params* p, const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  return fa_bwd_sinks(p, 0, q, k, v, o, dout, lse, dq, dk, dv, ws, ws_bytes, stream);
}

size_t fa_bwd_sinks_workspace_size(const fa_params* p, int32_t sinks) {
  if (p == nullptr || p->N < 1 || p->B < 1 || p->H < 1) return 256;
  const int hkv = p->H_kv == 0 ? p->H : p->H_kv;
  if (hkv < 1 || p->H % hkv != 0) return 256;
  return layout(p, true, sink_plan(p, sinks)).total;
}

fa_status fa_bwd_sinks(const fa_params* p, int32_t sinks, const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                       void* stream) {
  fa_status s = check_params(p);
  if (s != FA_OK) return s;
  if (sinks < 0) return FA_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_MISALIGNED;
  const SinkPlan sk = sink_plan(p, sinks);
  const Layout L = layout(p, true, sk);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const Strides sd = strides_of(p), skv = kv_strides_of(p);
  const int hkv = hkv_of(p);

  BwdArgs a{};
  a.B = p->B; a.H = p->H; a.N = p->N;
  a.group = p->H / hkv;
  a.H_kv = hkv;
  a.nq = L.nq;
  a.npad = L.npad;
  a.scale = scale_of(p);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.mask = mask_of(p, L, w, sk);
  a.sink_tiles = sk.tiles;
  a.sink_chunks = sk.chunks;
  a.sink_steps = sk.steps;
  a.part = reinterpret_cast<float*>(w + L.part);
  a.few = sk.few;
  a.few_chunks = sk.few_chunks;
  a.few_part = reinterpret_cast<float*>(w + L.few);
  if (sk.few > 0) a.mask.sinks = 0;
  a.dk = dk;
  a.dv = dv;
  a.kst = skv;
  a.drop = dropout_of(p);
  a.lse2 = reinterpret_cast<const float*>(w + L.lse2);
  a.dvec = reinterpret_cast<const float*>(w + L.dvec);
  a.status = reinterpret_cast<int*>(w + L.status);

  if ((s = prepare_common(p, L, w, st)) != FA_OK) return s;
  float* dqacc = p->dtype == FA_DT_F32 ? nullptr : reinterpret_cast<float*>(w + L.dqacc);
  a.sched = reinterpret_cast<int*>(w + L.sched);
  // The bf16 backward kernels fold tau into dS (dS' = (tau dP - tau D) o P
  // with one packed FMA against -tau D), so their dQ, dK products come out
  // scaled; the fp16 and fp32 kernels read D itself.
  const float dscale = p->dtype == FA_DT_BF16 ? -a.scale : 1.f;
  float* const lse2 = reinterpret_cast<float*>(w + L.lse2);
  float* const dvec = reinterpret_cast<float*>(w + L.dvec);
  cudaError_t e = a.few > 0 ? launch_sink_few(p->dtype, p->d, q, k, v, o, dout, sd, lse, lse2, dvec, dqacc, dscale, a, st)
                            : launch_bwd_prep(p->dtype, o, dout, sd, lse, p->B, p->H, p->N, L.npad, p->d, lse2, dvec, dqacc,
                                              a.sched, dscale, st);
  if (e != cudaSuccess) return FA_ERR_CUDA;
  if (p->dtype == FA_DT_F32) {
    ProfScope prof(p, st);
    e = launch_bwd_simt((const float*)q, (const float*)k, (const float*)v, (const float*)dout, (float*)dq, (float*)dk,
                        (float*)dv, sd, skv, a, st);
    return cuda_status(e == cudaSuccess ? launch_sink_sum(p->dtype, p->d, a, a.scale, st) : e);
  }
  // d = 64: 128-row query steps; d = 128: 64-row query steps (Q, dO and the
  // float32 dQ accumulator are moved in 64-row boxes)
  CUtensorMap mq, mk, mv, mdo, macc;
  const int qrows = p->d == 128 ? 64 : kTile;
  Strides acc_st{(int64_t)p->H * p->N * p->d, (int64_t)p->N * p->d, p->d};
  if ((s = map16(&mq, q, p, p->H, sd, qrows)) != FA_OK || (s = map16(&mk, k, p, hkv, skv)) != FA_OK ||
      (s = map16(&mv, v, p, hkv, skv)) != FA_OK || (s = map16(&mdo, dout, p, p->H, sd, qrows)) != FA_OK ||
      (s = make_map(&macc, dqacc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p->d, 32, p, p->H, acc_st, qrows)) != FA_OK)
    return s;
  // 32-byte row pieces (16 columns of 16 bits) can go out as single 32-byte stores
  a.dkv_v8 = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0 &&
             skv.n % 16 == 0 && skv.h % 16 == 0 && skv.b % 16 == 0;
  {
    ProfScope prof(p, st);
    e = p->d == 128 ? launch_bwd_tc128(p->dtype, mq, mk, mv, mdo, macc, a, st)
                    : launch_bwd_tc(p->dtype, mq, mk, mv, mdo, macc, a, st);
    if (e != cudaSuccess) return FA_ERR_CUDA;
  }
  const float kscale = p->dtype == FA_DT_BF16 ? 1.f : a.scale;   // bf16: dK comes out scaled
  if (a.few > 0) return cuda_status(launch_few_finish(p->dtype, p->d, a, kscale, dqacc, dq, sd, st));
  if (launch_sink_sum(p->dtype, p->d, a, kscale, st) != cudaSuccess) return FA_ERR_CUDA;
  return cuda_status(launch_dq_convert(p->dtype, dqacc, dq, sd, p->B, p->H, p->N, p->d, st));
}

fa_status fa_check_status(const void* ws, void* stream) {
  if (ws == nullptr) return FA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return FA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
  return v == 0 ? FA_OK : (fa_status)v;
}

fa_status fa_dropout_mask(const fa_params* p, int32_t b, int32_t h, int32_t row0, int32_t nrows, uint8_t* out,
                          void* stream) {
  if (p == nullptr || out == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 1 || p->H < 1 || p->N < 1) return FA_ERR_INVALID_ARG;
  if (!(p->dropout_p >= 0.f && p->dropout_p < 1.f)) return FA_ERR_INVALID_ARG;
  if (b < 0 || b >= p->B || h < 0 || h >= p->H || row0 < 0 || nrows < 0 || row0 + (int64_t)nrows > p->N)
    return FA_ERR_INVALID_ARG;
  if ((long long)p->B * p->H * p->N >= (1ll << 32)) return FA_ERR_UNSUPPORTED;
  return cuda_status(launch_dropout_mask(dropout_of(p), p->H, p->N, b, h, row0, nrows, out,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_selftest_wait_timeout(void* ws, int32_t* out, uint64_t* out_ns, void* stream) {
  if (ws == nullptr || out == nullptr || out_ns == nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned16(ws) || (reinterpret_cast<uintptr_t>(out_ns) & 7u) != 0) return FA_ERR_MISALIGNED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), st);
  if (e == cudaSuccess)
    e = launch_wait_selftest(static_cast<int*>(ws), reinterpret_cast<int*>(out),
                             reinterpret_cast<unsigned long long*>(out_ns), st);
  return cuda_status(e);
}

fa_status fa_fp8_buffer_layout(const fa_params* p, fa_fp8_layout* out) {
  if (p == nullptr || out == nullptr || p->B < 1 || p->H < 1 || p->N < 1 || p->d < 1) return FA_ERR_INVALID_ARG;
  const int hkv = hkv_of(p);
  if (hkv < 1 || p->H % hkv != 0) return FA_ERR_INVALID_ARG;
  const Fp8Layout L = fp8_layout(p);
  out->q8 = L.q8; out->k8 = L.k8; out->v8t = L.v8t;
  out->sq = L.sq; out->sk = L.sk; out->sv = L.sv; out->amax = L.amax;
  out->total = L.total;
  return FA_OK;
}

fa_status fa_fp8_quantize(const fa_params* p, const fa_fp8_params* f, const void* q, const void* k, const void* v,
                          void* buf, size_t buf_bytes, void* stream) {
  fa_status s = check_fp8(p, f);
  if (s != FA_OK) return s;
  if (!q || !k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return FA_ERR_MISALIGNED;
  const Fp8Layout L = fp8_layout(p);
  if (buf == nullptr || buf_bytes < L.total || !aligned16(buf)) return FA_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(buf);
  const int hkv = hkv_of(p);
  Fp8QuantArgs a{};
  a.src[0] = q; a.src[1] = k; a.src[2] = v;
  a.st[0] = strides_of(p); a.st[1] = a.st[2] = kv_strides_of(p);
  a.heads[0] = p->H; a.heads[1] = a.heads[2] = hkv;
  a.dst[0] = w + L.q8; a.dst[1] = w + L.k8; a.dst[2] = w + L.v8t;
  a.scale[0] = reinterpret_cast<float*>(w + L.sq);
  a.scale[1] = reinterpret_cast<float*>(w + L.sk);
  a.scale[2] = reinterpret_cast<float*>(w + L.sv);
  a.amax = reinterpret_cast<float*>(w + L.amax);
  a.signs = f->signs;
  a.B = p->B; a.N = p->N; a.nt = L.nt; a.npad = L.npad;
  a.d = p->d;
  return cuda_status(launch_fp8_quantize(p->dtype, a, f->per_tensor, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_fwd_fp8(const fa_params* p, const fa_fp8_params* f, const void* buf, size_t buf_bytes, void* o,
                     float* lse, void* ws, size_t ws_bytes, void* stream) {
  fa_status s = check_fp8(p, f);
  if (s != FA_OK) return s;
  if (!o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const Fp8Layout Q = fp8_layout(p);
  if (buf == nullptr || buf_bytes < Q.total || !aligned16(buf)) return FA_ERR_WORKSPACE;
  const Layout L = layout(p, false);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const uint8_t* qb = static_cast<const uint8_t*>(buf);
  const int hkv = hkv_of(p);

  FwdArgs a{};
  a.B = p->B; a.H = p->H; a.N = p->N;
  a.group = p->H / hkv;
  a.nq = L.nq;
  a.npairs = (L.nq + 1) / 2;
  a.scale_log2 = scale_of(p) * 1.4426950408889634f;
  a.mask = mask_of(p, L, w, sink_plan(p, 0));
  a.drop = dropout_of(p);
  a.lse = lse;
  a.o_f32 = p->o_f32;
  a.status = reinterpret_cast<int*>(w + L.status);
  a.f8.sq = reinterpret_cast<const float*>(qb + Q.sq);
  a.f8.sk = reinterpret_cast<const float*>(qb + Q.sk);
  a.f8.sv = reinterpret_cast<const float*>(qb + Q.sv);
  a.f8.signs = f->signs;
  a.f8.nt = Q.nt;
  a.f8.o_bf16 = p->dtype == FA_DT_BF16 ? 1 : 0;

  const cuuint64_t N = (cuuint64_t)p->N, npad = (cuuint64_t)Q.npad, H = (cuuint64_t)p->H, Hk = (cuuint64_t)hkv;
  const cuuint64_t d = (cuuint64_t)p->d;
  // Q8 / K8 rows are d bytes: 64-byte swizzle for d = 64, 128-byte for d = 128
  const CUtensorMapSwizzle swqk = p->d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap mq, mk, mv, mo;
  if ((s = map_u8(&mq, qb + Q.q8, {d, N, H, (cuuint64_t)p->B}, {d, d * N, d * N * H}, (cuuint32_t)d, kTile, swqk)) !=
          FA_OK ||
      (s = map_u8(&mk, qb + Q.k8, {d, N, Hk, (cuuint64_t)p->B}, {d, d * N, d * N * Hk}, (cuuint32_t)d, kTile, swqk)) !=
          FA_OK ||
      (s = map_u8(&mv, qb + Q.v8t, {npad, d, Hk, (cuuint64_t)p->B}, {npad, d * npad, d * npad * Hk}, kTile,
                  (cuuint32_t)d, CU_TENSOR_MAP_SWIZZLE_128B)) != FA_OK ||
      (s = map16(&mo, o, p, p->H, strides_of(p))) != FA_OK)
    return s;
  if ((s = prepare_common(p, L, w, st)) != FA_OK) return s;
  ProfScope prof(p, st);
  return cuda_status(launch_fwd_fp8(p->d, mq, mk, mv, mo, a, st));
}

size_t fa_diff_fwd_workspace_size(const fa_diff_params* p) {
  if (p == nullptr || p->N < 1) return 256;
  return diff_layout(p, false).total;
}

size_t fa_diff_bwd_workspace_size(const fa_diff_params* p) {
  if (p == nullptr || p->N < 1 || p->B < 1 || p->H < 1 || p->d < 1) return 256;
  return diff_layout(p, true).total;
}

fa_status fa_diff_fwd(const fa_diff_params* p, const void* q, const void* k, const void* v, void* o, void* o2,
                      float* lse, void* ws, size_t ws_bytes, void* stream) {
  DiffStrides sd;
  fa_status s = check_diff(p, sd, false);
  if (s != FA_OK) return s;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(o2) || !aligned16(lse))
    return FA_ERR_MISALIGNED;
  const DiffLayout L = diff_layout(p, false);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int hkv = diff_hkv(p);
  DiffFwdArgs a{};
  a.B = p->B; a.H = p->H; a.N = p->N;
  a.group = p->H / hkv;
  a.nq = L.nq;
  a.causal = p->causal ? 1 : 0;
  a.window = p->window;
  a.scale_log2 = diff_scale(p) * 1.4426950408889634f;
  a.seqlens_k = p->seqlens_k;
  a.lam = p->lam;
  a.lse = lse;
  a.has_o2 = o2 != nullptr ? 1 : 0;
  a.status = reinterpret_cast<int*>(w + L.status);
  a.sched = a.status + 1;
  CUtensorMap mq, mk, mv, mo, mo2;
  if ((s = diff_map(&mq, q, p, 2 * p->H, 64, sd.q, kTile)) != FA_OK ||
      (s = diff_map(&mk, k, p, 2 * hkv, 64, sd.k, kTile)) != FA_OK ||
      (s = diff_map(&mv, v, p, hkv, 128, sd.v, kTile)) != FA_OK ||
      (s = diff_map(&mo, o, p, p->H, 128, sd.o, kTile)) != FA_OK ||
      (s = diff_map(&mo2, o2 != nullptr ? o2 : o, p, p->H, 128, sd.o, kTile)) != FA_OK)
    return s;
  if (cudaMemsetAsync(a.status, 0, 2 * sizeof(int), st) != cudaSuccess) return FA_ERR_CUDA;
  return cuda_status(launch_diff_fwd(p->dtype, mq, mk, mv, mo, mo2, a, st));
}

fa_status fa_diff_bwd(const fa_diff_params* p, const void* q, const void* k, const void* v, const void* o,
                      const void* o2, const void* dout, const float* lse, void* dq, void* dk, void* dv, float* dlam,
                      void* ws, size_t ws_bytes, void* stream) {
  DiffStrides sd;
  fa_status s = check_diff(p, sd, true);
  if (s != FA_OK) return s;
  if (!q || !k || !v || !o || !o2 || !dout || !lse || !dq || !dk || !dv || !dlam) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(o2) || !aligned16(dout) ||
      !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      (reinterpret_cast<uintptr_t>(dlam) & 3u))
    return FA_ERR_MISALIGNED;
  const DiffLayout L = diff_layout(p, true);
  if (ws == nullptr || ws_bytes < L.total || !aligned16(ws)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int hkv = diff_hkv(p);
  DiffBwdArgs a{};
  a.B = p->B; a.H = p->H; a.H_kv = hkv; a.N = p->N;
  a.group = p->H / hkv;
  a.nq = L.nq; a.npad = L.npad;
  a.causal = p->causal ? 1 : 0;
  a.window = p->window;
  a.scale = diff_scale(p);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.seqlens_k = p->seqlens_k;
  a.lam = p->lam;
  a.rows = reinterpret_cast<const float*>(w + L.rows);
  a.dlam_part = reinterpret_cast<float*>(w + L.part);
  a.sched = reinterpret_cast<int*>(w + L.sched);
  a.status = reinterpret_cast<int*>(w + L.status);
  a.dk = dk; a.dv = dv;
  a.kst = sd.k; a.vst = sd.v;
  a.dkv_v8 = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0 &&
             (sd.k.n | sd.k.h | sd.k.b | sd.v.n | sd.v.h | sd.v.b) % 16 == 0;
  float* dqacc = reinterpret_cast<float*>(w + L.dqacc);
  a.dqacc = dqacc;
  CUtensorMap mq, mk, mv, mdo;
  if ((s = diff_map(&mq, q, p, 2 * p->H, 64, sd.q, 64)) != FA_OK ||
      (s = diff_map(&mk, k, p, 2 * hkv, 64, sd.k, kTile)) != FA_OK ||
      (s = diff_map(&mv, v, p, hkv, 128, sd.v, kTile)) != FA_OK ||
      (s = diff_map(&mdo, dout, p, p->H, 128, sd.dout, 64)) != FA_OK)
    return s;
  if (cudaMemsetAsync(w + L.status, 0, sizeof(int), st) != cudaSuccess) return FA_ERR_CUDA;
  // bf16 kernels fold tau into dS; see diff_bwd.cu
  const float c1 = p->dtype == FA_DT_BF16 ? a.scale : 1.f;
  cudaError_t e = launch_diff_prep(p->dtype, o, o2, sd.o, dout, sd.dout, lse, p->lam, p->B, p->H, p->N, L.npad, c1,
                                   reinterpret_cast<float*>(w + L.rows), dqacc, a.sched, st);
  if (e == cudaSuccess) e = launch_diff_d1(p->dtype, q, k, v, dout, sd.q, sd.dout, c1, lse, a, st);
  if (e == cudaSuccess) e = launch_diff_bwd(p->dtype, mq, mk, mv, mdo, a, st);
  if (e == cudaSuccess) e = launch_dq_convert(p->dtype, dqacc, dq, sd.q, p->B, 2 * p->H, p->N, 64, st);
  if (e == cudaSuccess) e = launch_diff_dlam(a.dlam_part, dlam, p->B, p->H, a.group, L.nq, st);
  return cuda_status(e);
}

size_t fa_prefix_workspace_size(const fa_prefix_params* in) {
  fa_prefix_params p;
  PrefixStrides sd;
  if (check_prefix(in, p, sd) != FA_OK) return 256;
  return prefix_workspace(&p);
}

fa_status fa_prefix_fwd(const fa_prefix_params* in, const void* q, const void* k_prefix, const void* v_prefix,
                        const void* k, const void* v, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  fa_prefix_params p;
  PrefixStrides sd;
  fa_status s = check_prefix(in, p, sd);
  if (s != FA_OK) return s;
  if (!q || !o || !lse || p.seqlens_k == nullptr) return FA_ERR_INVALID_ARG;
  if ((p.P > 0 && (!k_prefix || !v_prefix)) || (p.M > 0 && (!k || !v))) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(p.seqlens_k) & 3u))
    return FA_ERR_MISALIGNED;
  if ((p.P > 0 && (!aligned16(k_prefix) || !aligned16(v_prefix))) || (p.M > 0 && (!aligned16(k) || !aligned16(v))))
    return FA_ERR_MISALIGNED;
  if (ws == nullptr || !aligned16(ws) || ws_bytes < prefix_workspace(&p)) return FA_ERR_WORKSPACE;
  CUtensorMap m[4] = {};
  const int maps = p.lam != nullptr ? 2 : 1;
  const CUtensorMapDataType dt =
      p.dtype == FA_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  fa_params bn{};
  bn.B = 1;
  bn.N = p.P;
  if (p.P > 0 && ((s = make_map(&m[0], k_prefix, dt, 2, p.d, 64, &bn, maps * p.H_kv, sd.kp, 32)) != FA_OK ||
                  (s = make_map(&m[1], v_prefix, dt, 2, maps * p.d, 64, &bn, p.H_kv, sd.vp, 32)) != FA_OK))
    return s;
  bn.B = p.B;
  bn.N = p.M;
  if (p.M > 0 && ((s = make_map(&m[2], k, dt, 2, p.d, 64, &bn, maps * p.H_kv, sd.k, 32)) != FA_OK ||
                  (s = make_map(&m[3], v, dt, 2, maps * p.d, 64, &bn, p.H_kv, sd.v, 32)) != FA_OK))
    return s;
  const float scale = (p.scale > 0.f && std::isfinite(p.scale)) ? p.scale : 1.f / std::sqrt((float)p.d);
  return cuda_status(launch_prefix(&p, m, q, sd.q, o, sd.o, lse, scale * 1.4426950408889634f,
                                   static_cast<uint8_t*>(ws), reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_cache8_append(const fa_cache8_params* in, const void* k, const void* v, void* k_cache, void* v_cache,
                           float* k_scale, float* v_scale, void* stream) {
  fa_cache8_params p;
  Cache8Strides sd;
  fa_status s = check_cache8(in, p, sd, true);
  if (s != FA_OK || (s = cache8_pointers(k_cache, v_cache, k_scale, v_scale)) != FA_OK) return s;
  if (!k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return FA_ERR_MISALIGNED;
  return cuda_status(launch_cache8_append(p.dtype, cache8_rows(p, sd, k_cache, v_cache, k_scale, v_scale, k, v),
                                          reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_cache8_read(const fa_cache8_params* in, const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, void* k, void* v, void* stream) {
  fa_cache8_params p;
  Cache8Strides sd;
  fa_status s = check_cache8(in, p, sd, true);
  if (s != FA_OK || (s = cache8_pointers(k_cache, v_cache, k_scale, v_scale)) != FA_OK) return s;
  if (!k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return FA_ERR_MISALIGNED;
  return cuda_status(launch_cache8_read(p.dtype, cache8_rows(p, sd, k_cache, v_cache, k_scale, v_scale, k, v),
                                        reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_cache8_workspace_size(const fa_cache8_params* in) {
  fa_cache8_params p;
  Cache8Strides sd;
  if (check_cache8(in, p, sd, false) != FA_OK) return 256;
  return cache8_workspace(&p);
}

fa_status fa_cache8_fwd(const fa_cache8_params* in, const void* q, const void* k_cache, const void* v_cache,
                        const float* k_scale, const float* v_scale, void* o, float* lse, void* ws, size_t ws_bytes,
                        void* stream) {
  fa_cache8_params p;
  Cache8Strides sd;
  fa_status s = check_cache8(in, p, sd, false);
  if (s != FA_OK || (s = cache8_pointers(k_cache, v_cache, k_scale, v_scale)) != FA_OK) return s;
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_MISALIGNED;
  if (ws == nullptr || !aligned16(ws) || ws_bytes < cache8_workspace(&p)) return FA_ERR_WORKSPACE;
  const Cache8Rows rows = cache8_rows(p, sd, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr);
  // boxes of up to one stage of the kernel; rows of d bytes: 64-byte swizzle for d = 64, 128-byte for d = 128
  const cuuint32_t box = (cuuint32_t)std::min(p.page, p.d == 64 ? 64 : 32);
  const CUtensorMapSwizzle sw = p.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t d = (cuuint64_t)p.d, n = (cuuint64_t)p.page, h = (cuuint64_t)p.H_kv, np = (cuuint64_t)p.pages;
  CUtensorMap m[2];
  for (int y = 0; y < 2; ++y) {
    const Strides& c = rows.cs[y];
    if ((s = map_u8(&m[y], rows.code[y], {d, n, h, np}, {(cuuint64_t)c.n, (cuuint64_t)c.h, (cuuint64_t)c.b},
                    (cuuint32_t)p.d, box, sw)) != FA_OK)
      return s;
  }
  Cache8Args a{};
  a.B = p.B; a.H = p.H; a.Hkv = p.H_kv; a.T = p.T; a.G = p.H / p.H_kv;
  a.page = p.page; a.lg = rows.lg; a.pages = p.pages; a.width = p.width; a.cap = p.width * p.page;
  a.window = p.window;
  a.sinks = p.sinks;
  a.q = q; a.o = o; a.qs = sd.q; a.os = sd.o;
  a.lse = lse;
  a.lens = p.seqlens_k; a.table = p.table; a.table_stride = p.table_stride;
  a.ks = k_scale; a.vs = v_scale;
  a.scale_log2 = ((p.scale > 0.f && std::isfinite(p.scale)) ? p.scale : 1.f / std::sqrt((float)p.d)) * 1.4426950408889634f;
  return cuda_status(launch_cache8_fwd(p.dtype, p.d, m[0], m[1], a, static_cast<uint8_t*>(ws),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_MISALIGNED: return "FA_ERR_MISALIGNED";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
  }
  return "FA_ERR_UNKNOWN";
}

int32_t fa_version(void) { return 105; }

}  // extern "C"
