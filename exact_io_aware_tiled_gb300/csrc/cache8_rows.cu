// cache8_rows.cu -- new rows into a paged cache of 8-bit codes, and its rows out.
//
// Mathematics.  A page of one K/V head has a scale 2^e, e the smallest whole number
// (-126 at least) with max |x| <= 448 2^e over the rows written to it; its codes
// are E4M3(x 2^-e), round to nearest even.  A power of two scales exactly, so the
// code's is the only rounding, and a page whose scale has to grow is re-scaled
// without a second one except where codes leave E4M3's normal range.  A new row
// that is the first of its page starts the page afresh; otherwise the page keeps
// the larger of its scale and the new rows'.  Zeros alone give the scale 0.
//
// What bounds it: HBM for long chunks (new rows read once, codes written), the
// launch for single tokens.  One CTA per page, K/V head and tensor: nobody else
// writes that page, and the page's maximum is known before its first code.
#include <algorithm>

#include "cache8.cuh"
#include "fp8.cuh"

namespace fa {
namespace {

__device__ __forceinline__ float2 widen2(uint32_t two) {        // two E4M3 codes, exact
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return make_float2(Cvt<__half>::lo(r), Cvt<__half>::hi(r));
}

// |x| of 8 elements, the largest that is finite
template <typename T> __device__ __forceinline__ float amax8(const uint4& v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fabsf(Cvt<T>::lo(w[i])), b = fabsf(Cvt<T>::hi(w[i]));
    m = a < INFINITY ? fmaxf(m, a) : m;
    m = b < INFINITY ? fmaxf(m, b) : m;
  }
  return m;
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126..127

// The scale's exponent for rows up to m > 0
__device__ __forceinline__ int exponent_of(float m) {
  const uint32_t u = __float_as_uint(m);
  return max(-126, (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0));     // 448 = 1.75 2^8
}

// A thread holds up to kHeld 8-element pieces of the page's new rows: each is read once, all at the same time.
constexpr int kHeld = 8, kAppendThreads = 256;
static_assert(kHeld * kAppendThreads * 8 >= 128 * 128, "a page's rows in registers");

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, 3) cache8_append_kernel(const Cache8Rows a, int touched) {
  __shared__ float smax[kAppendThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int u = (int)blockIdx.x;
  const int pi = u % touched;
  u /= touched;
  const int y = u & 1;                               // K, V
  u >>= 1;
  const int hk = u % a.Hkv, b = u / a.Hkv;
  const int tokens = max(0, a.lens[b]), L = min(a.width * a.page, tokens);      // L: those that the table has room for
  const int first = tokens - a.T, from = max(first, 0);   // position of token 0; the first that is written
  if (from >= L) return;
  const int w = (from >> a.lg) + pi, base = w << a.lg;
  if (base >= L) return;
  const int id = a.table[(int64_t)b * a.table_stride + w];
  const int r0 = max(from - base, 0), r1 = min(L - base, a.page);     // rows of the page that are new
  const int per = a.d >> 3, lgp = a.d == 64 ? 3 : 4; // 8-element pieces of a row
  const int n = (r1 - r0) * per;
  const Strides xs = a.xs[y], cs = a.cs[y];
  const T* src = static_cast<const T*>(a.x[y]) + (int64_t)b * xs.b + (int64_t)hk * xs.h + (int64_t)(base + r0 - first) * xs.n;
  uint4 held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = threadIdx.x + k * blockDim.x, row = i >> lgp;
    held[k] = i < n ? *reinterpret_cast<const uint4*>(src + (int64_t)row * xs.n + (i & (per - 1)) * 8) : make_uint4(0u, 0u, 0u, 0u);
  }
  // the rows are on their way before the page is known
  if ((unsigned)id >= (unsigned)a.pages) return;     // an absent page takes nothing
  uint8_t* page = a.code[y] + (int64_t)id * cs.b + (int64_t)hk * cs.h;
  float* scale = a.scale[y] + (size_t)id * a.Hkv + hk;
  const float was = r0 > 0 ? *scale : 0.f;
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) m = amax8<T>(held[k], m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (blockDim.x > 32) {
    if ((threadIdx.x & 31) == 0) smax[threadIdx.x >> 5] = m;
    __syncthreads();
    m = smax[0];
    for (int i = 1; i < (int)blockDim.x >> 5; ++i) m = fmaxf(m, smax[i]);
  }
  const int e = m > 0.f ? exponent_of(m) : -126;
  const float need = m > 0.f ? power_of_two(e) : 0.f;
  const float now = fmaxf(need, was);
  // every thread has read the old scale before one writes the new one
  if (blockDim.x > 32) __syncthreads();
  else __syncwarp();
  if (threadIdx.x == 0 && now != was) *scale = now;
  if (threadIdx.x == 0 && r0 == 0 && now == 0.f) *scale = 0.f;
  if (r0 > 0 && was > 0.f && now > was) {            // the rows that were there, at the new scale
    const float f = was / now;
    const int per16 = a.d >> 4, n16 = r0 * per16;
    for (int i = threadIdx.x; i < n16; i += blockDim.x) {
      const int row = i / per16;
      uint4* at = reinterpret_cast<uint4*>(page + (int64_t)row * cs.n + (i - row * per16) * 16);
      const uint4 v = *at;
      uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 p = widen2(c[k] & 0xFFFFu), q = widen2(c[k] >> 16);
        c[k] = e4m3x4(p.x * f, p.y * f, q.x * f, q.y * f);
      }
      *at = make_uint4(c[0], c[1], c[2], c[3]);
    }
  }
  // 1 / now: a power of two too where the cache was written here
  const float f = now > 0.f ? 1.f / now : 0.f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = threadIdx.x + k * blockDim.x, row = i >> lgp;
    if (i >= n) break;
    const uint32_t t[4] = {held[k].x, held[k].y, held[k].z, held[k].w};
    uint32_t o[2];
#pragma unroll
    for (int y = 0; y < 2; ++y)
      o[y] = e4m3x4(Cvt<T>::lo(t[2 * y]) * f, Cvt<T>::hi(t[2 * y]) * f, Cvt<T>::lo(t[2 * y + 1]) * f,
                    Cvt<T>::hi(t[2 * y + 1]) * f);
    *reinterpret_cast<uint2*>(page + (int64_t)(r0 + row) * cs.n + (i & (per - 1)) * 8) = make_uint2(o[0], o[1]);
  }
}

// Rows out: a thread turns 8 codes into 8 values at a time, so that the lanes' stores lie side by side; zeros behind the
// last row and for absent pages.
constexpr int kReadRows = 64;                        // rows of a CTA
template <typename T>
__global__ void __launch_bounds__(128) cache8_read_kernel(const Cache8Rows a, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int u = (int)blockIdx.x;
  const int n0 = (u % chunks) * kReadRows;
  u /= chunks;
  const int y = u & 1;
  u >>= 1;
  const int hk = u % a.Hkv, b = u / a.Hkv;
  const int L = max(0, min(a.width * a.page, a.lens[b]));
  const int per = a.d >> 3, lgp = a.d == 64 ? 3 : 4;
  const Strides xs = a.xs[y], cs = a.cs[y];
  T* dst = static_cast<T*>(a.x[y]) + (int64_t)b * xs.b + (int64_t)hk * xs.h;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int n = min(kReadRows, a.T - n0) * per;
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * 128) {
    int id[4];
    float sc[4];
    uint2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * 128, at = n0 + (i >> lgp);
      id[k] = i < n && at < L ? table[at >> a.lg] : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * 128, at = n0 + (i >> lgp);
      sc[k] = 0.f;
      v[k] = make_uint2(0u, 0u);
      if ((unsigned)id[k] < (unsigned)a.pages) {
        sc[k] = a.scale[y][(size_t)id[k] * a.Hkv + hk];
        v[k] = *reinterpret_cast<const uint2*>(a.code[y] + (int64_t)id[k] * cs.b + (int64_t)hk * cs.h +
                                              (int64_t)(at & (a.page - 1)) * cs.n + (i & (per - 1)) * 8);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * 128;
      if (i >= n) break;
      const float2 p0 = widen2(v[k].x & 0xFFFFu), p1 = widen2(v[k].x >> 16), p2 = widen2(v[k].y & 0xFFFFu), p3 = widen2(v[k].y >> 16);
      const float s = sc[k];
      // streaming: 27.7 us against 30.7 for 4 x 8 heads x 8,192 rows of 128
      __stcs(reinterpret_cast<uint4*>(dst + (int64_t)(n0 + (i >> lgp)) * xs.n + (i & (per - 1)) * 8),
             make_uint4(Cvt<T>::pack(p0.x * s, p0.y * s), Cvt<T>::pack(p1.x * s, p1.y * s), Cvt<T>::pack(p2.x * s, p2.y * s),
                        Cvt<T>::pack(p3.x * s, p3.y * s)));
    }
  }
}

// Launched over the end of the kernel before it (griddepcontrol.wait before the first access): 0.5 us less a launch.
cudaError_t launch_over(void (*kernel)(Cache8Rows, int), unsigned grid, int threads, cudaStream_t s, const Cache8Rows& a, int n) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3((unsigned)threads);
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a, n);
}

}  // namespace

cudaError_t launch_cache8_append(int dtype, const Cache8Rows& a, cudaStream_t s) {
  const int touched = (a.T + a.page - 2) / a.page + 1;          // pages that T rows can touch
  const long long grid = 2ll * a.B * a.Hkv * std::min(touched, a.width);     // < 2^31, here and below (api.cu)
  // threads that hold kHeld pieces each: 2,047 new rows of 4 sequences and 8 heads of 128 in pages of 64 take 9.8 us with
  // 8 pieces a thread, 15 with 4, in pages of 16 9.7 and 15 (one piece: 46)
  const long long pieces = (long long)std::min(a.T, a.page) * a.d / 8;
  const int threads = (int)std::clamp<long long>((pieces / 8 + 31) / 32 * 32, 32, kAppendThreads);
  const int t = std::min(touched, a.width);
  return dtype == FA_DT_BF16 ? launch_over(cache8_append_kernel<__nv_bfloat16>, (unsigned)grid, threads, s, a, t)
                             : launch_over(cache8_append_kernel<__half>, (unsigned)grid, threads, s, a, t);
}

cudaError_t launch_cache8_read(int dtype, const Cache8Rows& a, cudaStream_t s) {
  const int chunks = (a.T + kReadRows - 1) / kReadRows;
  const long long grid = 2ll * a.B * a.Hkv * chunks;
  return dtype == FA_DT_BF16 ? launch_over(cache8_read_kernel<__nv_bfloat16>, (unsigned)grid, 128, s, a, chunks)
                             : launch_over(cache8_read_kernel<__half>, (unsigned)grid, 128, s, a, chunks);
}

}  // namespace fa
