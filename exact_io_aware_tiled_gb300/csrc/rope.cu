// rope.cu -- rotary positions: q and k rotated by their positions, or
// gradients rotated back.
//
// Mathematics.  Pair i of a row at position p turns by the angle p f_i:
//     (x0, x1) -> m (x0 cos - x1 sin, x1 cos + x0 sin),
// with f_i the pair's inverse frequency and m one factor for all pairs.  The
// transposed map, which the gradient needs, has the sign of sin flipped.
// Pairs are (i, i + rot/2) in the half layout and (2i, 2i + 1) interleaved;
// columns from rot on are copied.
//
// The angle.  p f in float32 is wrong by p f 2^-24 radians: 0.06 at a million,
// more than a 16-bit rounding.  Here the turn f / 2 pi is held as a 64-bit
// binary fraction F = f / 2 pi 2^64 and p F is taken modulo 2^64, which drops
// whole turns exactly; what is left is the fraction of a turn, read as a signed
// number in [-1/2, 1/2) and handed to sincospif.  One float64 product per CTA
// and pair makes F; everything else is integer and float32.  Rounded to float32 the
// fraction is off by up to 2^-25 half turns (9e-8 radians), as much as sincospif's
// own result: float32 outputs lose a fifth to it against 64-bit angles, 16-bit ones
// nothing, and float64 sines are slow on this GPU.
//
// What bounds it: HBM.  Each element is read and written once, and the angles
// are computed, not read.  A thread owns V pairs (16-byte vectors where rot / 2
// allows) of one token and walks over the heads of q and then k, so a sine and
// cosine serve all heads; the heads are split over blockIdx.y only as far as
// the grid needs to fill the GPU.  Measured: 537 MB of GPT-2-medium q and k in
// 93 us (5.8 TB/s, 0.85 of the copy rate), 387 MB with interleaved pairs in 63 us
// (0.90).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "rope.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
  const void* x[2];        // q, k
  void* y[2];
  Strides xs[2], ys[2];
  int heads[2];
  int inplace[2];          // y is x: the copied columns are left alone
  int N, rot, units, hp;   // units: threads per token; hp: heads per blockIdx.y
  uint32_t total;          // B * N * units
  const void* pos;         // int32 / int64 positions, or nullptr: start + n
  int pos64;
  int64_t pos_b, pos_n, start;
  const double* inv_freq;
  float mscale, sgn;
};

// The half layout: V pairs (c0 + e, c0 + rot/2 + e) per rotating thread.
// Interleaved: the V / 2 pairs of one vector; a vector that straddles rot
// rotates its first pairs and copies the rest.
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr int NP = kInter ? (V + 1) / 2 : V;       // pairs of a thread
  // heads whose loads are in flight together.  Measured at d = 128, rot = 48, f16,
  // interleaved, 387 MB: 2 -> 63 us, 4 -> 69, 8 -> 85; half layout, 537 MB of
  // bf16: 2 -> 91, 4 -> 93, 8 -> 110; 63 MB of float32: 2 -> 20.0, 4 -> 18.7 us
  constexpr int HB = kInter ? 2 : 4;
  __shared__ unsigned long long sF[128];
  __shared__ float sM[128];                          // m, or NaN where the frequency is not finite
  const int half = a.rot >> 1;
  // float64 is slow on this GPU: the turns are made once per CTA, not once per thread
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const double f = a.inv_freq[i];
    sF[i] = turns_of(f);
    sM[i] = isfinite(f) ? a.mscale : nanf("");
  }
  __syncthreads();
  const uint32_t t = blockIdx.x * kRopeThreads + threadIdx.x;
  if (t >= a.total) return;
  const uint32_t token = t / (uint32_t)a.units;
  const int u = (int)(t - token * (uint32_t)a.units);
  const uint32_t b = token / (uint32_t)a.N;
  const uint32_t n = token - b * (uint32_t)a.N;
  const int nrot = kInter ? (a.rot + V - 1) / V : half / V;
  const bool rotates = u < nrot;
  const int c0 = kInter || rotates ? u * V : a.rot + (u - nrot) * V;
  using Vec = RVec<T, V>;

  float cs[NP], sn[NP];
  if (rotates) {
    long long p = a.start + (long long)n;
    if (a.pos != nullptr) {
      const int64_t at = (int64_t)b * a.pos_b + (int64_t)n * a.pos_n;
      p = a.pos64 ? static_cast<const long long*>(a.pos)[at] : (long long)static_cast<const int*>(a.pos)[at];
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const int i = kInter ? c0 / 2 + e : c0 + e;
      if (!kInter || i < half) turn(p, sF[i], sM[i], a.sgn * sM[i], cs[e], sn[e]);
    }
  }
  const int first = blockIdx.y * a.hp;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {                      // q's heads, then k's
    const int off = w ? a.heads[0] : 0;
    const int h0 = max(first - off, 0), h1 = min(first + a.hp - off, a.heads[w]);
    if (h0 >= h1 || (!rotates && a.inplace[w])) continue;
    const Strides xs = a.xs[w], ys = a.ys[w];
    const T* src = static_cast<const T*>(a.x[w]) + (int64_t)b * xs.b + (int64_t)h0 * xs.h + (int64_t)n * xs.n + c0;
    T* dst = static_cast<T*>(a.y[w]) + (int64_t)b * ys.b + (int64_t)h0 * ys.h + (int64_t)n * ys.n + c0;
    for (int h = h0; h < h1; h += HB, src += HB * xs.h, dst += HB * ys.h) {
      Vec v0[HB], v1[HB];
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if (h + j >= h1) break;
        v0[j] = *reinterpret_cast<const Vec*>(src + j * xs.h);
        if (!kInter && rotates) v1[j] = *reinterpret_cast<const Vec*>(src + j * xs.h + half);
      }
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if (h + j >= h1) break;
        if (rotates) {
          float x0[V];
          unpack<T, V>(v0[j], x0);
          if constexpr (kInter) {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              if (c0 / 2 + e >= half) continue;
              const float y0 = x0[2 * e], y1 = x0[2 * e + 1];
              x0[2 * e] = y0 * cs[e] - y1 * sn[e];
              x0[2 * e + 1] = y1 * cs[e] + y0 * sn[e];
            }
          } else {
            float x1[V];
            unpack<T, V>(v1[j], x1);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float y0 = x0[e], y1 = x1[e];
              x0[e] = y0 * cs[e] - y1 * sn[e];
              x1[e] = y1 * cs[e] + y0 * sn[e];
            }
            *reinterpret_cast<Vec*>(dst + j * ys.h + half) = pack<T, V>(x1);
          }
          v0[j] = pack<T, V>(x0);
        }
        *reinterpret_cast<Vec*>(dst + j * ys.h) = v0[j];
      }
    }
  }
}

template <typename T, int V, bool kInter>
cudaError_t launch_v(RopeArgs a, int B, int d, int sms, cudaStream_t s) {
  a.units = kInter ? d / V : a.rot / 2 / V + (d - a.rot) / V;
  const unsigned long long total = (unsigned long long)B * a.N * a.units;
  if (total >= (1ull << 32) - kRopeThreads) return cudaErrorInvalidValue;
  a.total = (uint32_t)total;
  const int heads = a.heads[0] + a.heads[1];
  const unsigned gx = (unsigned)((total + kRopeThreads - 1) / kRopeThreads);
  // split the heads until the grid fills the GPU about twice at 1,024 threads a
  // SM (once: 5 % slower for want of balance; 16 times: 12 % slower for sines)
  const long long want = 2ll * sms * 1024 / kRopeThreads;
  int split = (int)std::min<long long>((want + gx - 1) / gx, heads);
  split = std::min(split, 65535);
  a.hp = (heads + split - 1) / split;
  if (a.hp > 4) a.hp = (a.hp + 3) / 4 * 4;          // whole batches of loads
  split = (heads + a.hp - 1) / a.hp;
  rope_kernel<T, V, kInter><<<dim3(gx, (unsigned)split), kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, bool inter, int B, int d, int sms, cudaStream_t s) {
  constexpr int VM = 16 / (int)sizeof(T);
  if (inter) return launch_v<T, VM, true>(a, B, d, sms, s);
  // the widest vector that rot / 2 is a multiple of
  const int half = a.rot / 2;
  if (half % VM == 0) return launch_v<T, VM, false>(a, B, d, sms, s);
  if (VM > 4 && half % 4 == 0) return launch_v<T, 4, false>(a, B, d, sms, s);
  if (half % 2 == 0) return launch_v<T, 2, false>(a, B, d, sms, s);
  return launch_v<T, 1, false>(a, B, d, sms, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of one [B,heads,N,d] tensor: a dimension of one element may carry any stride.
fa_status check_strides(Strides& s, int B, int heads, int N, int d, int unit, bool output) {
  if (N == 1) s.n = d;
  if (heads == 1) s.h = (int64_t)N * s.n;
  if (B == 1) s.b = (int64_t)heads * s.h;
  const int64_t least = output ? 1 : 0;          // an input may be broadcast (stride 0)
  if (s.n < (output ? d : 0) || s.h < least || s.b < least) return FA_ERR_INVALID_ARG;
  if (s.n % unit || s.h % unit || s.b % unit) return FA_ERR_MISALIGNED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rope(const fa_rope_params* p, const void* q, const void* k, void* q_out, void* k_out, void* stream) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 1 || p->H < 1 || p->H_kv < 0 || p->N < 1 || p->d < 1) return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_DT_F32 && p->dtype != FA_DT_F16 && p->dtype != FA_DT_BF16) return FA_ERR_INVALID_ARG;
  if (p->rot < 2 || p->rot > p->d || (p->rot & 1)) return FA_ERR_INVALID_ARG;
  if (p->d % 8 != 0 || p->d > 256) return FA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->mscale)) return FA_ERR_INVALID_ARG;
  if (q == nullptr || q_out == nullptr || p->inv_freq == nullptr) return FA_ERR_INVALID_ARG;
  if (p->H_kv > 0 && (k == nullptr || k_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (!al16(q) || !al16(q_out) || (p->H_kv > 0 && (!al16(k) || !al16(k_out)))) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->inv_freq) & 7u) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->positions) & (p->positions_i64 ? 7u : 3u)) return FA_ERR_MISALIGNED;
  // 32-bit thread index at one pair per thread
  if ((unsigned long long)p->B * p->N * p->d >= (1ull << 32) - 4096) return FA_ERR_UNSUPPORTED;
  const int unit = p->dtype == FA_DT_F32 ? 4 : 8;
  RopeArgs a{};
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out;
  a.xs[0] = {p->q_stride_b, p->q_stride_h, p->q_stride_n};
  a.ys[0] = {p->q_out_stride_b, p->q_out_stride_h, p->q_out_stride_n};
  a.xs[1] = {p->k_stride_b, p->k_stride_h, p->k_stride_n};
  a.ys[1] = {p->k_out_stride_b, p->k_out_stride_h, p->k_out_stride_n};
  a.heads[0] = p->H; a.heads[1] = p->H_kv;
  for (int w = 0; w < (p->H_kv > 0 ? 2 : 1); ++w) {
    fa_status s = check_strides(a.xs[w], p->B, a.heads[w], p->N, p->d, unit, false);
    if (s == FA_OK) s = check_strides(a.ys[w], p->B, a.heads[w], p->N, p->d, unit, true);
    if (s != FA_OK) return s;
    a.inplace[w] = a.x[w] == a.y[w] && std::memcmp(&a.xs[w], &a.ys[w], sizeof(Strides)) == 0;
    if (a.x[w] == a.y[w] && !a.inplace[w]) return FA_ERR_INVALID_ARG;   // rows would overwrite one another
  }
  a.N = p->N; a.rot = p->rot;
  a.pos = p->positions; a.pos64 = p->positions_i64;
  a.pos_b = p->pos_stride_b; a.pos_n = p->pos_stride_n;
  a.start = p->start;
  a.inv_freq = p->inv_freq;
  a.mscale = p->mscale;
  a.sgn = p->backward ? -1.f : 1.f;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool inter = p->interleaved != 0;
  cudaError_t e;
  if (p->dtype == FA_DT_F32) e = launch_rope<float>(a, inter, p->B, p->d, sms, st);
  else if (p->dtype == FA_DT_F16) e = launch_rope<__half>(a, inter, p->B, p->d, sms, st);
  else e = launch_rope<__nv_bfloat16>(a, inter, p->B, p->d, sms, st);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, int64_t original_len,
                              double beta_fast, double beta_slow, double* inv_freq, float* mscale) {
  if (inv_freq == nullptr || mscale == nullptr) return FA_ERR_INVALID_ARG;
  if (rot < 2 || (rot & 1) || !(base > 1.0) || !std::isfinite(base)) return FA_ERR_INVALID_ARG;
  if (scaling < FA_ROPE_NONE || scaling > FA_ROPE_YARN) return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor))) return FA_ERR_INVALID_ARG;
  if (scaling == FA_ROPE_YARN && (original_len < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0)))
    return FA_ERR_INVALID_ARG;
  const int n = rot / 2;
  const double kTwoPi = 6.283185307179586476925;
  double b = base;
  if (scaling == FA_ROPE_NTK && rot > 2) b = base * std::pow(factor, rot / (rot - 2.0));
  double lo = 0.0, hi = 0.0;
  if (scaling == FA_ROPE_YARN) {
    // the (fractional) pair whose wavelength fits `turns` times into the original length
    auto pair_of = [&](double turns) { return rot * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::min(std::ceil(pair_of(beta_slow)), rot - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(b, -2.0 * i / rot);
    if (scaling == FA_ROPE_LINEAR) f /= factor;
    if (scaling == FA_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[i] = f;
  }
  *mscale = scaling == FA_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return FA_OK;
}

}  // extern "C"
