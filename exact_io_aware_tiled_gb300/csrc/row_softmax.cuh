// row_softmax.cuh -- one step of the online softmax on a 128 x 64 score tile in
// tensor memory, one thread per query row (= tensor-memory lane).  Shared by the
// forward kernels with two 128-row score streams and two 128-column accumulators
// per CTA (differential attention, shared prefix).
//
// Tensor memory of a stream (256 columns): S 64 | P of even steps 32 | P of odd
// steps 32 | O 128.  S is free for the next scores as soon as it is in registers,
// and P alternates, so neither the next S nor the next P waits for a product:
// the chain S -> softmax -> P V is bound by its slowest link, the softmax.
#pragma once
#include "common.cuh"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr uint32_t kStream = 256;           // columns of a stream
constexpr uint32_t kColP = 64, kColO = 128; // within a stream

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

// Barrier of a fixed group of warps (an mbarrier whose count is the number of
// warps): bounded like every wait, so that a warp that gave up leaves none behind.
struct WarpMeet {
  uint64_t* bar;
  uint32_t phase;
  __device__ __forceinline__ bool sync(const WaitCtl& ctl) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    return warp_wait(bar, phase++ & 1u, ctl);
  }
};

struct RowSoftmax {
  float m_run = -INFINITY;                // reference maximum, log2 units
  float l_true = 0.f, l_rnd = 0.f;        // sums of the unrounded and of the rounded weights

  // S of this row (64 columns from tS) -> P in 16 bits (32 columns from tP); O
  // (OC columns from tO) rescaled where the reference maximum moved.  Columns
  // c > jl are hidden, with kWin also c < jlo.  `first`: O holds nothing yet.
  // The caller has waited for S, whose issuer has waited for the product that
  // read this P last; s_read() is called once S is in registers, o_ready()
  // returns once the last product into O is done (false: gave up).  Afterwards
  // the caller signals P.
  template <typename T, int OC, bool kWin, typename Read, typename Ready>
  __device__ __forceinline__ bool step(uint32_t tS, uint32_t tP, uint32_t tO, int jl, int jlo, float sl2, bool first,
                                       Read&& s_read, Ready&& o_ready) {
    uint32_t sr[2][32];
    tmem_ld32(tS, sr[0]);
    tmem_ld32(tS + 32, sr[1]);
    tmem_wait_ld();
    reg_fence32(sr[0]);
    reg_fence32(sr[1]);
    tc_fence_before();
    s_read();
    if (jl < 63 || (kWin && jlo > 0)) {
#pragma unroll
      for (int c = 0; c < 64; ++c)
        if (c > jl || (kWin && c < jlo)) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
    }
    // row max: 8 independent chains of 3-input max, then a short tree
    float m8[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) m8[t] = __uint_as_float(sr[0][t]);
#pragma unroll
    for (int c = 8; c < 64; c += 16) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int c0 = c + t, c1 = c + 8 + t;
        m8[t] = (c1 < 64) ? max3f(m8[t], __uint_as_float(sr[c0 >> 5][c0 & 31]), __uint_as_float(sr[c1 >> 5][c1 & 31]))
                          : fmaxf(m8[t], __uint_as_float(sr[c0 >> 5][c0 & 31]));
      }
    }
    const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sl2;
    // the reference maximum moves only when the tile's exceeds it by 2^8: any
    // reference gives the same quotient, and most steps skip the rescale
    const float m_new = mx > m_run + kRescaleThreshold ? mx : m_run;
    const bool moved = m_new != m_run && m_run != -INFINITY;
    const float alpha = moved ? ex2(m_run - m_new) : 1.f;
    m_run = m_new;
    l_true *= alpha;
    l_rnd *= alpha;
    const float nm = (m_run == -INFINITY) ? 0.f : -m_run;
    // P = exp2(S tau log2e - m) in 16 bits, the product's operand type (half a
    // step per weight).  l_true sums the unrounded P for the logsumexp, l_rnd
    // exactly what the product consumes, so O / l_rnd is a convex combination
    // of V rows.
    float lt[4] = {0.f, 0.f, 0.f, 0.f}, lr[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
      const int ch = (c >> 1) & 1;
      float x0, x1;
      fma2(x0, x1, __uint_as_float(sr[c >> 5][c & 31]), __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]), sl2, sl2, nm,
           nm);
      const float p0 = ex2(x0), p1 = ex2(x1);
      add2(lt[2 * ch], lt[2 * ch + 1], p0, p1);
      const uint32_t u = Cvt<T>::pack(p0, p1);
      Cvt<T>::acc2(lr[2 * ch], lr[2 * ch + 1], u);
      pk[c >> 1] = u;
    }
    tmem_st32(tP, pk);
    l_true += (lt[0] + lt[1]) + (lt[2] + lt[3]);
    l_rnd += (lr[0] + lr[1]) + (lr[2] + lr[3]);
    // tcgen05.ld / st are warp-collective: the warp rescales together when any
    // of its rows needs it (alpha is exactly 1 for the others)
    if (__any_sync(0xffffffffu, moved && !first)) {
      if (!o_ready()) return false;
#pragma unroll
      for (int hf = 0; hf < OC / 32; ++hf) {
        uint32_t o[32];
        tmem_ld32(tO + hf * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
        tmem_st32(tO + hf * 32, o);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    return true;
  }
};

}  // namespace
}  // namespace fa
