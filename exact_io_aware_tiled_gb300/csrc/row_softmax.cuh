// row_softmax.cuh -- one step of the online softmax on a score tile of 128 rows in
// tensor memory, one thread per query row (= tensor-memory lane).  Shared by the
// forward kernels whose P lies over S (differential attention, shared prefix).
#pragma once
#include "common.cuh"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;   // log2 units

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

struct RowSoftmax {
  float m_run = -INFINITY;                // reference maximum, log2 units
  float l_true = 0.f, l_rnd = 0.f;        // sums of the unrounded and of the rounded weights

  // S of this row (NC columns from tS) -> P in 16 bits over its first NC / 2
  // columns; O (OC columns from tO) rescaled where the reference maximum moved.
  // Columns c > jl are hidden, with kWin also c < jlo.  `first`: O holds
  // nothing yet.  The caller has waited for S; o_ready() returns once the last
  // product into O is done (false: gave up).  The caller calls tmem_wait_st, a
  // fence and the arrival afterwards.
  template <typename T, int NC, int OC, bool kWin, typename Ready>
  __device__ __forceinline__ bool step(uint32_t tS, uint32_t tO, int jl, int jlo, float sl2, bool first,
                                       Ready&& o_ready) {
    uint32_t sr[NC / 32][32];
#pragma unroll
    for (int cc = 0; cc < NC / 32; ++cc) tmem_ld32(tS + cc * 32, sr[cc]);
    tmem_wait_ld();
#pragma unroll
    for (int cc = 0; cc < NC / 32; ++cc) reg_fence32(sr[cc]);
    if (jl < NC - 1 || (kWin && jlo > 0)) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c > jl || (kWin && c < jlo)) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
    }
    // row max: 8 independent chains of 3-input max, then a short tree
    float m8[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) m8[t] = __uint_as_float(sr[0][t]);
#pragma unroll
    for (int c = 8; c < NC; c += 16) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int c0 = c + t, c1 = c + 8 + t;
        m8[t] = (c1 < NC) ? max3f(m8[t], __uint_as_float(sr[c0 >> 5][c0 & 31]), __uint_as_float(sr[c1 >> 5][c1 & 31]))
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
#pragma unroll
    for (int hf = 0; hf < NC / 64; ++hf) {
      uint32_t pk[32];
#pragma unroll
      for (int c2 = 0; c2 < 64; c2 += 2) {
        const int c = hf * 64 + c2;
        const int ch = (c >> 1) & 1;
        float x0, x1;
        fma2(x0, x1, __uint_as_float(sr[c >> 5][c & 31]), __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]), sl2, sl2, nm,
             nm);
        const float p0 = ex2(x0), p1 = ex2(x1);
        add2(lt[2 * ch], lt[2 * ch + 1], p0, p1);
        const uint32_t u = Cvt<T>::pack(p0, p1);
        Cvt<T>::acc2(lr[2 * ch], lr[2 * ch + 1], u);
        pk[c2 >> 1] = u;
      }
      tmem_st32(tS + hf * 32, pk);     // over this row's S, which is in registers
    }
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
    return true;
  }
};

}  // namespace
}  // namespace fa
