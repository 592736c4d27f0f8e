// prefix.cuh -- arguments shared by the two kernels of the shared-prefix attention.
#pragma once
#include "common.cuh"

namespace fa {

constexpr int kKT = 32;          // rows of the K / V maps' boxes; keys per stage of the register-product kernel

struct PArgs {
  int B, H, Hkv, T, G;         // H, Hkv: score heads of q and k; G = H / Hkv
  int P, M;
  int R, r;                    // rows of a K/V head: B*G*T against the prefix, G*T against an own cache
  int ptile, stile;            // row tiles: 16, 32 or 64; the prefix also 256 (tensor-memory kernel)
  int pt, st;                  // row tiles per head
  int pchunk, schunk;          // keys per split (multiples of 64, pchunk of 128 with 256-row tiles)
  int np, ns;                  // splits
  int fold;                    // tensor-memory kernel: a CTA works at two splits of one 128-row tile
  int pitems, items;           // prefix items and all items of prefix_kernel
  const void* q;
  Strides qs;
  const int32_t* lens;
  float scale_log2;
  float* part;                 // [rows][D] unnormalised O
  float4* stat;                // [rows]: max (log2), true sum, sum of the rounded weights
  long long srow0;             // first own-cache row of part / stat
  const float* lam;            // differential form (kDiff): device [H / 2], else nullptr
  int* status;
  int* sched;                  // work counter, cleared with the status word
};

// The differential form has two score heads per head pair and one value head for
// both: score head 2 p + x is map x of pair p, in q and in k alike.
template <bool kDiff> __device__ __forceinline__ int value_head(int hk) { return kDiff ? hk >> 1 : hk; }
// j-th query head of the group that reads K head hk
template <bool kDiff> __device__ __forceinline__ int query_head(const PArgs& a, int hk, int j) {
  return kDiff ? 2 * ((hk >> 1) * a.G + j) + (hk & 1) : hk * a.G + j;
}

// Token t of sequence b in the j-th query head that reads K head hk.
template <typename T, bool kDiff>
__device__ __forceinline__ const T* prefix_row(const PArgs& a, int hk, int b, int j, int t) {
  return static_cast<const T*>(a.q) + (int64_t)b * a.qs.b + (int64_t)query_head<kDiff>(a, hk, j) * a.qs.h + (int64_t)t * a.qs.n;
}

// Many rows against the prefix (prefix_tc.cu): items of 256 rows and pchunk keys, or of
// up to 128 rows and two splits.
// d: columns of q and k; the differential form (a.lam set) has d = 64 and 128 value columns.
cudaError_t launch_prefix_tc(int dtype, int d, const CUtensorMap& k, const CUtensorMap& v, const PArgs& a,
                             cudaStream_t s);

}  // namespace fa
