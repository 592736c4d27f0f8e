// bwd_items.cuh -- the work items of the backward kernels (head dims 64 and
// 128): which query tiles see a 128-key tile of one K/V head, under the
// causal, padding, block-sparse and sliding-window masks.
#pragma once
#include "common.cuh"

namespace fa {
namespace {

// One work item: key tile jt of K/V head hk of batch b, and its steps:
// every query tile that sees the key tile, for each of the g query heads
// that share the K/V head (head-major: step t is tile t % n of query head
// h0 + t / n; the loops track both with counters).
struct Item {
  int b, hk, jt, Lk;
  int n;                  // query tiles per query head
  int i0;                 // first query tile (dense)
  int h0;                 // first query head of the group
  const int16_t* list;    // sparse list or nullptr
  int steps;              // n * g; of a first key tile's item, its part of them
  int t0;                 // kWindowSinks: the first step's number among the tile's
  int part;               // where dK and dV go: -1 the tensors, else this place of BwdArgs::part
  FA_PLAN int qt(int u) const { return list ? (int)list[u] : i0 + u; }
};

// Work items of the launch.
template <int kWin> FA_PLAN int item_count(const BwdArgs& a) {
  const int heads = a.B * a.H_kv;
  if constexpr (kWin == kWindowSinks) return heads * (a.sink_tiles * a.sink_chunks + a.nq - a.sink_tiles);
  return a.nq * heads;
}

// Under kWindowSinks the items of the first key tiles come first, the longest ones: every query tile sees those, so
// that one item of them would outlast all others, and each is cut into sink_chunks items of sink_steps steps.
template <int kWin>
FA_PLAN Item make_item(const BwdArgs& a, int u) {
  Item it;
  int bk, chunk = 0;
  bool first_keys = false;
  it.t0 = 0;
  it.part = -1;
  if constexpr (kWin == kWindowSinks) {
    const int first = a.B * a.H_kv * a.sink_tiles * a.sink_chunks;
    if (u < first) {
      first_keys = true;
      if (a.sink_chunks > 1) it.part = u;
      const int tile = u / a.sink_chunks;
      chunk = u - tile * a.sink_chunks;
      bk = tile / a.sink_tiles;
      it.jt = tile - bk * a.sink_tiles;
    } else {
      const int rest = a.nq - a.sink_tiles;
      bk = (u - first) / rest;
      it.jt = a.sink_tiles + (u - first) - bk * rest;
    }
  } else {
    bk = u / a.nq;
    it.jt = u - bk * a.nq;
    if (kWin == kWindowFew && it.jt == 0) it.part = bk;
  }
  it.b = bk / a.H_kv;
  it.hk = bk - it.b * a.H_kv;
  it.Lk = a.N;
  if (a.mask.seqlens_k != nullptr) it.Lk = max(0, min(a.N, a.mask.seqlens_k[it.b]));
  it.list = nullptr;
  it.i0 = a.mask.causal ? it.jt : 0;
  it.h0 = it.hk * a.group;
  it.n = 0;
  // last query tile that sees this key tile: under a sliding window of w keys,
  // key j is seen by queries j .. j + w - 1.  kAllKeys knows of no window: tested for at run time, one that is not
  // there costs the backward kernel 606 us instead of 584 (GPT-2-medium, causal).
  int qlast = a.nq - 1;
  if (kWin != kAllKeys && !first_keys) qlast = min(qlast, (it.jt * kTile + kTile - 1 + a.mask.window - 1) / kTile);
  if (it.jt * kTile < it.Lk) {
    if (a.mask.col_list != nullptr) {
      const int16_t* list = a.mask.col_list + (size_t)it.jt * a.mask.nb;
      const int cnt = a.mask.col_cnt[it.jt];
      int s0 = 0;
      if (a.mask.causal) while (s0 < cnt && list[s0] < it.jt) ++s0;
      int e = s0;
      while (e < cnt && list[e] <= qlast) ++e;
      it.list = list + s0;
      it.n = e - s0;
    } else {
      it.n = max(0, qlast - it.i0 + 1);
    }
  }
  it.steps = it.n * a.group;
  if constexpr (kWin == kWindowSinks) {
    if (it.part >= 0) {
      it.t0 = chunk * a.sink_steps;
      it.steps = max(0, min(a.sink_steps, it.steps - it.t0));
    }
  }
  return it;
}

}  // namespace
}  // namespace fa
