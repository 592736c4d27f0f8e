// simt_lists.cuh -- which tiles and sub-tiles of the other side the float32
// kernels (simt_f32.cu) visit, under the causal, padding, block-sparse and
// window masks.
#pragma once
#include "common.cuh"

namespace fa {
namespace {

constexpr int kSub = 32;     // staged rows per sub-tile

FA_PLAN int kv_limit_tiles(int Lk) { return (Lk + kTile - 1) / kTile; }

// Number of 128-row tiles on the other side visible from tile `t`, and the
// tile at position s of that list.
struct TileList {
  int n;
  int head, gap;          // steps at the first keys' tiles, and what lies between those and the others
  const int16_t* list;
  FA_PLAN int at(int s) const {
    const int t = s < head ? s : s + gap;
    return list ? (int)list[t] : t;
  }
};

FA_PLAN TileList fwd_list(const MaskArgs& m, int qt, int Lk) {
  TileList tl{0, 0, 0, nullptr};
  int lim = kv_limit_tiles(Lk);
  if (m.causal) lim = min(lim, qt + 1);
  const int lo = m.window > 0 ? max(0, qt * kTile - m.window + 1) / kTile : 0;
  const int tiles = min(sink_tiles(m.sinks), min(lo, lim));
  if (m.row_list) {
    const int16_t* list = m.row_list + (size_t)qt * m.nb;
    const int cnt = m.row_cnt[qt];
    while (tl.head < cnt && list[tl.head] < tiles) ++tl.head;
    int s0 = tl.head;
    while (s0 < cnt && list[s0] < lo) ++s0;
    int n = s0;
    while (n < cnt && list[n] < lim) ++n;
    tl.list = list;
    tl.gap = s0 - tl.head;
    tl.n = tl.head + n - s0;
  } else {
    tl.head = tiles;
    tl.gap = lo - tiles;
    tl.n = tiles + max(0, lim - lo);
  }
  return tl;
}

FA_PLAN TileList bwd_list(const MaskArgs& m, int jt, int nq, int Lk) {
  TileList tl{0, 0, 0, nullptr};
  if (jt * kTile >= Lk) return tl;
  int qlast = nq - 1;   // key j is seen by queries j .. j + w - 1 under a window
  if (m.window > 0 && jt >= sink_tiles(m.sinks)) qlast = min(qlast, (jt * kTile + kTile - 1 + m.window - 1) / kTile);
  if (m.col_list) {
    const int16_t* list = m.col_list + (size_t)jt * m.nb;
    const int cnt = m.col_cnt[jt];
    int s0 = 0;
    if (m.causal) while (s0 < cnt && list[s0] < jt) ++s0;
    int e = s0;
    while (e < cnt && list[e] <= qlast) ++e;
    tl.list = list;
    tl.gap = s0;
    tl.n = e - s0;
  } else {
    tl.gap = m.causal ? jt : 0;
    tl.n = max(0, qlast - tl.gap + 1);
  }
  return tl;
}

// Keys j0 .. j0 + kSub - 1 that none of n queries from i0 on sees under the causal mask, the window and its first
// keys: a sub-tile that a block leaves out, or (forward) a warp: 32 heads x 2,048, window 128 235 -> 211 us (192
// since its kernel knows that there are no first keys), with 4 first keys 330 -> 235.
FA_PLAN bool hidden(const MaskArgs& m, int j0, int i0, int n) {
  return (m.causal && j0 >= i0 + n) || (m.window > 0 && j0 >= m.sinks && j0 + kSub <= i0 - m.window + 1);
}

}  // namespace
}  // namespace fa
