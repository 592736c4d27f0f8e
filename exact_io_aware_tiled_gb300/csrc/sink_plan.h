// sink_plan.h -- window and first keys of a call, and how the backward pass
// cuts the items of the first key tiles.
#pragma once
#include <algorithm>

#include "fa_internal.h"

namespace fa {
namespace {

// The window and its first keys as the kernels take them (a window or first keys that hide nothing: none of either),
// and the items of the first key tiles in the backward pass.
struct SinkPlan {
  int window = 0, sinks = 0;
  int tiles = 0, chunks = 0, steps = 0;
  int few = 0, few_chunks = 0;   // backward, 16 bits: see BwdArgs
};

SinkPlan sink_plan(const fa_params* p, int32_t sinks) {
  SinkPlan k;
  k.window = p->window < p->N ? p->window : 0;       // the kernels add a key's index to a window < N
  if (sinks <= 0 || k.window <= 0) return k;
  if (sinks >= p->N) {
    k.window = 0;
    return k;
  }
  k.sinks = sinks;
  const int hkv = p->H_kv == 0 ? p->H : p->H_kv;
  const long long nq = (p->N + kTile - 1) / kTile, g = p->H / hkv, steps = nq * g, heads = (long long)p->B * hkv;
  // An item of a first key tile may take a CTA's whole share of all steps (query tiles at key tiles), as it starts
  // among the first: cutting it further costs more, in dK and dV that go through float32, than it balances.  us,
  // backward in one run, items of 8 / 16 / a share's steps: 64 heads of 64 x 4,096, window 512, 9 first keys 264 / 256 /
  // 243 (32 steps, one item each), 8 padded sequences x 4 K/V heads x 2,047 with 3 query heads and 150 first keys 147 /
  // 140 / 135.  At least 16 steps; float32, whose steps are
  // longer and whose blocks are two on an SM, 2: with 1 / 2 32 heads x 2,048 take 760 / 715 us, 2 heads x 1,000 119 / 127.
  // No more than about four items for each CTA: a part takes 64 KB (d = 128: 128 KB).  Up to kFewSinks first keys of 16
  // bits go the way of sink_few.cu instead, with both sides' times.
  const bool f32 = p->dtype == FA_DT_F32;
  if (!f32 && sinks <= kFewSinks) {
    // the CTAs of launch_sink_few, 3 (d = 128: 2) on an SM, in one round where that fills 0.7 of it, else in four
    const long long all = (long long)p->B * p->H, slots = 152 * (p->d == 128 ? 2 : 3);
    const long long one = slots / all, cut = 10 * one * all >= 7 * slots ? one : (4 * slots + all - 1) / all;
    k.few = sinks;
    k.few_chunks = (int)std::max<long long>(1, std::min({cut, nq * kTile / 64, 256 / g}));
    return k;
  }
  k.tiles = (sinks + kTile - 1) / kTile;
  const long long span = std::min<long long>(nq, (p->window + kTile - 1) / kTile + 1);
  const long long share = heads * g * (nq * span + k.tiles * nq) / (f32 ? 2 * 152 : 152);
  const long long least = std::max<long long>(f32 ? 2 : 16, share);
  const long long most = std::max<long long>(1, 4 * 152 / (heads * k.tiles));
  const long long chunks = std::max<long long>(1, std::min((steps + least / 2) / least, most));
  k.steps = (int)((steps + chunks - 1) / chunks);
  k.chunks = (int)((steps + k.steps - 1) / k.steps);
  return k;
}

}  // namespace
}  // namespace fa
