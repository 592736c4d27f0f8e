// The kernels' planning arithmetic, compiled for the host from the headers that the kernels include (test_planning.py).
#include "bwd_items.cuh"
#include "cache8_plan.cuh"
#include "fwd_plan.cuh"
#include "simt_lists.cuh"
#include "sink_plan.h"

using namespace fa;

template <int kWin, typename S> static int walk(const S& s, int* out) {
  for (int i = 0; i < s.n; ++i) out[i] = s.template kv<kWin>(i);
  return s.n;
}

extern "C" {

void plan_constants(int* out) {
  const int c[] = {kItemUnits, kGroup, kCMax, kTile, kFewSinks, kSub};
  for (int i = 0; i < 6; ++i) out[i] = c[i];
}

// ---- the 8-bit cache
void plan_units(int ks, int n, int T, int window, int sinks, int cap, int* out) {
  Cache8Args a{};
  a.T = T; a.window = window; a.sinks = sinks; a.cap = cap;
  const Units u = ks == 64 ? units_of<64>(a, n) : units_of<32>(a, n);
  out[0] = u.n; out[1] = u.ns; out[2] = u.skip; out[3] = u.line();
}
int plan_first_seen(int window, int p) {
  Cache8Args a{};
  a.window = window;
  return first_seen(a, p);
}
void plan_share(long long X, int C, long long* begins) {
  Share s;
  s.cut(X, C);
  for (int c = 0; c <= C; ++c) begins[c] = s.begin(c);
}
void plan_owners(long long X, int C, int n, const long long* x, int* out) {
  Share s;
  s.cut(X, C);
  for (int i = 0; i < n; ++i) out[i] = s.owner(x[i]);
}
int plan_piece_slot(int c0, int piece) { return piece_slot(c0, piece); }
int plan_key(int D, int m, int e) { return D == 64 ? key_of<64>(m, e) : key_of<128>(m, e); }

// ---- windows with first keys
void plan_sink(int B, int H, int H_kv, int N, int d, int dtype, int window, int sinks, int* out) {
  fa_params p{};
  p.B = B; p.H = H; p.H_kv = H_kv; p.N = N; p.d = d; p.dtype = dtype; p.causal = 1; p.window = window;
  const SinkPlan k = sink_plan(&p, sinks);
  const int v[] = {k.window, k.sinks, k.tiles, k.chunks, k.steps, k.few, k.few_chunks};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}

static MaskArgs mask(int causal, int window, int sinks, const int32_t* lens, int nb, const int16_t* rl, const int32_t* rc,
                     const int16_t* cl, const int32_t* cc) {
  MaskArgs m{};
  m.causal = causal; m.window = window; m.sinks = sinks; m.seqlens_k = lens;
  m.nb = nb; m.row_list = rl; m.row_cnt = rc; m.col_list = cl; m.col_cnt = cc;
  return m;
}

// The backward items as the 16-bit kernels take them.  out: 6 integers an item (b, hk, jt, part, n, steps), then its
// steps' query tiles and heads, walked as the kernels walk them; returns the integers written, -1 past `room`.
long long plan_items(int kind, int B, int H, int H_kv, int N, int causal, int window, int sinks, int tiles, int chunks,
                     int steps, const int32_t* lens, int nb, const int16_t* rl, const int32_t* rc, const int16_t* cl,
                     const int32_t* cc, int* out, long long room) {
  BwdArgs a{};
  a.B = B; a.H = H; a.H_kv = H_kv; a.group = H / H_kv; a.N = N;
  a.nq = (N + kTile - 1) / kTile;
  a.mask = mask(causal, window, sinks, lens, nb, rl, rc, cl, cc);
  a.sink_tiles = tiles; a.sink_chunks = chunks; a.sink_steps = steps;
  const int count = kind == kAllKeys ? item_count<kAllKeys>(a) : kind == kWindow ? item_count<kWindow>(a)
                    : kind == kWindowSinks ? item_count<kWindowSinks>(a) : item_count<kWindowFew>(a);
  long long at = 0;
  for (int u = 0; u < count; ++u) {
    const Item it = kind == kAllKeys ? make_item<kAllKeys>(a, u) : kind == kWindow ? make_item<kWindow>(a, u)
                    : kind == kWindowSinks ? make_item<kWindowSinks>(a, u) : make_item<kWindowFew>(a, u);
    if (at + 6 + 2ll * it.steps > room) return -1;
    const int head[] = {it.b, it.hk, it.jt, it.part, it.n, it.steps};
    for (int x : head) out[at++] = x;
    if (it.steps == 0) continue;
    int qu = it.t0 % it.n, hq = it.h0 + it.t0 / it.n;
    for (int t = 0; t < it.steps; ++t) {
      out[at++] = it.qt(qu);
      out[at++] = hq;
      if (++qu == it.n) { qu = 0; ++hq; }
    }
  }
  return at;
}

// The key tiles of a query tile.  which: 0 the two-tile kernels, 1 the one-tile kernel, 2 float32
int plan_forward(int which, int N, int causal, int window, int sinks, int Lk, int nb, const int16_t* rl, const int32_t* rc,
                 int qt, int* out) {
  FwdArgs a{};
  a.N = N;
  a.nq = (N + kTile - 1) / kTile;
  a.mask = mask(causal, window, sinks, nullptr, nb, rl, rc, nullptr, nullptr);
  const int kind = window == 0 ? kAllKeys : sinks == 0 ? kWindow : kWindowSinks;
  if (which == 2) {
    const TileList t = fwd_list(a.mask, qt, Lk);
    for (int i = 0; i < t.n; ++i) out[i] = t.at(i);
    return t.n;
  }
  if (which == 0) {
    if (kind == kAllKeys) return walk<kAllKeys>(make_slot<kAllKeys>(a, qt, Lk), out);
    if (kind == kWindow) return walk<kWindow>(make_slot<kWindow>(a, qt, Lk), out);
    return walk<kWindowSinks>(make_slot<kWindowSinks>(a, qt, Lk), out);
  }
  if (kind == kAllKeys) return walk<kAllKeys>(make_tile1<kAllKeys>(a, qt, Lk), out);
  if (kind == kWindow) return walk<kWindow>(make_tile1<kWindow>(a, qt, Lk), out);
  return walk<kWindowSinks>(make_tile1<kWindowSinks>(a, qt, Lk), out);
}

// The query tiles of a key tile, float32
int plan_f32_backward(int N, int causal, int window, int sinks, int Lk, int nb, const int16_t* cl, const int32_t* cc, int jt,
                      int* out) {
  const MaskArgs m = mask(causal, window, sinks, nullptr, nb, nullptr, nullptr, cl, cc);
  const TileList t = bwd_list(m, jt, (N + kTile - 1) / kTile, Lk);
  for (int i = 0; i < t.n; ++i) out[i] = t.at(i);
  return t.n;
}
int plan_hidden(int causal, int window, int sinks, int j0, int i0, int n) {
  return hidden(mask(causal, window, sinks, nullptr, 0, nullptr, nullptr, nullptr, nullptr), j0, i0, n);
}

}  // extern "C"
