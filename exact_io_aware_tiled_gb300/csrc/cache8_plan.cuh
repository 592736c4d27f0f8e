// cache8_plan.cuh -- how the attention over a paged 8-bit cache (cache8.cu)
// cuts its work: the units of keys that a sequence's rows read, their line's
// equal shares, the places of rows that are cut, and the keys' order in a
// product.
#pragma once
#include "cache8.cuh"

namespace fa {
namespace {

// What a CTA spends on a sequence's rows of a K/V head besides their keys, in units.  us with 0 / 6 / 12 / 16: 64
// sequences of up to 8,191 keys 123 / 97 / 97 / 98, 300 of up to 2,047 193 / 132 / 131 / 137, 8 of 16,384 with 4
// heads 29 / 27 / 25 / 24, 6 of five tokens with a window of 4,096 21 / 17 / 17 / 17.
constexpr int kItemUnits = 12;
// Pieces that are joined at once; 32 against 16: 102 against 98 us, 8 heads of 128 125 against 101, one head of
// 131,072 keys 38 against 26.
constexpr int kGroup = 16;
// Units of one sequence of n tokens, of which the table has room for L: [0, ns) and, behind a gap of `skip`, the others.
struct Units {
  int n, ns, skip;
  // On the line each sequence's rows of a K/V head count kItemUnits more, in front: what a CTA spends on them besides
  // their keys (their q, joins and stores).  Without them the CTAs that drew short sequences ended last.
  FA_PLAN int line() const { return n > 0 ? n + kItemUnits : 0; }
};
// The first key that the window leaves to a query at position p, 0 where it leaves all
FA_PLAN int first_seen(const Cache8Args& a, int p) { return p + 1 > a.window ? p + 1 - a.window : 0; }
template <int KS> FA_PLAN Units units_of(const Cache8Args& a, int n) {
  Units u{0, 0, 0};
  if (n <= 0) return u;
  const int L = min(n, a.cap), hi = (L + KS - 1) / KS;
  int lo = 0;
  if (a.window > 0) lo = min(hi, first_seen(a, n - a.T) / KS);     // the first query's first key
  u.ns = min((min(a.sinks, L) + KS - 1) / KS, lo);
  u.skip = lo - u.ns;
  u.n = u.ns + hi - lo;
  return u;
}

// The CTAs' shares of the line of X units
struct Share {
  long long X, each;       // every CTA has `each` units, the first `more` CTAs one more
  int C, more;
  FA_PLAN void cut(long long units, int ctas) {
    X = units;
    C = ctas;
    if (X < 1ll << 31) {   // a 64-bit division takes as long as a load from L2
      each = (unsigned)X / (unsigned)C;
      more = (int)((unsigned)X - (unsigned)each * (unsigned)C);
    } else {
      each = X / C;
      more = (int)(X - each * C);
    }
  }
  FA_PLAN long long begin(int c) const { return each * c + min(c, more); }
  FA_PLAN int owner(long long x) const {
    const long long wide = (each + 1) * more;
    return (int)(x < wide ? x / (each + 1) : more + (x - wide) / each);
  }
};

// Where piece `piece` of rows that begin in CTA c0 leaves its partial rows: the first in its CTA's second place, as its
// rows begin there, the others, whose rows a CTA before began, in the first
FA_PLAN int piece_slot(int c0, int piece) { return 2 * (c0 + piece) + (piece == 0 ? 1 : 0); }

// Which of the 8 keys of a product's column tile is column n = 2 m + e: any order
// serves, as K's and V's agree.  These let the lanes that read K rows together
// (both e of an m) and those that read V rows together (all m of an e) meet
// different banks of the swizzled tiles.
template <int D> FA_PLAN int key_of(int m, int e) {
  return D == 64 ? ((m & 2) << 1 | e << 1 | ((m & 1) ^ e)) : (((m >> 1) ^ e) << 2 | (m & 1) << 1 | e);
}

}  // namespace
}  // namespace fa
