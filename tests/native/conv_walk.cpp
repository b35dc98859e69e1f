// The rows that the packed convolution's walk loads and stores, for boundaries of any contents, by
// the kernel's own index functions; exits 1 at the first one out of range.  For boundaries as they
// should be, every row of a sequence is computed exactly once, with its own history.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "seq_walk.h"

using std::max;
using std::min;

static void need(bool ok, const char* what, const std::vector<int>& cu, int tokens, int H, int c0) {
  if (ok) return;
  std::printf("%s: tokens %d, history %d, chunk at %d, boundaries", what, tokens, H, c0);
  for (int v : cu) std::printf(" %d", v);
  std::printf("\n");
  std::exit(1);
}

static void walk(const std::vector<int>& cu, int tokens, int H, int c0, int first, std::vector<int>* done) {
  constexpr int K = 8;
  const int nseq = (int)cu.size() - 1;
  const int lo = max(cu[0], 0), hi = min(cu[nseq], tokens), tend = min(c0 + K, hi);
  int t = max(c0, lo), s = first, turns = 0;
  while (t < tend) {
    need(++turns < 1000, "walk without an end", cu, tokens, H, c0);
    const int end = min(cu[s + 1], hi);
    if (end <= t) {
      if (++s >= nseq) break;
      continue;
    }
    const sss::ConvPiece p = sss::conv_piece(cu[s], end, t, c0, tend, H);
    need(p.next > t, "no progress", cu, tokens, H, c0);
    if (!p.mine) {
      t = p.next;
      continue;
    }
    need(p.beg <= t && p.next <= tokens && t >= 0, "rows", cu, tokens, H, c0);
    if (t > p.beg) {
      need(t - H >= 0, "history before the tensor", cu, tokens, H, c0);
    } else {  // the slot's new contents: rows end - H .. end - 1 of the sequence
      for (int k = 0; k < H; ++k) {
        const int q = end - p.beg + k - H;
        if (q >= 0) need(p.beg + q >= 0 && p.beg + q < tokens, "last rows", cu, tokens, H, c0);
      }
    }
    if (done) {
      need(t == p.beg ? cu[s] == t : t - H >= cu[s], "history of another sequence", cu, tokens, H, c0);
      for (int r = t; r < p.next; ++r) ++(*done)[r];
    }
    t = p.next;
  }
}

int main() {
  const int big = 0x7FFFFFFF;
  std::mt19937 rng(1);
  for (int a = -2; a <= 12; ++a)
    for (int b = -2; b <= 12; ++b)
      for (int c = -2; c <= 12; ++c)
        for (int H = 0; H < 8; ++H)
          for (int c0 = 0; c0 < 10; c0 += 8)
            for (int first = 0; first < 2; ++first) walk({a, b, c}, 10, H, c0, first, nullptr);
  for (int i = 0; i < 40000; ++i) {
    const int nseq = 1 + (int)(rng() % 6), tokens = 1 + (int)(rng() % 60), H = (int)(rng() % 8);
    std::vector<int> cu;
    for (int s = 0; s <= nseq; ++s) {
      const unsigned kind = rng() % 8;
      cu.push_back(kind == 0 ? -big - 1 : kind == 1 ? big : (int)(rng() % 80) - 10);
    }
    if (i & 1) std::sort(cu.begin(), cu.end());
    for (int c0 = 0; c0 < tokens; c0 += 8)
      for (int first = 0; first < nseq; ++first) walk(cu, tokens, H, c0, first, nullptr);
  }
  for (int i = 0; i < 40000; ++i) {  // as they should be: not decreasing, in [0, tokens]
    const int nseq = 1 + (int)(rng() % 8), tokens = 1 + (int)(rng() % 60), H = (int)(rng() % 8);
    std::vector<int> cu, done(tokens, 0);
    for (int s = 0; s <= nseq; ++s) cu.push_back((int)(rng() % (unsigned)(tokens + 1)));
    std::sort(cu.begin(), cu.end());
    for (int c0 = 0; c0 < tokens; c0 += 8) {
      const int t = max(c0, cu[0]);
      int s = (int)(std::upper_bound(cu.begin(), cu.end(), t) - cu.begin()) - 1;  // the last boundary <= t
      walk(cu, tokens, H, c0, min(max(s, 0), nseq - 1), &done);
    }
    for (int r = 0; r < tokens; ++r)
      need(done[r] == (r >= cu[0] && r < cu[nseq] ? 1 : 0), "a row not computed once", cu, tokens, H, r);
  }
  std::printf("ok\n");
}
