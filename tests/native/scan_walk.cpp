// The rows, workspace chunks and state slots that the packed scan's passes take, for boundaries of
// any contents, by the kernels' own index functions; exits 1 at the first one out of range.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "seq_walk.h"

using std::max;
using std::min;

static void need(bool ok, const char* what, const std::vector<int>& cu, int tokens, int K, int c0) {
  if (ok) return;
  std::printf("%s: tokens %d, chunk of %d at %d, boundaries", what, tokens, K, c0);
  for (int v : cu) std::printf(" %d", v);
  std::printf("\n");
  std::exit(1);
}

static void check(const std::vector<int>& cu, int tokens, int K) {
  const int nseq = (int)cu.size() - 1, chunks = (tokens + K - 1) / K;
  const int lo = max(cu[0], 0), hi = min(cu[nseq], tokens);
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int c0 = chunk * K, tend1 = c0 + K;
    if (chunk + 1 < chunks && tend1 > lo && tend1 < hi)  // pass 1
      for (int s = 0; s < nseq; ++s) {
        if (min(cu[s + 1], hi) <= tend1) continue;
        const int beg = min(max(cu[s], 0), tend1), t = max(beg, c0);
        need(t >= 0 && tend1 <= tokens, "rows of pass 1", cu, tokens, K, c0);
      }
    const int tend = min(tend1, hi);
    for (int first = 0; first < nseq; ++first) {  // pass 2, whichever sequence the search finds
      int t = max(c0, lo), s = first, turns = 0;
      while (t < tend) {
        need(++turns < 1000, "walk without an end", cu, tokens, K, c0);
        const int end = min(cu[s + 1], hi);
        if (end <= t) {
          if (++s >= nseq) break;
          continue;
        }
        // a state from the workspace: only where an earlier chunk can have left one
        if (sss::began_before(cu[s], c0)) need(chunk > 0, "entering state of the first chunk", cu, tokens, K, c0);
        else if (end > tend) need(chunk < chunks - 1, "kept state of the last chunk", cu, tokens, K, c0);
        const int e = min(end, tend);
        need(t >= 0 && t < e && e <= tokens, "rows of pass 2", cu, tokens, K, c0);
        t = e;
      }
    }
  }
}

int main() {
  const int big = 0x7FFFFFFF;
  std::mt19937 rng(1);
  for (int a = -3; a <= 12; ++a)
    for (int b = -3; b <= 12; ++b)
      for (int c = -3; c <= 12; ++c)
        for (int K : {3, 8, 16}) check({a, b, c}, 10, K);
  for (int i = 0; i < 40000; ++i) {
    const int nseq = 1 + (int)(rng() % 6), tokens = 1 + (int)(rng() % 60);
    std::vector<int> cu;
    for (int s = 0; s <= nseq; ++s) {
      const unsigned kind = rng() % 8;
      cu.push_back(kind == 0 ? -big - 1 : kind == 1 ? big : (int)(rng() % 80) - 10);
    }
    if (i & 1) std::sort(cu.begin(), cu.end());
    check(cu, tokens, 1 + (int)(rng() % 20));
  }
  std::printf("ok\n");
}
