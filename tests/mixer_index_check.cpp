// Holds the places of segments that keep whole states against their buffer, on the
// host.  Prints what is wrong and ends with 1, or with 0.
#include "../linear_recurrence_amd/csrc/seq_index.hpp"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using namespace rssm;

static void fail(const char* what, long a, long b, long c) {
  std::printf("%s: %ld %ld %ld\n", what, a, b, c);
  std::exit(1);
}

// A good table: every segment of a longer sequence has a place of its own, found from the
// sequence and from the place.
static void check_good(const std::vector<int32_t>& cu, int seg) {
  const int n = (int)cu.size() - 1, tokens = cu.back();
  const long places = long_places(tokens, n, seg);
  const bool few = long_few(tokens, n, seg);
  if (places > scan_slots(tokens, n, seg) || places > 4L * tokens / seg) fail("more places than needed", places, n, tokens);
  std::vector<int> taken(places, -1);
  for (int i = 0; i < n; ++i) {
    const int len = cu[i + 1] - cu[i];
    if (len <= seg) continue;
    for (int k = 0; k < (len + seg - 1) / seg; ++k) {
      const long p = (long)long_base(cu.data(), i, seg, tokens, few) + k;
      if (p < 0 || p >= places) fail("outside", p, places, i);
      if (taken[p] >= 0) fail("taken twice", p, taken[p], i);
      taken[p] = i;
      const Segment s = find_long(cu.data(), n, tokens, seg, few, (int)p);
      if (s.bad || s.seq != i || s.k != k || s.tok != cu[i] + k * seg) fail("another segment there", p, s.seq, s.k);
    }
  }
  for (long p = 0; p < places; ++p) {  // and nothing but short sequences at the others
    if (taken[p] >= 0) continue;
    const Segment s = find_long(cu.data(), n, tokens, seg, few, (int)p);
    if (s.len && !(s.first && s.last)) fail("a segment at no place of its own", p, s.seq, s.k);
  }
}

// Any table at all: what may be written or read lies inside.
static void check_any(const std::vector<int32_t>& cu, int tokens, int seg) {
  const int n = (int)cu.size() - 1;
  const long places = long_places(tokens, n, seg);
  const bool few = long_few(tokens, n, seg);
  for (int i = 0; i < n; ++i) {
    const SeqSpan sp = seq_span(cu.data(), i, n, tokens);
    const long segs = ((long)sp.len + seg - 1) / seg, base = long_base(cu.data(), i, seg, tokens, few);
    if (segs > 1 && (base < 0 || base + segs > places)) fail("bad table: places", i, base, segs);
  }
  for (long p = 0; p < places; ++p) {
    const Segment s = find_long(cu.data(), n, tokens, seg, few, (int)p);
    if (s.seq < 0 || s.seq >= n || s.len < 0 || s.len > seg || s.tok < 0 || (long)s.tok + s.len > tokens)
      fail("bad table: segment", p, s.seq, s.len);
  }
}

int main() {
  std::mt19937 rnd(1);
  const auto upto = [&](int n) { return (int)(rnd() % (unsigned)(n + 1)); };
  const int segs[] = {8 * kQ, 9 * kQ, 13 * kQ, 64 * kQ};
  std::vector<std::vector<int>> lens = {{513}, {512, 513}, {1, 1, 1, 1, 513, 1, 1, 0, 0, 1025}, {768, 767, 0, 769},
                                        {0, 0, 0, 0, 0, 0, 600, 0, 0, 0, 600}, {4096, 1, 4095, 1, 1, 1}};
  for (int k = 0; k < 600; ++k) {
    std::vector<int> l(1 + upto(k % 3 ? 40 : 3));
    const int most = 512 << upto(4);
    for (int& v : l) v = upto(3) == 0 ? upto(most) : upto(3) ? upto(20) : 0;
    lens.push_back(l);
  }
  for (const auto& l : lens) {
    std::vector<int32_t> cu(1, 0);
    for (int v : l) cu.push_back(cu.back() + v);
    for (int seg : segs) {
      if (cu.back() <= seg) continue;  // no call has segments then
      check_good(cu, seg);
      for (int k = 0; k < 4; ++k) {
        std::vector<int32_t> bad = cu;
        for (int q = 0; q <= upto(3); ++q) {
          const int pick[] = {-1, INT32_MIN, INT32_MAX, cu.back() + 1, upto(cu.back() + 1)};
          bad[upto((int)bad.size() - 1)] = pick[upto(4)];
        }
        check_any(bad, cu.back(), seg);
      }
    }
  }
  const int big = INT32_MAX;  // sizes near the largest
  std::vector<int32_t> cu = {0, 5, big - 5000, big};
  check_any(cu, big, 64 * kQ);
  cu.assign(1 << 20, 0);
  cu.push_back(big - 4097);
  cu.push_back(big);
  check_any(cu, big, 64 * kQ);
  std::puts("ok");
  return 0;
}
