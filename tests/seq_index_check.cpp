// Holds every index of csrc/seq_index.hpp against its buffer, on the host.
// Prints what is wrong and ends with 1, or with 0.
#include "../linear_recurrence_amd/csrc/seq_index.hpp"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

using namespace rssm;

static void fail(const char* what, long a, long b, long c) {
  std::printf("%s: %ld %ld %ld\n", what, a, b, c);
  std::exit(1);
}

// A good table: every token in one segment, every empty sequence met once, chunk
// and segment places distinct and inside the workspace.
static void check_good(const std::vector<int32_t>& cu, int seg) {
  const int n = (int)cu.size() - 1, tokens = cu.back();
  const long slots = scan_slots(tokens, n, seg), cslots = scan_slots(tokens, n, kQ);
  std::vector<int> seen(tokens, 0), empty(n, 0), place(cslots, 0), ends(n, 0), begins(n, 0);
  for (long slot = 0; slot < slots; ++slot) {
    const Segment s = find_segment(cu.data(), n, tokens, seg, (int)slot);
    if (s.bad) fail("a good table is called bad", slot, s.seq, seg);
    if (s.seq < 0 || s.seq >= n) fail("sequence out of range", slot, s.seq, seg);
    if (s.empty) ++empty[s.seq];
    if (s.empty && s.len) fail("empty and not", slot, s.seq, s.len);
    if (!s.len) continue;
    if (s.len < 1 || s.len > seg) fail("length", slot, s.len, seg);
    if (s.tok < cu[s.seq] || s.tok + s.len > cu[s.seq + 1]) fail("tokens of another sequence", slot, s.tok, s.len);
    for (int t = s.tok; t < s.tok + s.len; ++t) ++seen[t];
    begins[s.seq] += s.first;
    ends[s.seq] += s.last;
    if (s.first != (s.tok == cu[s.seq]) || s.last != (s.tok + s.len == cu[s.seq + 1]))
      fail("first or last", slot, s.tok, s.len);
    // the combining launches find the segment from the sequence
    if (seg_base(cu.data(), s.seq, seg, tokens) + s.k != slot) fail("place of a segment", slot, s.seq, s.k);
    if (seg % kQ == 0) {
      const long base = seg_base(cu.data(), s.seq, kQ, tokens) + (long)s.k * (seg / kQ);
      for (int c = 0; c < (s.len + kQ - 1) / kQ; ++c) {
        if (base + c < 0 || base + c >= cslots) fail("place of a chunk", slot, base + c, cslots);
        if (place[base + c]++) fail("place taken twice", slot, base + c, seg);
        // the launches that take one chunk each find it there
        const Segment q = find_segment(cu.data(), n, tokens, kQ, (int)(base + c));
        if (q.seq != s.seq || q.tok != s.tok + c * kQ) fail("another chunk there", slot, base + c, q.tok);
      }
    }
  }
  for (int t = 0; t < tokens; ++t)
    if (seen[t] != 1) fail("token met other than once", t, seen[t], seg);
  for (int i = 0; i < n; ++i) {
    const int len = cu[i + 1] - cu[i];
    if (empty[i] != (len == 0) || begins[i] != (len > 0) || ends[i] != (len > 0))
      fail("sequence met other than once", i, empty[i], begins[i]);
  }
  for (int t = 0; t < tokens; ++t) {
    const int i = seq_of_token(cu.data(), n, t);
    if (t < cu[i] || t >= cu[i + 1]) fail("sequence of a token", t, i, seg);
  }
}

// Any table at all: nothing outside the tokens, the sequences or the workspace.
static void check_any(const std::vector<int32_t>& cu, int tokens, int seg) {
  const int n = (int)cu.size() - 1;
  const long slots = scan_slots(tokens, n, seg), cslots = scan_slots(tokens, n, kQ);
  for (long slot = 0; slot < slots; ++slot) {
    const Segment s = find_segment(cu.data(), n, tokens, seg, (int)slot);
    if (s.seq < 0 || s.seq >= n) fail("bad table: sequence", slot, s.seq, seg);
    if (s.len < 0 || s.len > seg || s.tok < 0 || (long)s.tok + s.len > tokens)
      fail("bad table: tokens", slot, s.tok, s.len);
    if (!s.len) continue;
    const long base = seg_base(cu.data(), s.seq, kQ, tokens) + (long)s.k * (seg / kQ);
    if (base < 0 || base + (s.len + kQ - 1) / kQ > cslots) fail("bad table: chunk", slot, base, cslots);
  }
  for (int i = 0; i < n; ++i) {
    const SeqSpan sp = seq_span(cu.data(), i, n, tokens);
    if (sp.start < 0 || sp.len < 0 || (long)sp.start + sp.len > tokens) fail("bad table: span", i, sp.start, sp.len);
    const long segs = ((long)sp.len + seg - 1) / seg, base = seg_base(cu.data(), i, seg, tokens);
    if (segs > 0 && (base < 0 || base + segs > slots)) fail("bad table: segments", i, base, segs);
  }
  for (int t = 0; t < tokens; t += 7) {
    const int i = seq_of_token(cu.data(), n, t);
    if (i < 0 || i >= n) fail("bad table: sequence of a token", t, i, n);
  }
}

// The elements that the 64 lanes of a column fragment take from an LDS tile of
// rows x ld: 32 rows from k0, 16 columns, each once, inside the tile.
template <int BYTES, bool PAIRED>
static void check_cols(int rows, int ld, int width, int k0, int c0) {
  std::set<long> got;
  for (int lane = 0; lane < 64; ++lane) {
    const long at = cols_offset<BYTES, PAIRED>(ld, k0, c0, lane);
    for (int e = 0; e < 8; ++e) {
      const long el = BYTES == 2 ? at + (e < 4 ? 0 : 16 * ld) + (e & 3) : at + (long)(e < 4 ? e : 12 + e) * ld;
      if (el < 0 || el >= (long)rows * ld || el % ld >= width) fail("tile", lane, el, ld);
      if (!got.insert(el).second) fail("element taken twice", lane, el, ld);
      const long r = el / ld;
      if (r < k0 || r >= k0 + 32) fail("row", lane, r, k0);
    }
  }
  for (int i = 0; i < 16; ++i) {
    const int col = PAIRED ? c0 + 8 * (i >> 2) + (i & 3) : c0 + i;
    for (int r = k0; r < k0 + 32; ++r)
      if (!got.count((long)r * ld + col)) fail("element not taken", r, col, ld);
  }
}

template <int BYTES>
static void check_tiles() {
  const int pad = BYTES == 2 ? 8 : 4;
  for (int n : {16, 32, 64, 128, 256}) {
    const int np = n < 32 ? 32 : n, ln = np + pad;
    for (int pb : {32, 64}) {
      const int lx = pb + pad, lm = kQ + pad;
      for (int s = 0; s < pb / 32; ++s)
        for (int p = 0; p < 2; ++p) {
          for (int kb = 0; kb < kQ / 32; ++kb)        // x, dy: tokens x state rows
            check_cols<BYTES, true>(kQ, lx, pb, 32 * kb, 32 * s + pair_base(p));
          for (int kb = 0; kb < np / 32; ++kb)        // dS: state columns x state rows
            check_cols<BYTES, true>(np, lx, pb, 32 * kb, 32 * s + pair_base(p));
        }
      for (int kb = 0; kb < kQ / 32; ++kb)
        for (int j = 0; j < 4; ++j) check_cols<BYTES, false>(kQ, lm, kQ, 32 * kb, 16 * j);  // K
    }
    for (int kb = 0; kb < kQ / 32; ++kb)
      for (int nt = 0; nt < n / 16; ++nt) check_cols<BYTES, false>(kQ, ln, np, 32 * kb, 16 * nt);  // B, C
  }
}

int main() {
  std::mt19937 rnd(1);
  const auto upto = [&](int n) { return (int)(rnd() % (unsigned)(n + 1)); };
  const int segs[] = {kQ, 3 * kQ, 4 * kQ, 5 * kQ, 11 * kQ, 64 * kQ};
  std::vector<std::vector<int>> lens = {{1}, {0}, {0, 0}, {3, 0, 1, 63, 64, 65, 0}, {64}, {128, 64}, {4096, 1, 4095},
                                        {0, 300, 0}, {257, 1, 0, 300}, {1, 1, 1, 1, 1, 1, 1, 1}};
  for (int k = 0; k < 400; ++k) {
    std::vector<int> l(1 + upto(30));
    const int most = 1 << upto(12);
    for (int& v : l) v = upto(4) == 0 ? 0 : upto(most);
    lens.push_back(l);
  }
  for (const auto& l : lens) {
    std::vector<int32_t> cu(1, 0);
    for (int v : l) cu.push_back(cu.back() + v);
    for (int seg : segs) check_good(cu, seg);
    for (int k = 0; k < 4; ++k) {                      // some entries spoilt
      std::vector<int32_t> bad = cu;
      for (int q = 0; q <= upto(3); ++q) {
        const int pick[] = {-1, INT32_MIN, INT32_MAX, cu.back() + 1, upto(cu.back() + 1)};
        bad[upto((int)bad.size() - 1)] = pick[upto(4)];
      }
      for (int seg : segs) check_any(bad, cu.back(), seg);
    }
  }
  for (int seg : segs) {                               // sizes near the largest
    const int big = INT32_MAX;
    const std::vector<int32_t> cu = {0, 5, big - 3, big};
    for (long slot : {0L, 1L, (long)big / seg, (long)big / seg + 2}) {
      const Segment s = find_segment(cu.data(), 3, big, seg, (int)slot);
      if (s.len < 0 || s.len > seg || (s.len && (s.tok < 0 || s.tok > big - s.len))) fail("large", slot, s.tok, s.len);
    }
  }
  for (int tile = 0; tile < 4; ++tile)
    for (int i = 0; i < 16; ++i)
      if (tile_col(tile, i) / 32 != tile / 2 || (tile_col(tile, i) / 4) % 2 != tile % 2) fail("tile_col", tile, i, 0);
  check_tiles<2>();
  check_tiles<4>();
  std::puts("ok");
  return 0;
}
