// Index arithmetic of the sequence operators: which tokens, slots and elements a
// workgroup and a lane work on.  Plain integer functions, compiled for the host
// too, where every index they give can be held against its buffer.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define RSSM_HD __host__ __device__
#else
#define RSSM_HD
#endif

namespace rssm {

constexpr int kQ = 64;   // tokens of a chunk
constexpr int kPT = 32;  // state rows of a wave

// Bounds of sequence i in a packed batch, forced into [0, tokens] so that a
// malformed table can only give wrong values, never a wrong address.
struct SeqSpan {
  int start, len;
  bool bad;
};
RSSM_HD static inline SeqSpan seq_span(const int32_t* cu, int i, int nseq, int tokens) {
  if (!cu) return {0, tokens, false};
  const int a = cu[i], b = cu[i + 1];
  const bool bad = a < 0 || b < a || b > tokens || (i == 0 && a != 0) ||
                   (i == nseq - 1 && b != tokens);
  const int s = a < 0 ? 0 : (a > tokens ? tokens : a);
  const int e = b < s ? s : (b > tokens ? tokens : b);
  return {s, e - s, bad};
}

// The last sequence whose start is at or before token t (binary search over
// the nseq starts; the table is monotone, or the result is merely arbitrary).
RSSM_HD static inline int seq_of_token(const int32_t* cu, int nseq, int t) {
  if (!cu) return 0;
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cu[m] <= t) lo = m; else hi = m;
  }
  return lo;
}

// Segments: runs of seg tokens (a multiple of kQ) of one sequence, worked on
// independently.  Segment k of sequence i has the slot start_i/seg + i + k:
// distinct for all, because a sequence of n tokens spans at least n/seg
// (rounded up) less one multiples of seg.  At most tokens/seg + seqs slots,
// so the host needs no lengths.
struct Segment {
  int seq, k, tok, len;  // len 0: nothing here, unless `empty`
  bool first, last, empty, bad;
};
RSSM_HD static inline int seg_base(const int32_t* cu, int i, int seg, int tokens) {
  if (!cu) return 0;
  const int a = cu[i];
  return (a < 0 ? 0 : (a > tokens ? tokens : a)) / seg + i;
}
// Segment k of sequence i.
RSSM_HD static inline Segment segment_of(const int32_t* cu, int i, int nseq, int tokens, int seg, int k) {
  const SeqSpan sp = seq_span(cu, i, nseq, tokens);
  Segment r;
  r.seq = i;
  r.bad = sp.bad;
  r.k = k;
  const long off = (long)r.k * seg;
  r.empty = sp.len == 0 && r.k == 0;
  r.len = r.k < 0 || off >= sp.len ? 0 : (sp.len - off < seg ? (int)(sp.len - off) : seg);
  r.tok = sp.start + (r.len ? (int)off : 0);
  r.first = r.k == 0;
  r.last = off + seg >= sp.len;
  return r;
}
RSSM_HD static inline Segment find_segment(const int32_t* cu, int nseq, int tokens, int seg,
                                              int slot) {
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (seg_base(cu, m, seg, tokens) <= slot) lo = m; else hi = m;
  }
  return segment_of(cu, lo, nseq, tokens, seg, slot - seg_base(cu, lo, seg, tokens));
}

// Slots that the segments of a call may take.
RSSM_HD static inline long scan_slots(long tokens, long seqs, long seg) { return tokens / seg + seqs; }

// Places of the segments of sequences longer than one, where each keeps whole states:
// short sequences, however many, add none.  Sequence i's begin at start_i/seg + i as
// above while there are few sequences, and otherwise at 2 start_i/seg: n tokens, n > seg,
// have n/seg (rounded up) segments, and 2 n/seg (rounded down) are at least as many.
// At most 4 tokens/seg places.  (13 sequences of 16383 tokens, segments of 2048: the first
// way 20 places, the second 15, whose search takes the combining launch 20 us for 8.)
RSSM_HD static inline bool long_few(long tokens, long seqs, long seg) { return seqs <= 3 * (tokens / seg); }
RSSM_HD static inline long long_places(long tokens, long seqs, long seg) {
  return long_few(tokens, seqs, seg) ? tokens / seg + seqs : 2 * tokens / seg;
}
RSSM_HD static inline int long_base(const int32_t* cu, int i, int seg, int tokens, bool few) {
  if (few || !cu) return seg_base(cu, i, seg, tokens);
  const int a = cu[i];
  return (int)(2L * (a < 0 ? 0 : (a > tokens ? tokens : a)) / seg);
}
// The segment of a place: the last sequence that begins at it or before (later ones
// begin behind a long one's places).  Sequences of one segment are `first` and `last`.
RSSM_HD static inline Segment find_long(const int32_t* cu, int nseq, int tokens, int seg, bool few, int place) {
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (long_base(cu, m, seg, tokens, few) <= place) lo = m; else hi = m;
  }
  return segment_of(cu, lo, nseq, tokens, seg, place - long_base(cu, lo, seg, tokens, few));
}

// Columns of the two tiles of a pair (32 columns) interleave in granules of 4,
// tile j's index i standing for column 8*(i/4) + 4*j + i%4: a lane that holds
// rows 4g..4g+3 of both tiles' results then holds 8 neighbours (16 bytes of
// bf16), as global loads and stores want them.
RSSM_HD static inline int pair_base(int tile) { return 32 * (tile >> 1) + 4 * (tile & 1); }
RSSM_HD static inline int tile_col(int tile, int i) {
  return pair_base(tile) + 8 * (i >> 2) + (i & 3);
}

// A lane's place in a column fragment, in elements from the tile's start: K block
// starting at row k0, the 16 columns of a tile that start at c0 and, in a `paired`
// operand, come in granules of 4 every 8 columns (see tile_col).  Two-byte
// elements: row 4g + i/4 of the block, the granule that a transposing read takes;
// it takes row 16 + 4g + i/4 too.  Four bytes: the lane's column in row 4g, and the
// seven rows to 19 + 4g of order D.
template <int BYTES, bool PAIRED>
RSSM_HD static inline int cols_offset(int ld, int k0, int c0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  return BYTES == 2 ? (k0 + 4 * g + (i >> 2)) * ld + c0 + (i & 3) * (PAIRED ? 8 : 4)
                    : (k0 + 4 * g) * ld + c0 + (PAIRED ? 8 * (i >> 2) + (i & 3) : i);
}

}  // namespace rssm
