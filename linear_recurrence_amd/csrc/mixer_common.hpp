// Shared pieces of linear attention and the gated delta rule over sequences.
//
// Per value head, with S [K, V] (the pools hold its transpose), g the decay's
// logarithm, DELTA the gated delta rule:
//   S <- e^{g_t} S;  d_t = beta_t (v_t - S^T k_t)  (linear attention: d_t = v_t)
//   S <- S + k_t d_t^T;  o_t = scale S^T q_t
// Tokens of a sequence are taken in chunks of 64.  With G the running sum of g in
// the chunk (inclusive), c_ij = e^{G_i - G_j} and S the state before the chunk,
//   A_ij = beta_i c_ij k_i.k_j  (i > j),  T = (I + A)^-1
//   D = T X,  X_i = beta_i (v_i - e^{G_i} S^T k_i)
//   o_i = scale [ e^{G_i} S^T q_i + sum_{j<=i} c_ij (q_i.k_j) d_j ]
//   S' = e^{G_Q} S + sum_j e^{G_Q - G_j} k_j d_j^T
// so all the work is small dense products for the matrix cores (fragments and
// their orders C and D: scan_common.hpp).
//
// A wave owns 16 columns of S as eight (K = 128) or four accumulators, rows in
// 4g + r: they are the second operand of K S and Q S as they stand, K S's result is
// that of T X, and its result that of K^T D, so nothing moves between lanes.
#pragma once

#include "scan_common.hpp"

namespace rssm {

struct MixArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;      // [v_heads] or [tokens, v_heads] by decay
  const float* beta;   // [tokens, v_heads]
  const int32_t* cu;
  const float* init;
  const uint8_t* has_init;
  const int32_t* slot_idx;
  float* final_state;
  void* o;
  void* tinv;          // [chunk slots][v_heads][6 (12) fragments][terms][64]
  int32_t* status;
  float* seg_state;    // [places][v_heads][V][K] (long_base: seq_index.hpp)
  float* seg_grad;     // the same
  float* seg_decay;    // [places][v_heads]
  const int32_t* order;  // [segment slots]: the longest first, or null
  void* trans;         // [places][v_heads][K K / 512 (twice) fragments][terms][64]
  long q_stride, k_stride, v_stride;
  int32_t tokens, seqs, k_heads, v_heads, vpk, dv, num_slots, decay;
  int32_t seg, slots, few;  // tokens of a segment, segment slots, long_few
  float scale;
};

__device__ static inline int mix_slot(const MixArgs& a, int i) {
  const int s = a.slot_idx ? a.slot_idx[i] : i;
  return s >= 0 && s < a.num_slots ? s : -1;
}

// (-1, 0) and (0, -1) as pairs of bf16, in registers that the compiler knows nothing
// about: as constants of a two-product instruction they come out as other values.
struct Minus {
  uint32_t lo = 0x0000bf80u, hi = 0xbf800000u;
  __device__ inline Minus() { asm volatile("" : "+v"(lo), "+v"(hi)); }
};

// Split::set with half the instructions for what a term leaves: x - bf16(x) is exact, and
// one two-product with (-1, 0) forms it from the packed pair (0 times an infinity next to
// it is NaN: the eight values are factors of the same sums).  The terms were most of the
// vector unit's work, which stands beside the products'.
template <typename T, int TERMS>
__device__ static inline Split<T, TERMS> split(const float* f, const Minus& m) {
  Split<T, TERMS> s;
  if constexpr (TERMS == 1) {
    s.t[0] = Mat<T>::pack(f);
  } else {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      s.t[k] = Mat<T>::pack(r);
      if (k + 1 == TERMS) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t pair = s.t[k][q];
        const bf16x2_t h = __builtin_bit_cast(bf16x2_t, pair);
        r[2 * q] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2_t, m.lo), r[2 * q], false);
        r[2 * q + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2_t, m.hi), r[2 * q + 1], false);
      }
    }
  }
  return s;
}

// The 64x64 lower triangle as fragments of 16 rows and 32 columns: six are not zero.
RSSM_HD static inline int low_frag(int it, int kb) { return it < 2 ? it : 2 * it - 2 + kb; }
// The upper triangle's (a lower one's transpose).
RSSM_HD static inline int up_frag(int it, int kb) { return low_frag(3 - it, 1 - kb); }

// N results at once of a split operand (a fragment for each: load(n, term)) and another
// that they share: every pair of terms whose weight fp32 can hold.  Neighbouring
// products do not wait for each other, as a result's own terms would.  SWAP: the shared
// one is the first operand.
template <typename T, int TA, int TB, int N, bool SWAP = false, typename Load>
__device__ static inline void mma_many(const Load& load, const Split<T, TB>& y, f32x4* acc) {
  constexpr int M = TA > TB ? TA : TB;
#pragma unroll
  for (int i = TA - 1; i >= 0; --i) {
    typename Mat<T>::Frag x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = load(n, i);
#pragma unroll
    for (int j = TB - 1; j >= 0; --j) {
      if (i + j >= M) continue;
#pragma unroll
      for (int n = 0; n < N; ++n)
        acc[n] = SWAP ? Mat<T>::mma(y.t[j], x[n], acc[n]) : Mat<T>::mma(x[n], y.t[j], acc[n]);
    }
  }
}
template <typename T, int TA, int TB>
__device__ static inline f32x4 mma_split(const Split<T, TA>& x, const Split<T, TB>& y, f32x4 c) {
  mma_many<T, TA, TB, 1>([&](int, int i) { return x.t[i]; }, y, &c);
  return c;
}

// A decay exponent in log2.  -1e4 already takes any state to zero, and keeps sums of 64
// and their differences finite; NaN passes.
__device__ static inline double gate_log2(float g) {
  return (double)(g < -1e4f ? -1e4f : g) * 1.4426950408889634074;
}
// log g and beta of the chunk's tokens, one a lane, on their way from memory.  Loads
// without conditions (a lane without a token takes the first one's, and drops it): in
// branches, each would be waited for before the next is issued.
struct GateLoad {
  const float *g, *b;  // of the chunk's first token
  long step_g;         // floats between two tokens' log g
  int heads;
  float rg, rb;
  bool have_g, have_b;
  __device__ inline void start(const MixArgs& a, long t0, int hv, bool delta) {
    heads = a.v_heads;
    step_g = a.decay == RSSM_DECAY_TOKEN ? heads : 0;
    have_g = a.decay != RSSM_DECAY_NONE;
    have_b = delta;
    g = have_g ? a.g + hv + t0 * step_g : reinterpret_cast<const float*>(a.k);
    b = delta ? a.beta + t0 * heads + hv : g;
  }
  __device__ inline void step(int chunks) {
    g += chunks * kQ * step_g;
    if (have_b) b += (long)chunks * kQ * heads;
  }
  __device__ inline void fetch(int rows, int lane) {
    const long t = lane < rows ? lane : 0;
    rg = g[t * step_g];
    rb = have_b ? b[t * heads] : 0.f;
  }
  __device__ inline float log_g(int rows, int lane) const { return have_g && lane < rows ? rg : 0.f; }
  __device__ inline float beta(int rows, int lane) const { return lane < rows ? rb : 0.f; }
};

// Inclusive sum over the wave's lanes in double, by lane shifts within the vector unit:
// it stands on every chunk's path, and through LDS it took six round trips.
template <int CTRL, int ROWS>
__device__ static inline double dpp_moved(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ static inline double lane_sums(double v) {
  v += dpp_moved<0x111, 0xF>(v);  // from 1, 2, 4 and 8 lanes below in the row of 16
  v += dpp_moved<0x112, 0xF>(v);
  v += dpp_moved<0x114, 0xF>(v);
  v += dpp_moved<0x118, 0xF>(v);
  v += dpp_moved<0x142, 0xA>(v);  // a row's last lane to the next row
  v += dpp_moved<0x143, 0xC>(v);  // lane 31 to the upper half
  return v;
}
__device__ static inline double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// fp32 lane shifts within rows of 16, for sums over the 16 lanes of a group.
template <int CTRL>
__device__ static inline float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// Every lane gets its group's sum.
__device__ static inline float row16_sum(float v) {
  v += dpp_f32<0x128>(v);  // 8 lanes round
  v += dpp_f32<0x141>(v);  // mirrored in halves
  v += dpp_f32<0x4E>(v);   // the other pair of a quad
  v += dpp_f32<0xB1>(v);   // the other lane of a pair
  return v;
}
// The sum over the four groups of 16 lanes, in every lane.
__device__ static inline float groups_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// Sixteen sums over a group at once: lane l%16 gets item l%16's.  At each level a lane keeps half
// of its items and takes the partner's sums of them: 15 shifts instead of 64.
template <int LEVEL>
__device__ static inline void row16_sums(float (&v)[16], int lane) {
  if constexpr (LEVEL < 4) {
    constexpr int bit = 8 >> LEVEL, half = 8 >> LEVEL;
    constexpr int ctrl = LEVEL == 0 ? 0x128 : (LEVEL == 1 ? 0x141 : (LEVEL == 2 ? 0x4E : 0xB1));
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float send = up ? v[j] : v[j + half], keep = up ? v[j + half] : v[j];
      v[j] = keep + dpp_f32<ctrl>(send);
    }
    row16_sums<LEVEL + 1>(v, lane);
  }
}

// A chunk's decays, one token a lane, as the kernels read them from LDS.
struct ChunkGates {
  float2 G[kQ];                                      // log2 of the decay since the chunk began
  __attribute__((aligned(16))) float eg[kQ];         // e^{G_t}
  __attribute__((aligned(16))) float et[kQ];         // e^{G_Q - G_t}
  __attribute__((aligned(16))) float beta[kQ];
  float all;                                         // e^{G_Q}
  __device__ inline void set(float log_g, float b, int lane) {
    const double cum = lane_sums(gate_log2(log_g)), last = last_lane(cum);
    const float hi = (float)cum;
    G[lane] = make_float2(hi, (float)(cum - (double)hi));
    eg[lane] = exp2_f32(hi);
    et[lane] = exp2_f32((float)(last - cum));
    beta[lane] = b;
    if (lane == 0) all = exp2_f32((float)last);
  }
};

// Row i of a state's 16-row tile kt: two tiles share 32 rows in turns of four, so that a
// lane's rows 4g + r of both are eight neighbours, which fragments of K and Q in order C
// hold too: one 16-byte read each.  (In order D, two reads of 8 bytes, the compiler paired
// reads of different fragments and moved their halves together again.)
RSSM_HD static inline int mix_row(int kt, int i) { return 32 * (kt >> 1) + 8 * (i >> 2) + 4 * (kt & 1) + (i & 3); }

// A tile of 64 tokens' rows in LDS.  bf16: 16-byte pieces of a row change places by the
// row, so that the 16 rows of a fragment, and the four rows that 16 lanes of a
// transposing read take, lie in different banks without padding.  fp32: padded rows.
template <typename T, int COLS>
struct Tile {
  typedef typename Mat<T>::E E;
  typedef typename Mat<T>::Frag Frag;
  static constexpr bool kSwap = sizeof(E) == 2;
  static constexpr int LD = kSwap ? COLS : COLS + Mat<T>::kPad, SIZE = kQ * LD;
  __device__ static inline int place(int row) {
    return COLS == 64 ? ((row >> 1 & 1) << 2) | (row >> 2 & 3) : ((row & 3) << 2) | (row >> 2 & 3);
  }
  __device__ static inline int at(int row, int col) {
    return kSwap ? row * LD + (((col >> 3) ^ place(row)) << 3) + (col & 7) : row * LD + col;
  }
  // fragments of rows 16 it + l%16, 32 columns from c, in order C and in order D
  __device__ static inline Frag rows_c(const E* p, int it, int c, int lane) {
    return Mat<T>::rows_c(p + at(16 * it + (lane & 15), c + 8 * (lane >> 4)));
  }
  __device__ static inline Frag rows_d(const E* p, int it, int c, int lane) {
    const int row = 16 * it + (lane & 15), col = c + 4 * (lane >> 4);
    if constexpr (kSwap) {
      const u32x2 a = *reinterpret_cast<const u32x2*>(p + at(row, col));
      const u32x2 b = *reinterpret_cast<const u32x2*>(p + at(row, col + 16));
      return Frag{a[0], a[1], b[0], b[1]};
    } else {
      return Mat<T>::rows_d(p + at(row, col));
    }
  }
  // of 32 rows from k0, the columns of a state's tile kt (see mix_row)
  __device__ static inline Frag cols_of(const E* p, int k0, int kt, int lane) {
    const int i = lane & 15, g = lane >> 4, c = 32 * (kt >> 1) + 4 * (kt & 1);
    if constexpr (kSwap) return Mat<T>::cols(p + at(k0 + 4 * g + (i >> 2), c + 8 * (i & 3)), LD);
    else return Mat<T>::cols(p + at(k0 + 4 * g, c + 8 * (i >> 2) + (i & 3)), LD);
  }
  // of 32 rows from k0, columns c .. c + 15
  __device__ static inline Frag cols(const E* p, int k0, int c, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (kSwap) return Mat<T>::cols(p + at(k0 + 4 * g + (i >> 2), c + 4 * (i & 3)), LD);
    else return Mat<T>::cols(p + at(k0 + 4 * g, c + i), LD);
  }
};

// Such a tile on its way from memory, chunk after chunk: a thread keeps one address,
// from which its pieces are whole rows (multiples of 16) apart.  Loads without
// conditions, so that all are issued at once: a piece behind the last row takes the first
// one's, and is put as zero.
template <typename T, int COLS, int THREADS>
struct TileLoad {
  typedef typename Mat<T>::E E;
  static constexpr int V = 16 / sizeof(E), PER = COLS / V, N = kQ * PER / THREADS, R = THREADS / PER;
  static_assert(kQ * PER % THREADS == 0 && THREADS % PER == 0, "whole rounds");
  static_assert(sizeof(E) == 4 || R % 16 == 0, "a thread's pieces keep their place");
  const E *p, *p0;  // of this thread's first row, and of the chunk's
  long stride;
  u32x4 r[N];
  __device__ inline void start(const E* src, long s, int tid) {
    stride = s;
    p0 = src;
    p = src + (tid / PER) * s + (tid % PER) * V;
  }
  __device__ inline void step(int chunks) {
    p += chunks * kQ * stride;
    p0 += chunks * kQ * stride;
  }
  __device__ inline void fetch(int rows, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      r[i] = *reinterpret_cast<const u32x4*>(tid / PER + i * R < rows ? p + i * (R * stride) : p0);
  }
  __device__ inline void put(E* tile, int rows, int tid) {
    if (rows < kQ) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (tid / PER + i * R >= rows) r[i] = u32x4{0, 0, 0, 0};
    }
    E* const to = tile + Tile<T, COLS>::at(tid / PER, (tid % PER) * V);
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(to + i * R * Tile<T, COLS>::LD) = r[i];
  }
};

// The fragments of T in the same way; the last piece may be taken twice.
template <int PIECES, int THREADS>
struct FragLoad {
  static constexpr int N = (PIECES + THREADS - 1) / THREADS;
  const u32x4* p;
  u32x4 r[N];
  __device__ static inline int at(int i, int tid) {
    return PIECES % THREADS == 0 || i * THREADS + tid < PIECES ? i * THREADS + tid : PIECES - 1;
  }
  __device__ inline void fetch(int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = p[at(i, tid)];
  }
  __device__ inline void put(u32x4* to, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) to[at(i, tid)] = r[i];
  }
};

// Fragments kept in memory or LDS as lanes hold them.
template <typename T>
__device__ static inline typename Mat<T>::Frag frag_at(const void* base, int i, int lane) {
  typename Mat<T>::Frag f;
  __builtin_memcpy(&f, __builtin_assume_aligned(static_cast<const char*>(base) + (i * 64 + lane) * sizeof(f), 16),
                   sizeof(f));
  return f;
}
template <typename T, int TERMS>
__device__ static inline void put_split(void* base, int i, const Split<T, TERMS>& s, int lane) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k)
    __builtin_memcpy(__builtin_assume_aligned(static_cast<char*>(base) + ((i * TERMS + k) * 64 + lane) * sizeof(s.t[k]), 16),
                     &s.t[k], sizeof(s.t[k]));
}
template <typename T, int TERMS>
__device__ static inline Split<T, TERMS> split_at(const void* base, int i, int lane) {
  Split<T, TERMS> s;
#pragma unroll
  for (int k = 0; k < TERMS; ++k) s.t[k] = frag_at<T>(base, i * TERMS + k, lane);
  return s;
}

// Units (a segment's key head) are dealt to the eight dies in turn, so that a long
// sequence's heads are spread over them and a key head's workgroups share one L2.
struct MixUnit {
  int slot, hk, rest;
  bool live;
};
__device__ static inline MixUnit mix_unit(const MixArgs& a, int id, int per) {
  const int j = id >> 3, u = (j / per) * 8 + (id & 7);
  MixUnit m;
  m.live = u < a.slots * a.k_heads;
  m.slot = m.live ? u / a.k_heads : 0;
  if (m.live && a.order) m.slot = a.order[m.slot];
  m.hk = m.live ? u % a.k_heads : 0;
  m.rest = j % per;
  return m;
}
static inline long mix_grid(long slots, long k_heads, long per) { return (slots * k_heads + 7) / 8 * 8 * per; }

// 16x16x16 in fp32: operand registers hold four values of k = 4g + e.
__device__ static inline f32x4 mm16(f32x4 x, f32x4 y, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
  return c;
}

// T = (I + A)^-1 of one chunk and value head, a wave each, in fp32: the four 16x16
// diagonal blocks by substitution (a lane a column), the others from them in order,
//   T_ij = -T_ii sum_{j<=m<i} A_im T_mj,
// then split into the products' terms and stored as fragments (lower triangle; BOTH:
// and the transpose's, for the backward pass).  Each block of A is computed so that a
// lane holds its row's values: it is a first operand as it stands.  The substitutions'
// chains bound it: 2048 matrices (4096 tokens of 32 heads) take 22 us, and in front of a
// backward pass 4096 with their transposes 40 us, of it 150 MB written.
template <typename T, int K, bool BOTH>
static __global__ void __launch_bounds__(256) mix_inverse_kernel(const MixArgs a) {
  typedef Mat<T> M;
  typedef typename M::Frag Frag;
  typedef typename M::E E;
  constexpr int LB = 20, TERMS = M::kTerms, KB = K / 32;
  __shared__ __attribute__((aligned(16))) float sBlk[4][10][16 * LB];
  __shared__ float2 sG[4][kQ];
  __shared__ __attribute__((aligned(16))) float sBeta[4][kQ];
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = (a.v_heads + 3) / 4;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / per, hv = (id % per) * 4 + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, kQ, slot);
  if (sg.len == 0 || hv >= a.v_heads) return;
  const int rows = sg.len, hk = hv / a.vpk;
  const long t0 = sg.tok;
  {
    GateLoad ld;
    ld.start(a, t0, hv, true);
    ld.fetch(rows, lane);
    const double cum = lane_sums(gate_log2(ld.log_g(rows, lane)));
    const float hi = (float)cum;
    sG[wave][lane] = make_float2(hi, (float)(cum - (double)hi));
    sBeta[wave][lane] = ld.beta(rows, lane);
  }
  // k_m.k_i: rows m of block bm, columns i of block bi <= bm is left out
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m <= i; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const E* const src = static_cast<const E*>(a.k) + t0 * a.k_stride + (long)hk * K;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    Frag f[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int t = 16 * b + i16;
      u32x4 z[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      if (t < rows) {
        const E* p = src + t * a.k_stride + 32 * kb + 8 * g;
        z[0] = *reinterpret_cast<const u32x4*>(p);
        if (sizeof(E) == 4) z[1] = *reinterpret_cast<const u32x4*>(p + 4);
      }
      __builtin_memcpy(&f[b], z, sizeof(Frag));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m <= i; ++m) acc[i][m] = M::mma(f[m], f[i], acc[i][m]);
  }
  wave_sync();
  // A_im in the lane of row i = i16, columns m = 4g + r
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 gi = sG[wave][16 * i + i16];
    const float bi = sBeta[wave][16 * i + i16];
#pragma unroll
    for (int m = 0; m <= i; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = bi * exp2_f32(gap2(gi, sG[wave][16 * m + 4 * g + r])) * acc[i][m][r];
        acc[i][m][r] = m < i || 4 * g + r < i16 ? w : 0.f;
      }
    *reinterpret_cast<f32x4*>(&sBlk[wave][i][i16 * LB + 4 * g]) = acc[i][i];
  }
  wave_sync();
  float x[16];
  {
    const float* blk = sBlk[wave][g];  // lane 16 b + c: column c of block b
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == i16 ? 1.f : 0.f;
#pragma unroll
      for (int m4 = 0; m4 < 16; m4 += 4) {
        if (m4 >= i) break;
        const f32x4 row = *reinterpret_cast<const f32x4*>(blk + i * LB + m4);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (m4 + m < i) s = fmaf(-row[m], x[m4 + m], s);
      }
      x[i] = s;
    }
  }
  wave_sync();
#pragma unroll
  for (int i = 0; i < 16; ++i) sBlk[wave][g][i * LB + i16] = x[i];
  wave_sync();
  f32x4 Ad[4], t[4][4];  // t[i][j]: rows 4g + r, column i16
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    Ad[b] = *reinterpret_cast<const f32x4*>(&sBlk[wave][b][i16 * LB + 4 * g]);
#pragma unroll
    for (int r = 0; r < 4; ++r) t[b][b][r] = sBlk[wave][b][(4 * g + r) * LB + i16];
  }
#pragma unroll
  for (int dist = 1; dist < 4; ++dist)
#pragma unroll
    for (int j = 0; j + dist < 4; ++j) {
      const int i = j + dist;
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = j; m < i; ++m) s = mm16(acc[i][m], t[m][j], s);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = -s[r];
      t[i][j] = mm16(Ad[i], s, f32x4{0.f, 0.f, 0.f, 0.f});
    }
  // off-diagonal blocks by rows
#pragma unroll
  for (int i = 1; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < i; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sBlk[wave][4 + i * (i - 1) / 2 + j][(4 * g + r) * LB + i16] = t[i][j][r];
  wave_sync();
  const Minus minus;
  char* const out = static_cast<char*>(a.tinv) +
      ((long)slot * a.v_heads + hv) * ((BOTH ? 12 : 6) * TERMS * 64 * sizeof(Frag));
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int kb = 0; kb <= it / 2; ++kb) {
      float f[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * kb + h;
        f32x4 row = {0.f, 0.f, 0.f, 0.f};
        if (j == it) row = Ad[it];
        if (j < it) row = *reinterpret_cast<const f32x4*>(&sBlk[wave][4 + it * (it - 1) / 2 + j][i16 * LB + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[4 * h + r] = row[r];
      }
      const auto s = split<T, TERMS>(f, minus);
      put_split<T, TERMS>(out, low_frag(it, kb), s, lane);
    }
  if (BOTH) {
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
#pragma unroll
      for (int kb = jt / 2; kb < 2; ++kb) {
        float f[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) f[4 * h + r] = 2 * kb + h >= jt ? t[2 * kb + h][jt][r] : 0.f;
        const auto s = split<T, TERMS>(f, minus);
        put_split<T, TERMS>(out, 6 + up_frag(jt, kb), s, lane);
      }
  }
}

static inline size_t mix_inverse_bytes(bool f32, bool both) {
  return (size_t)(both ? 12 : 6) * 64 * (f32 ? 32 : 3 * 16);
}

template <typename T, bool BOTH>
static inline int launch_inverse(const MixArgs& a, int dk, long cslots, hipStream_t stream) {
  const void* fn = dk == 64 ? reinterpret_cast<const void*>(&mix_inverse_kernel<T, 64, BOTH>)
                            : reinterpret_cast<const void*>(&mix_inverse_kernel<T, 128, BOTH>);
  return launch_kernel(fn, (unsigned)(cslots * ((a.v_heads + 3) / 4)), 256, 0, stream, a);
}

static inline int mix_check(const rssm_mixer_dims* d, bool delta) {
  if (!d) return RSSM_EINVAL;
  if (d->tokens < 0 || d->seqs < 0 || d->k_heads < 1 || d->v_heads < 1 || d->v_heads % d->k_heads ||
      d->num_slots < 0)
    return RSSM_EINVAL;
  if (!valid_dtype(d->io_dtype)) return RSSM_EDTYPE;
  if (d->decay < RSSM_DECAY_NONE || d->decay > RSSM_DECAY_TOKEN) return RSSM_EINVAL;
  if (!(d->dk == 64 || d->dk == 128) || !(d->dv == 64 || d->dv == 128)) return RSSM_ESHAPE;
  if (delta && d->dk != d->dv) return RSSM_ESHAPE;
  if (delta && d->decay != RSSM_DECAY_TOKEN) return RSSM_EINVAL;
  if (d->scale != d->scale) return RSSM_EINVAL;
  // heads in a row and in a pool slot are indexed in 32 bits
  if ((long)d->v_heads > (1L << 20)) return RSSM_ESHAPE;
  const long es = d->io_dtype == RSSM_F32 ? 4 : 2;
  const long qk = (long)d->k_heads * d->dk, v = (long)d->v_heads * d->dv;
  const int64_t rows[4] = {d->q_stride, d->k_stride, d->v_stride, d->do_stride};
  for (int i = 0; i < 4; ++i)
    if (rows[i] != 0 && (rows[i] < (i < 2 ? qk : v) || rows[i] * es % 16)) return RSSM_EINVAL;
  return RSSM_OK;
}

static inline void mix_fill(MixArgs& a, const rssm_mixer_dims& d) {
  a.q_stride = d.q_stride ? d.q_stride : (long)d.k_heads * d.dk;
  a.k_stride = d.k_stride ? d.k_stride : (long)d.k_heads * d.dk;
  a.v_stride = d.v_stride ? d.v_stride : (long)d.v_heads * d.dv;
  a.tokens = d.tokens;
  a.seqs = d.seqs;
  a.k_heads = d.k_heads;
  a.v_heads = d.v_heads;
  a.vpk = d.v_heads / d.k_heads;
  a.dv = d.dv;
  a.num_slots = d.num_slots;
  a.decay = d.decay;
  a.scale = d.scale > 0.f ? d.scale : 1.f / sqrtf((float)d.dk);
}

// Whether a dense result with these heads' rows shares memory with q, k or v, which other
// workgroups may still read when it is written.
static inline bool mix_meets(const MixArgs& a, const rssm_mixer_dims& d, const void* out, long columns) {
  const long es = d.io_dtype == RSSM_F32 ? 4 : 2, qk = (long)d.k_heads * d.dk * es, v = (long)d.v_heads * d.dv * es;
  const long bytes = d.tokens * columns * es;
  return rows_meet(a.q, a.q_stride * es, qk, d.tokens, out, bytes) ||
         rows_meet(a.k, a.k_stride * es, qk, d.tokens, out, bytes) ||
         rows_meet(a.v, a.v_stride * es, v, d.tokens, out, bytes);
}
// The same of o, which may be v itself: a head's columns of v are read by the workgroup
// that writes them, each chunk's before its outputs go there.
static inline bool output_meets(const MixArgs& a, const rssm_mixer_dims& d, const void* o) {
  const long v = (long)d.v_heads * d.dv;
  MixArgs other = a;
  if (o == a.v && a.v_stride == v) other.v = nullptr;
  return mix_meets(other, d, o, v);
}
// Whether two pools that are not one share memory: a slot's new state would be over another's.
static inline bool pools_meet(const rssm_mixer_dims& d, const float* in, const float* out) {
  const long bytes = (long)d.num_slots * d.v_heads * d.dv * d.dk * 4;
  return in != out && rows_meet(in, bytes, bytes, d.num_slots > 0, out, bytes);
}

// Tokens of a segment.  A sequence longer than this is worked on in segments: what each
// adds from zero and (the delta rule) the matrix that its start goes through, then
// their combination, then all segments at once.  That is up to three times the
// recurrence's work for one sequence, and worth it where few sequences leave the
// compute units idle: so long that a workgroup for every 64 columns and segment fills
// them twice (one prompt of 4096 tokens, delta rule: 190 us; not cut it would walk 64
// chunks with 32 workgroups).  Half as long, where the batch's mean length is, was slower
// for 13 uneven sequences: 7% with the rule and without.
static inline int mix_seg(const rssm_mixer_dims& d) {
  const long chunks = (d.tokens + kQ - 1) / kQ, columns = (long)d.v_heads * (d.dv / 64);
  long seg = (chunks * columns + 511) / 512;
  if (seg < 8) seg = 8;
  return (int)(seg > (1 << 20) ? (1 << 20) : seg) * kQ;
}

// Parts of a workspace, in order; every one a multiple of 16 bytes.
struct MixTake {
  size_t at = 0;
  size_t operator()(size_t bytes) {
    const size_t p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  }
};
struct SegLayout {
  size_t state, grad, decay, trans, order;
};
static inline SegLayout seg_layout(const rssm_mixer_dims& d, bool delta, bool both, MixTake& take) {
  SegLayout l{};
  if (d.tokens <= mix_seg(d)) return l;
  const size_t units = (size_t)long_places(d.tokens, d.seqs, mix_seg(d)) * d.v_heads;
  const size_t st = units * d.dk * d.dv * 4;
  l.state = take(st);
  l.grad = take(both ? st : 0);
  l.decay = take(delta ? 0 : units * 4);
  l.order = take((size_t)scan_slots(d.tokens, d.seqs, mix_seg(d)) * 4);
  l.trans = take(delta ? units * d.dk * d.dk / 512 * (both ? 2 : 1) * 64 * (d.io_dtype == RSSM_F32 ? 32 : 48) : 0);
  return l;
}
static inline void seg_fill(MixArgs& a, const rssm_mixer_dims& d, const SegLayout& l, void* workspace) {
  char* const ws = static_cast<char*>(workspace);
  a.seg = mix_seg(d);
  a.slots = (int)scan_slots(d.tokens, d.seqs, a.seg);
  a.few = long_few(d.tokens, d.seqs, a.seg);
  a.seg_state = reinterpret_cast<float*>(ws + l.state);
  a.seg_grad = reinterpret_cast<float*>(ws + l.grad);
  a.seg_decay = reinterpret_cast<float*>(ws + l.decay);
  a.trans = ws + l.trans;
  a.order = d.tokens > a.seg ? reinterpret_cast<const int32_t*>(ws + l.order) : nullptr;
}

}  // namespace rssm
