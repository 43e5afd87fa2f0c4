// Selective scan over packed sequences, backward.
//
// With S_t the states, L_t = sum_{u>=t} e^{a_u-a_t} dy_u C_u^T + (what comes
// from later chunks) their gradients, and dS the gradient of a chunk's end
// state (forward form: scan_common.hpp):
//   dx_t = D dy_t + dt_t L_t B_t
//        = D dy_t + dt_t [ sum_{u>=t} e^{a_u-a_t} (C_u.B_t) dy_u + e^{a_Q-a_t} dS B_t ]
//   dB_t = sum_heads [ sum_{u>=t} K_ut C_u + dt_t e^{a_Q-a_t} dS^T x_t ]
//   dC_u = sum_heads [ sum_{t<=u} K_ut B_t + e^{a_u} S_in^T dy_u ]
//          with K_ut = e^{a_u-a_t} dt_t (dy_u.x_t)
//   dS' = e^{a_Q} dS + sum_t e^{a_t} dy_t C_t^T      (the chunk before's)
// and for the decay exponent alpha_t = dt_t A, with w_ut = K_ut (C_u.B_t) for
// u > t, i_t = e^{a_t} dy_t^T S_in C_t and e_t = e^{a_Q-a_t} x_t^T dS B_t:
//   dalpha_t = sum_{s<t<=u} w_us + sum_{k>=t} i_k + sum_{s<t} dt_s e_s
//            + e^{a_Q} <S_in, dS>
// (each sum over one chunk).  The first is summed as it stands, from the tiles'
// rows, columns and totals, and not as the difference of the rows' and the
// columns' running sums, whose rounding would not cancel.
// ddt_t = x_t.L_t B_t + A dalpha_t, times the softplus's derivative.
//
// Launches: (1) dt and the decays' running sums of every chunk and head, once
// for all that follow; (2) both recurrences over the chunks, S_in forward and
// dS backward, which leave every chunk's in the workspace (with two launches in
// front where sequences are longer than a segment); (3) everything else, a
// workgroup for one chunk and several heads of one group, which needs nothing
// from other chunks; (4) the sums over workgroups, in a fixed order.
//
// Every factor that is not an input (S_in, dS, K and e^{a_u-a_t} C_u.B_t) enters
// its products as three bf16 terms (fp32 inputs: as it is), so nothing is rounded
// to the io type but the results.  Two terms would be 5% faster (8 x 2048 tokens of
// 80 heads: 1156 us instead of 1240 on one card) and leave three times the fp32 sums' own
// error in dB and dC; one would take dx's error without D to 1.4 times that of
// rounding it.
#include "scan_common.hpp"

namespace rssm {

struct ScanBwdArgs {
  ScanArgs f;
  const void* dy;
  const float* dfinal;
  void* dx;
  void* ddt;
  void* dB;
  void* dC;
  float* dA;
  float* dD;
  float* ddt_bias;
  float* dinit;
  float* grad_state;   // [chunk slots][V][tiles][64][4]: dS, as chunk_state holds S_in
  float* seg_grad;     // [slots][V][32][N]
  float* grad_decay;   // [slots][V], log2
  float* ddt_part;     // [units][T]
  float* dB_part;      // [hb][T][G][N]
  float* dC_part;
  float* head_part;    // [chunk slots][units][4]: dA, ddt_bias, dD
  long dy_stride, slots, cslots;
  int32_t dir_blocks;
};

// The state tile pair of column tile nt, rows tile_col(pt, 4g + r), column
// 16 nt + l%16, from natural [32][N] memory.
template <int N>
__device__ static inline long row_at(int nt, int pt, int r, int lane) {
  return (long)(pair_base(pt) + 8 * (lane >> 4) + r) * N + 16 * nt + (lane & 15);
}

// One of the two recurrences over the chunks of a segment, a wave for 32 rows of
// one head's state.  Blocks below dir_blocks: S forward; the others: dS
// backward.  STORE: from the segment's starting value, leaving every chunk's in
// the workspace (and the gradient of the initial state); otherwise from zero,
// leaving what the segment adds.  The next chunk's tiles are on their way while
// one is worked on; three workgroups a compute unit (two with 256 columns).
// Slots without a segment lie in runs, so blocks go to the dies in turn (in
// contiguous ranges one die had twice the others': 484 us instead of 365 for
// 8 x 2048 tokens of 80 heads, which write 1.34 GB).
template <typename T, int N, bool STORE>
__global__ void __launch_bounds__(256, sizeof(typename Mat<T>::E) == 4 ? 1 : (N == 256 ? 2 : 3))
    scan_states_kernel(const ScanBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  constexpr int W = 4, TH = 64 * W, V = 16 / sizeof(E);
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad, NT = N / 16;
  constexpr int PN = N / V, QN = (kQ * PN + TH - 1) / TH;  // 16-byte pieces of a row, a thread's
  constexpr int PX = kPT / V, QX = kQ * PX / 64;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sX[W][kQ * LX];
  __shared__ __attribute__((aligned(16))) float sW[W][kQ];
  const ScanArgs& a = b.f;
  int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hb = (a.vpg + W - 1) / W;
  const bool grad = (int)blockIdx.x >= b.dir_blocks;
  const int id = grad ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const long sbase = ((long)sg.seq * a.vheads + v) * (kPT * N);
  const bool has = a.init && scan_slot(a, sg.seq) >= 0 && (!a.has_init || a.has_init[sg.seq]);
  if (sg.len == 0) {
    if (STORE && grad && live && sg.empty && b.dinit) {  // the state passes through
      for (int e = lane; e < kPT * N; e += 64)
        b.dinit[sbase + e] = has && b.dfinal ? b.dfinal[sbase + e] : 0.f;
    }
    return;
  }
  if (!STORE && (grad ? sg.first : sg.last)) return;  // nothing starts from it
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (STORE && live) {
    const bool edge = grad ? sg.last : sg.first;
    const void* src = grad ? (edge ? b.dfinal : b.seg_grad) : (edge ? (has ? a.init : nullptr) : a.seg_state);
    const long base = edge ? (grad ? sbase : ((long)(has ? scan_slot(a, sg.seq) : 0) * a.vheads + v) * (kPT * N))
                           : ((long)slot * a.vheads + v) * (kPT * N);
    const bool bf = !grad && edge && a.state_bf16;
    if (src) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const long e = base + row_at<N>(n, p, r, lane);
            S[n][p][r] = bf ? Elt<bf16>::load1(src, e) : Elt<float>::load1(src, e);
          }
    }
  }
  const E* const nsrc = static_cast<const E*>(grad ? a.C : a.B) + (long)grp * N;
  const E* const psrc = static_cast<const E*>(grad ? b.dy : a.x) + (long)h * a.headdim + p0;
  const long nstride = grad ? a.C_stride : a.B_stride, pstride = grad ? b.dy_stride : a.x_stride;
  float* const out = grad ? b.grad_state : static_cast<float*>(a.chunk_state);
  const long cbase = seg_base(a.cu, sg.seq, kQ, a.tokens) + (long)sg.k * (a.seg / kQ);
  const int chunks = (sg.len + kQ - 1) / kQ;
  u32x4 rn[QN], rx[QX];
  f32x4 rq;
  const auto fetch = [&](int c) {
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    const long t0 = sg.tok + (long)c * kQ;
#pragma unroll
    for (int q = 0; q < QN; ++q) {
      const int e = q * TH + tid, r = e / PN;
      rn[q] = u32x4{0, 0, 0, 0};
      if (r < rows) rn[q] = *reinterpret_cast<const u32x4*>(nsrc + (t0 + r) * nstride + (e % PN) * V);
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * 64 + lane, r = e / PX;
      rx[q] = u32x4{0, 0, 0, 0};
      if (live && r < rows) rx[q] = *reinterpret_cast<const u32x4*>(psrc + (t0 + r) * pstride + (e % PX) * V);
    }
    rq = a.dec[((cbase + c) * a.nheads + h) * kQ + lane];
  };
  float total = 0.f;
  fetch(grad ? chunks - 1 : 0);
  for (int ci = 0; ci < chunks; ++ci) {
    const int c = grad ? chunks - 1 - ci : ci;
    tid = threadIdx.x;
    forget(tid);
    lane = tid & 63;
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    if (STORE && live) {
      f32x4* dst = reinterpret_cast<f32x4*>(out) + ((cbase + c) * a.vheads + v) * (NT * 2 * 64) + lane;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) dst[(n * 2 + p) * 64] = S[n][p];
    }
    // the last value is read only as the gradient of the initial state
    if (STORE && ci + 1 == chunks && !(grad && sg.first && b.dinit)) break;
    __syncthreads();  // the previous chunk's tiles are no longer read
#pragma unroll
    for (int q = 0; q < QN; ++q) {
      const int e = q * TH + tid, r = e / PN;
      if (r < kQ) *reinterpret_cast<u32x4*>(sB + r * LN + (e % PN) * V) = rn[q];
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * 64 + lane;
      *reinterpret_cast<u32x4*>(&sX[wave][(e / PX) * LX + (e % PX) * V]) = rx[q];
    }
    const f32x4 all = lane_of(rq, 63);
    const float decay = exp2_f32(all[0] + all[1]);
    total += all[0];
    sW[wave][lane] = grad ? exp2_f32(rq[0] + rq[1]) : rq[2] * exp2_f32(gap2(all, rq));
    if (ci + 1 < chunks) fetch(grad ? c - 1 : c + 1);
    __syncthreads();
    if (!live) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] *= decay;
    rank_update<T, NT, LX, LN, true>(S, sX[wave], sB, sW[wave], rows, lane);
  }
  if (!live) return;
  if (!STORE) {
    const long base = ((long)slot * a.vheads + v) * (kPT * N);
    float* const dst = grad ? b.seg_grad : a.seg_state;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[base + row_at<N>(n, p, r, lane)] = S[n][p][r];
    if (lane == 0) (grad ? b.grad_decay : a.seg_decay)[(long)slot * a.vheads + v] = total;
  } else if (grad && sg.first && b.dinit) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          b.dinit[sbase + row_at<N>(n, p, r, lane)] = has ? S[n][p][r] : 0.f;
  }
}

// Each sequence's segments in order (from the first to the last for the states,
// blocks below dir_blocks; from the last to the first for their gradients):
// what a segment adds is replaced by the value that it starts from.
__global__ void __launch_bounds__(256) scan_combine_both_kernel(const ScanBwdArgs b) {
  const ScanArgs& a = b.f;
  const int elems = kPT * a.dstate;
  const int per = (elems / 4 + 255) / 256;
  const bool grad = (int)blockIdx.x >= b.dir_blocks;
  const long id = grad ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int e = ((int)(id % per) * 256 + (int)threadIdx.x) * 4;
  const int v = (int)(id / per % a.vheads), i = (int)(id / per / a.vheads);
  if (e >= elems) return;
  const SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  f32x4 g = {0.f, 0.f, 0.f, 0.f};
  if (grad) {
    if (b.dfinal) g = *reinterpret_cast<const f32x4*>(b.dfinal + ((long)i * a.vheads + v) * elems + e);
  } else {
    const int pool = a.init ? scan_slot(a, i) : -1;
    if (pool >= 0 && (!a.has_init || a.has_init[i]))
      g = load_state4(a.init, ((long)pool * a.vheads + v) * elems + e, a.state_bf16);
  }
  float* const part = grad ? b.seg_grad : a.seg_state;
  const float* const dec = grad ? b.grad_decay : a.seg_decay;
  const long base = seg_base(a.cu, i, a.seg, a.tokens);
  constexpr int U = 8;  // loads in flight: one after another would take a memory latency each
  for (int q0 = 0; q0 < segs; q0 += U) {
    f32x4 own[U];
    float d[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      own[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      d[q] = 0.f;
      if (q0 + q + 1 < segs) {
        const long at = (base + (grad ? segs - 1 - q0 - q : q0 + q)) * a.vheads + v;
        own[q] = *reinterpret_cast<const f32x4*>(part + at * elems + e);
        d[q] = dec[at];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (q0 + q >= segs) break;
      const long at = (base + (grad ? segs - 1 - q0 - q : q0 + q)) * a.vheads + v;
      *reinterpret_cast<f32x4*>(part + at * elems + e) = g;
      const float w = exp2_f32(d[q]);
#pragma unroll
      for (int r = 0; r < 4; ++r) g[r] = fmaf(w, g[r], own[q][r]);
    }
  }
}

// Lane moves within a row of 16 lanes (DPP).  Zero where nothing comes in.
template <int CTRL>
__device__ static inline float row_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// Sum over the lanes of each group of 16 (values of one g), in every lane:
// partners in the pair, the four, the half row (mirrored), the row (mirrored).
__device__ static inline float sum16(float v) {
  v += row_move<0xB1>(v);
  v += row_move<0x4E>(v);
  v += row_move<0x141>(v);
  return v + row_move<0x140>(v);
}
// Sum over the lanes below (before16) or at and above (from16) in the group.
__device__ static inline float before16(float v) {
  v = row_move<0x111>(v);
  v += row_move<0x111>(v);
  v += row_move<0x112>(v);
  v += row_move<0x114>(v);
  return v + row_move<0x118>(v);
}
__device__ static inline float from16(float v) {
  v += row_move<0x101>(v);
  v += row_move<0x102>(v);
  v += row_move<0x104>(v);
  return v + row_move<0x108>(v);
}
// Sum over the four groups g, in every lane.
__device__ static inline float sum_g(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
// Inclusive sums over the wave's lanes, up to and from each lane.
__device__ static inline float upto64(float v, int lane) {
  v += row_move<0x111>(v);
  v += row_move<0x112>(v);
  v += row_move<0x114>(v);
  v += row_move<0x118>(v);
  const float a = __shfl(v, 15, 64), b = __shfl(v, 31, 64), c = __shfl(v, 47, 64);
  const int g = lane >> 4;
  return v + (g == 0 ? 0.f : (g == 1 ? a : (g == 2 ? a + b : (a + b) + c)));
}
__device__ static inline float from64(float v, int lane) {
  v = from16(v);
  const float a = __shfl(v, 16, 64), b = __shfl(v, 32, 64), c = __shfl(v, 48, 64);
  const int g = lane >> 4;
  return v + (g == 3 ? 0.f : (g == 2 ? c : (g == 1 ? b + c : a + (b + c))));
}
__device__ static inline float sum64(float v) { return sum_g(sum16(v)); }

// Waves of a workgroup of the main launch: four, or eight from 128 state columns
// on (and four for fp32's 256 columns, whose tiles leave no room for more).
constexpr int bwd_waves(bool f32, int n) { return n >= 128 && !f32 ? 8 : 4; }
// State rows of one unit of its work: 64 of a head, or 32 (headdim 32; fp32, whose
// tiles of 64 would not fit; 256 columns, whose registers would not).
static inline int bwd_rows(const rssm_scan_dims& d) {
  return d.io_dtype == RSSM_F32 || d.headdim == 32 || d.dstate == 256 ? 32 : 64;
}

// One chunk, the units of one block.  A wave owns N/W state columns (16 at 128;
// with 32, 157 registers were spilled): it holds dB and dC of all 64 tokens there in
// registers and adds every head's to them, so the heads are joined without leaving
// the workgroup.  The products of the chunk's tokens with each other (dy.x, the
// decays, C.B, which is the same for all heads) are shared: each wave works out
// some of the ten 16x16 tiles on and below the diagonal and leaves them in LDS.
template <typename T, int N, int PB>
__global__ void __launch_bounds__(64 * bwd_waves(sizeof(typename Mat<T>::E) == 4, N),
                                  sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    scan_bwd_kernel(const ScanBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int W = bwd_waves(sizeof(E) == 4, N), TH = 64 * W, V = 16 / sizeof(E);
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = PB + M::kPad, LM = kQ + M::kPad;
  constexpr int NT = N / 16, NW = NT < W ? 1 : NT / W, KB = NP / 32, SL = PB / 32;
  constexpr int PX = PB / V, QX = (kQ * PX + TH - 1) / TH;
  constexpr int kXY = kQ * LX, kMM = kQ * LM, kS = NP * LX;
  constexpr int TK = M::kTerms;
  // bf16 with 64 columns: dS's terms take K's place, at the price of a barrier, since
  // beside it they would leave room for one workgroup a compute unit instead of
  // two (8 x 2048 tokens of 80 heads: 819 us instead of 1083).
  constexpr bool kOver = sizeof(E) == 2 && N == 64 && PB == 64;
  static_assert(!kOver || (NW == 1 && NT == W && kS <= kMM), "each wave keeps its tile until K is read");
  constexpr int kWork = 2 * kXY + TK * (kOver ? kMM : kMM + kS);
  static_assert(kWork >= kQ * LN, "C's tile fits where the units work");
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E work[kWork];
  __shared__ f32x4 sCB[10][64];     // C_u.B_t by tiles
  __shared__ f32x4 sQ[kQ];
  __shared__ float sR[kQ][4];       // w: a row's sum over each earlier tile
  __shared__ float sS[4][kQ];       // w / dt: a column's sum over each later tile
  __shared__ float sI[kQ], sDQ[kQ], sDD[kQ];
  __shared__ float sP[W][kQ], sE[W][kQ], sK0[W];
  E* const sC = work;               // at the start only
  E* const sX = work;
  E* const sY = work + kXY;
  E* const sK = work + 2 * kXY;     // [t][u]: K_ut's terms, one after another
  E* const sG = kOver ? sK : sK + TK * kMM;  // [n][p]: dS's terms

  const ScanArgs& a = b.f;
  const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lane = lane0, i16 = lane & 15, g = lane >> 4;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * a.hb), rest = id % (a.ngroups * a.hb);
  const int grp = rest / a.hb, hblk = rest % a.hb;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, kQ, slot);
  const int u0 = hblk * a.upb, u1 = u0 + a.upb < a.upg ? u0 + a.upb : a.upg;
  const int units = a.upg * a.ngroups, per = a.headdim / PB;
  if (blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if (threadIdx.x == 0 && rest == 0 && sg.first && a.status && a.init && scan_slot(a, sg.seq) < 0)
    atomicOr(a.status, RSSM_ST_BAD_SLOT);
  f32x4* const hp = reinterpret_cast<f32x4*>(b.head_part) + (long)slot * units + grp * a.upg;
  if (sg.len == 0) {
    for (int u = u0 + (int)threadIdx.x; u < u1; u += TH) hp[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    return;
  }
  const int rows = sg.len;
  const long t0 = sg.tok;

  stage_tile<T, N, NP, TH>(sB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N,
                           a.B_stride, rows, threadIdx.x);
  stage_tile<T, N, NP, TH>(sC, LN, static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N,
                           a.C_stride, rows, threadIdx.x);
  __syncthreads();
  // C_u.B_t of this wave's tiles (rows u, columns t), tile k = iu (iu+1)/2 + j
  constexpr int KT = (10 + W - 1) / W;
  f32x4 cb[KT];
#pragma unroll
  for (int q = 0; q < KT; ++q) {
    const int k = wave + q * W;
    cb[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (k < 10) {
      const int iu = k < 1 ? 0 : (k < 3 ? 1 : (k < 6 ? 2 : 3)), j = k - iu * (iu + 1) / 2;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        cb[q] = M::mma(M::rows_c(sC + (16 * iu + i16) * LN + 32 * kb + 8 * g),
                       M::rows_c(sB + (16 * j + i16) * LN + 32 * kb + 8 * g), cb[q]);
      sCB[k][lane] = cb[q];
    }
  }
  // this wave's columns of C as operands (rows n, k tokens) and C's values
  // where a product's result has them (n = 4g + r, token 16 j + i16); B's are
  // read again for each unit
  Frag fc[NW][2];
  typename M::Four rc[NW][4];
#pragma unroll
  for (int q = 0; q < NW; ++q) {
    const int nt = wave * NW + q;
    if (nt < NT) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        fc[q][kb] = M::cols(cols_at<T, false>(sC, LN, 32 * kb, 16 * nt, lane), LN);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        rc[q][j] = *reinterpret_cast<const typename M::Four*>(sC + (16 * j + i16) * LN + 16 * nt + 4 * g);
    }
  }
  f32x4 aB[NW][4], aC[NW][4];
#pragma unroll
  for (int q = 0; q < NW; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) aB[q][j] = aC[q][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();  // C's tile is no longer read
  // tiles (u, t) = (0, 1) and (2, 3), above the diagonal, are read as zeros
  const auto clear = [&]() {
    for (int e = threadIdx.x; e < TK * 128; e += TH) {
      const int at = ((e >> 6) & 1) * 32, row = 16 + at + ((e >> 2) & 15);
      *reinterpret_cast<typename M::Four*>(sK + (e >> 7) * kMM + row * LM + at + 4 * (e & 3)) =
          typename M::Four{0, 0};
    }
  };
  if (!kOver) clear();
  if (N < NP)
    for (int e = threadIdx.x; e < (NP - N) * LX; e += TH)
#pragma unroll
      for (int k = 0; k < TK; ++k) Elt<T>::store1(sG + k * kS, N * LX + e, 0.f);

  u32x4 rx[QX], ry[QX];
  f32x4 rq;
  const auto fetch = [&](int u) {
    const int hu = grp * a.upg + u, h = hu / per;
    const long col = (long)h * a.headdim + (long)(hu % per) * PB;
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * TH + (int)threadIdx.x, r = e / PX, c = (e % PX) * V;
      rx[q] = ry[q] = u32x4{0, 0, 0, 0};
      if (r < rows) {
        rx[q] = *reinterpret_cast<const u32x4*>(static_cast<const E*>(a.x) + (t0 + r) * a.x_stride + col + c);
        ry[q] = *reinterpret_cast<const u32x4*>(static_cast<const E*>(b.dy) + (t0 + r) * b.dy_stride + col + c);
      }
    }
    rq = a.dec[((long)slot * a.nheads + h) * kQ + lane];
  };
  fetch(u0);
  // a unit's states in this wave's column tile nt
  f32x4 ls[SL][2], lg[SL][2];
  const auto load = [&](f32x4 (&l)[SL][2], const void* from, int u, int nt) {
    const f32x4* const p = static_cast<const f32x4*>(from) +
        ((long)slot * a.vheads + (long)(grp * a.upg + u) * SL) * (NT * 2 * 64) + lane;
#pragma unroll
    for (int s = 0; s < SL; ++s)
#pragma unroll
      for (int q = 0; q < 2; ++q) l[s][q] = p[(s * NT + nt) * 128 + q * 64];
  };

#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    const int hu = grp * a.upg + u, h = hu / per, p0 = (hu % per) * PB;
    int again = 0;
    lane = lane0;
    forget(lane);
    forget(again);
    i16 = lane & 15;
    g = lane >> 4;
    const E* const tB = sB + again;
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) forget(rc[q][j]);
    // The states' first column tile is on its way during the tokens' products.
    // Unconditional from 64 columns on: behind a condition these loads could not
    // be told from the x and dy in flight, whose wait then took them in (1322 us
    // instead of 1250 for 8 x 2048 tokens of 80 heads).
    if (NT >= W || wave * NW < NT) {
      load(ls, a.chunk_state, u, wave * NW);
      load(lg, b.grad_state, u, wave * NW);
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * TH + (int)threadIdx.x, o = (e / PX) * LX + (e % PX) * V;
      if (e >= kQ * PX) break;
      *reinterpret_cast<u32x4*>(sX + o) = rx[q];
      *reinterpret_cast<u32x4*>(sY + o) = ry[q];
    }
    if (wave == 0) sQ[lane] = rq;
    if (kOver) clear();  // dS's terms lay there
    __syncthreads();
    if (u + 1 < u1) fetch(u + 1);
    // ---- the tokens' products with each other
#pragma unroll
    for (int q = 0; q < KT; ++q) {
      const int k = wave + q * W;
      if (k >= 10) break;
      const int iu = k < 1 ? 0 : (k < 3 ? 1 : (k < 6 ? 2 : 3)), j = k - iu * (iu + 1) / 2;
      const int t = 16 * j + i16, uu = 16 * iu + 4 * g;
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < SL; ++s)
        d = M::mma(M::rows_c(sY + (16 * iu + i16) * LX + 32 * s + 8 * g),
                   M::rows_c(sX + t * LX + 32 * s + 8 * g), d);
      const f32x4 qt = sQ[t];
      float kk[4], col = 0.f, rw[4], in = 0.f, dd = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = exp2_f32(gap2(sQ[uu + r], qt));
        const bool on = uu + r >= t;
        kk[r] = on ? e * d[r] * qt[2] : 0.f;
        const float s = on ? e * cb[q][r] * d[r] : 0.f;
        col += s;
        rw[r] = s * qt[2];
        if (iu == j) {
          // within the tile: sum of w_us over s < t <= u, for this t
          const float p = before16(uu + r > t ? rw[r] : 0.f);
          in += on ? p : 0.f;
          dd += uu + r == t ? d[r] : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < TK; ++k) {
        const typename M::Four k1 = M::pack4(kk);
        *reinterpret_cast<typename M::Four*>(sK + k * kMM + t * LM + uu) = k1;
        if (k + 1 < TK) {
          float q1[4];
          M::unpack4(k1, q1);
#pragma unroll
          for (int r = 0; r < 4; ++r) kk[r] -= q1[r];
        }
      }
      col = sum_g(col);
      if (iu == j) {
        in = sum_g(in);
        dd = sum_g(dd);
        if (g == 0) {
          sI[t] = in;
          sDQ[t] = col;
          sDD[t] = dd;
        }
      } else {
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = sum16(rw[r]);
          mine = (i16 & 3) == r ? s : mine;
        }
        if (i16 < 4) sR[uu + i16][j] = mine;
        if (g == 0) sS[iu][t] = col;
      }
      keep_order();
    }
    __syncthreads();

    // ---- dC, dB and the states' part of the decay's gradient
    const f32x4 qa = sQ[kQ - 1];
    Split<T, TK> kept[SL];  // dS's terms, until they may be written
    if (wave * NW < NT) {
      float et[4], ft[4], dti[4], doti[4], dote[4], k0 = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 q = sQ[16 * j + i16];
        et[j] = exp2_f32(q[0] + q[1]);
        ft[j] = exp2_f32(gap2(qa, q));
        dti[j] = q[2] * ft[j];
        doti[j] = dote[j] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const int nt = wave * NW + q;
        Split<T, TK> hs[SL];
        const auto split = [&](const f32x4 (&l)[SL][2]) {
#pragma unroll
          for (int s = 0; s < SL; ++s) {
            float f[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              f[r] = l[s][0][r];
              f[4 + r] = l[s][1][r];
            }
            hs[s].set(f);
          }
        };
#pragma unroll
        for (int s = 0; s < SL; ++s)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int r = 0; r < 4; ++r) k0 = fmaf(ls[s][p][r], lg[s][p][r], k0);
        split(ls);
        if (q + 1 < NW) load(ls, a.chunk_state, u, nt + 1);
        Frag fb[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          fb[kb] = M::cols(cols_at<T, false>(tB, LN, 32 * kb, 16 * nt, lane), LN);
        keep_order();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < SL; ++s)
            acc = hs[s].a_times(M::rows_c(sY + (16 * j + i16) * LX + 32 * s + 8 * g), acc);
#pragma unroll
          for (int kb = 0; kb <= j / 2; ++kb)
#pragma unroll
            for (int e = TK - 1; e >= 0; --e)
              aC[q][j] = M::mma(fb[kb], M::cols(cols_at<T, false>(sK + e * kMM, LM, 32 * kb, 16 * j, lane), LM),
                                aC[q][j]);
          float cv[4];
          M::unpack4(rc[q][j], cv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            doti[j] = fmaf(acc[r], cv[r], doti[j]);
            aC[q][j][r] = fmaf(et[j], acc[r], aC[q][j][r]);
          }
          keep_order();
        }
        split(lg);
        if (q + 1 < NW) load(lg, b.grad_state, u, nt + 1);
        if constexpr (kOver) {
#pragma unroll
          for (int s = 0; s < SL; ++s) kept[s] = hs[s];
        } else {
#pragma unroll
          for (int s = 0; s < SL; ++s)
#pragma unroll
            for (int k = 0; k < TK; ++k)
              *reinterpret_cast<Frag*>(sG + k * kS + (16 * nt + i16) * LX + 32 * s + 8 * g) = hs[s].t[k];
        }
        keep_order();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < SL; ++s)
            acc = hs[s].a_times(M::rows_c(sX + (16 * j + i16) * LX + 32 * s + 8 * g), acc);
#pragma unroll
          for (int kb = j / 2; kb < 2; ++kb)
#pragma unroll
            for (int e = TK - 1; e >= 0; --e)
              aB[q][j] = M::mma(fc[q][kb], M::rows_d(sK + e * kMM + (16 * j + i16) * LM + 32 * kb + 4 * g),
                                aB[q][j]);
          float bv[4];
          M::unpack4(*reinterpret_cast<const typename M::Four*>(tB + (16 * j + i16) * LN + 16 * nt + 4 * g), bv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            dote[j] = fmaf(acc[r], bv[r], dote[j]);
            aB[q][j][r] = fmaf(dti[j], acc[r], aB[q][j][r]);
          }
          keep_order();
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float i = sum_g(doti[j]) * et[j], e = sum_g(dote[j]) * ft[j];
        if (g == 0) {
          sP[wave][16 * j + i16] = i;
          sE[wave][16 * j + i16] = e;
        }
      }
      k0 = sum64(k0);
      if (lane == 0) sK0[wave] = k0;
    }
    __syncthreads();
    if constexpr (kOver) {
#pragma unroll
      for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int k = 0; k < TK; ++k)
          *reinterpret_cast<Frag*>(sG + k * kS + (16 * wave + i16) * LX + 32 * s + 8 * g) = kept[s].t[k];
      __syncthreads();
    }

    // ---- dx: a wave takes every other slice of 32 rows and some of the tokens
    {
      constexpr int NJ = 8 / W;  // token tiles of a wave: j and 3 - j, or one
      const int jw = wave >> 1;
      for (int s = wave & 1; s < SL; s += 2) {
        f32x4 X[NJ][2];
#pragma unroll
        for (int q = 0; q < NJ; ++q) X[q][0] = X[q][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          Frag f[2][TK];
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < TK; ++k)
              f[p][k] = M::cols(cols_at<T, true>(sG + k * kS, LX, 32 * kb, 32 * s + pair_base(p), lane), LX);
#pragma unroll
          for (int q = 0; q < NJ; ++q) {
            const int j = q ? 3 - jw : jw;
            const Frag bt = M::rows_d(tB + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
            for (int k = TK - 1; k >= 0; --k)
#pragma unroll
              for (int p = 0; p < 2; ++p) X[q][p] = M::mma(f[p][k], bt, X[q][p]);
          }
          keep_order();
        }
#pragma unroll
        for (int q = 0; q < NJ; ++q) {
          const int j = q ? 3 - jw : jw, t = 16 * j + i16;
          const f32x4 qt = sQ[t];
          const float ft = exp2_f32(gap2(qa, qt));
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int r = 0; r < 4; ++r) X[q][p][r] *= ft;
          for (int kb = j >> 1; kb < 2; ++kb) {
            // e^{a_u-a_t} C_u.B_t, as a product's result holds it and an operand wants it
            float m[8];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const int iu = 2 * kb + h2, uu = 16 * iu + 4 * g;
              const f32x4 c = sCB[iu < j ? 0 : iu * (iu + 1) / 2 + j][lane];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float e = exp2_f32(gap2(sQ[uu + r], qt)) * c[r];
                m[4 * h2 + r] = uu + r >= t ? e : 0.f;
              }
            }
            Split<T, TK> mf;
            mf.set(m);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              X[q][p] = mf.b_times(M::cols(cols_at<T, true>(sY, LX, 32 * kb, 32 * s + pair_base(p), lane), LX),
                                   X[q][p]);
          }
          if (t < rows) {
            const float Dh = a.D ? a.D[h] : 0.f;
            float o[8], yv[8];
            M::unpack(M::rows_c(sY + t * LX + 32 * s + 8 * g), yv);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              o[r] = fmaf(Dh, yv[r], qt[2] * X[q][0][r]);
              o[4 + r] = fmaf(Dh, yv[4 + r], qt[2] * X[q][1][r]);
            }
            Vec8<T>::store(b.dx, (t0 + t) * (long)a.nheads * a.headdim + (long)h * a.headdim + p0 +
                                     32 * s + 8 * g, o);
          }
        }
      }
    }
    // ---- the decay's gradient, one token per lane; the waves take turns
    if (wave == (u & (W - 1))) {
      const f32x4 q = sQ[lane];
      const float dt = q[2];
      float row = 0.f, cs = 0.f, pi = 0.f, pe = 0.f, k0 = 0.f;
#pragma unroll
      for (int k = 0; k < 3; ++k) row += k < g ? sR[lane][k] : 0.f;
#pragma unroll
      for (int k = 1; k < 4; ++k) cs += k > g ? sS[k][lane] : 0.f;
#pragma unroll
      for (int w = 0; w < (NT < W ? NT : W); ++w) {
        pi += sP[w][lane];
        pe += sE[w][lane];
        k0 += sK0[w];
      }
      // totals of the tiles later and earlier than this token's on either side
      const float s0 = sum16(g >= 2 ? sR[lane][0] : 0.f), s1 = sum16(g == 3 ? sR[lane][1] : 0.f);
      const float t20 = __shfl(s0, 32, 64), t30 = __shfl(s0, 48, 64), t31 = __shfl(s1, 48, 64);
      const float w = sI[lane] + from16(row) + before16(cs * dt) +
                      (g == 1 ? t20 + t30 : (g == 2 ? t30 + t31 : 0.f));
      const float ahead = dt * pe;
      const float dal = k0 * exp2_f32(qa[0] + qa[1]) + w + from64(pi, lane) + (upto64(ahead, lane) - ahead);
      const float sig = a.dt_softplus ? 1.f / (1.f + expf(-q[3])) : 1.f;
      const float dd = lane < rows ? (cs + sDQ[lane] + pe + a.A[h] * dal) * sig : 0.f;
      if (lane < rows) b.ddt_part[(long)hu * a.tokens + t0 + lane] = dd;
      const float sa = sum64(lane < rows ? dal * dt : 0.f), sb = sum64(dd), sd = sum64(sDD[lane]);
      if (lane == 0) hp[u] = f32x4{sa, sb, sd, 0.f};
    }
    __syncthreads();  // the unit's tiles are no longer read
  }

#pragma unroll
  for (int q = 0; q < NW; ++q) {
    const int nt = wave * NW + q;
    if (nt >= NT) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 16 * j + i16;
      if (t < rows) {
        const long o = (((long)hblk * a.tokens + t0 + t) * a.ngroups + grp) * N + 16 * nt + 4 * g;
        *reinterpret_cast<f32x4*>(b.dB_part + o) = aB[q][j];
        *reinterpret_cast<f32x4*>(b.dC_part + o) = aC[q][j];
      }
    }
  }
}

// The partial sums: dB and dC over the workgroups of a group's heads, ddt over
// a head's slices, dA, dD and ddt_bias over segments and slices.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_join_kernel(const ScanBwdArgs b, int nbc, int nd) {
  const ScanArgs& a = b.f;
  int id = blockIdx.x;
  const long tgn = (long)a.tokens * a.ngroups * a.dstate;
  if (id < 2 * nbc) {
    const float* part = id < nbc ? b.dB_part : b.dC_part;
    void* dst = id < nbc ? b.dB : b.dC;
    const long e = ((long)(id < nbc ? id : id - nbc) * 256 + threadIdx.x) * 8;
    if (e >= tgn) return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < a.hb; ++k) {
      float o[8];
      Vec8<float>::load(part + k * tgn, e, o);
#pragma unroll
      for (int r = 0; r < 8; ++r) s[r] += o[r];
    }
    Vec8<T>::store(dst, e, s);
    return;
  }
  id -= 2 * nbc;
  const int units = a.upg * a.ngroups, slices = units / a.nheads;
  if (id < nd) {
    // 64 tokens of 16 heads: read along tokens, written along heads
    __shared__ float tile[64][17];
    const int hblocks = (a.nheads + 15) / 16;
    const long t0 = (long)(id / hblocks) * 64;
    const int h0 = (id % hblocks) * 16;
    for (int e = threadIdx.x; e < 1024; e += 256) {
      const int t = e & 63, h = h0 + (e >> 6);
      float s = 0.f;
      if (t0 + t < a.tokens && h < a.nheads)
        for (int k = 0; k < slices; ++k)
          s += b.ddt_part[((long)h * slices + k) * a.tokens + t0 + t];
      tile[t][e >> 6] = s;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 1024; e += 256) {
      const int t = e >> 4, h = h0 + (e & 15);
      if (t0 + t < a.tokens && h < a.nheads)
        Elt<T>::store1(b.ddt, (t0 + t) * a.nheads + h, tile[t][e & 15]);
    }
    return;
  }
  id -= nd;
  // one wave a head
  const int h = id * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (h >= a.nheads) return;
  double s[3] = {0.0, 0.0, 0.0};
  for (long k = lane; k < b.cslots * slices; k += 64) {
    const f32x4 p = reinterpret_cast<const f32x4*>(b.head_part)[(k / slices) * units + (long)h * slices + k % slices];
#pragma unroll
    for (int r = 0; r < 3; ++r) s[r] += (double)p[r];
  }
#pragma unroll
  for (int r = 0; r < 3; ++r)
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[r] += __shfl_xor(s[r], o, 64);
  if (lane == 0) {
    b.dA[h] = (float)s[0];
    if (b.ddt_bias) b.ddt_bias[h] = (float)s[1];
    if (b.dD) b.dD[h] = (float)s[2];
  }
}

// Tokens of a segment of the recurrences: enough of them, over both directions,
// to give every one of the 1024 SIMDs two waves, and no shorter than four chunks.
static int bwd_seg(const rssm_scan_dims& d) {
  const long vheads = (long)d.nheads * (d.headdim / kPT);
  const long want = (d.tokens * vheads + 1023) / 1024;
  long seg = (want + kQ - 1) / kQ * kQ;
  if (seg < 4 * kQ) seg = 4 * kQ;
  if (seg > 64 * kQ) seg = 64 * kQ;
  return (int)seg;
}

// Units of a workgroup of the main launch: up to sixteen, which share the chunk's
// C.B and join dB and dC without memory, but so few that there are two
// workgroups for each place (one a compute unit with eight waves, two with
// four).  8 x 2048 tokens of 80 heads: 16 units 1250 us, 8 1291, 4 1393; two
// uneven sequences of 1291 tokens, 128 heads in 8 groups: two workgroups a place
// 264 us, one or four 288.
static int bwd_units(const rssm_scan_dims& d, int upg) {
  const long blocks = ((long)d.tokens / kQ + d.seqs) * d.ngroups;
  const long least = bwd_waves(d.io_dtype == RSSM_F32, d.dstate) == 8 ? 512 : 1024;
  int n = 16;
  while (n > 1 && blocks * ((upg + n - 1) / n) < least) n >>= 1;
  return n;
}

// The workspace, in order; every part a multiple of 16 bytes.
struct BwdLayout {
  size_t dec, chunk_state, grad_state, seg_state, seg_grad, seg_decay, grad_decay, ddt, dB, dC, head, end;
  int upg, upb, hb;
};
static BwdLayout bwd_layout(const rssm_scan_dims& d) {
  const size_t T = d.tokens, n = d.seqs, seg = bwd_seg(d);
  const size_t V = (size_t)d.nheads * (d.headdim / kPT), hpn = (size_t)d.nheads * d.headdim * d.dstate;
  const size_t slots = T / seg + n, cslots = T / kQ + n;
  BwdLayout l;
  l.upg = d.nheads / d.ngroups * (d.headdim / bwd_rows(d));
  l.upb = bwd_units(d, l.upg);
  l.hb = (l.upg + l.upb - 1) / l.upb;
  const size_t units = (size_t)l.upg * d.ngroups;
  const bool many = T > seg;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  l.dec = take(cslots * d.nheads * kQ * 16);
  l.chunk_state = take(cslots * hpn * 4);
  l.grad_state = take(cslots * hpn * 4);
  l.seg_state = take(many ? slots * hpn * 4 : 0);
  l.seg_grad = take(many ? slots * hpn * 4 : 0);
  l.seg_decay = take(many ? slots * V * 4 : 0);
  l.grad_decay = take(many ? slots * V * 4 : 0);
  l.ddt = take(units * T * 4);
  l.dB = take(l.hb * T * d.ngroups * d.dstate * 4);
  l.dC = take(l.hb * T * d.ngroups * d.dstate * 4);
  l.head = take(cslots * units * 16);
  l.end = at;
  return l;
}

enum { kStates, kSegments, kMain };
template <typename T, int N>
static const void* pick_bwd_n(int which, const rssm_scan_dims& d) {
  if (which == kStates) return reinterpret_cast<const void*>(&scan_states_kernel<T, N, true>);
  if (which == kSegments) return reinterpret_cast<const void*>(&scan_states_kernel<T, N, false>);
  if constexpr (sizeof(typename Mat<T>::E) == 2 && N < 256)
    if (bwd_rows(d) == 64) return reinterpret_cast<const void*>(&scan_bwd_kernel<T, N, 64>);
  return reinterpret_cast<const void*>(&scan_bwd_kernel<T, N, 32>);
}
template <typename T>
static const void* pick_bwd(int which, const rssm_scan_dims& d) {
  switch (d.dstate) {
    case 16: return pick_bwd_n<T, 16>(which, d);
    case 32: return pick_bwd_n<T, 32>(which, d);
    case 64: return pick_bwd_n<T, 64>(which, d);
    case 128: return pick_bwd_n<T, 128>(which, d);
    default: return pick_bwd_n<T, 256>(which, d);
  }
}

}  // namespace rssm

using namespace rssm;

extern "C" size_t ssu_scan_backward_workspace(const rssm_scan_dims* dims) {
  if (scan_check(dims)) return 0;
  return bwd_layout(*dims).end;
}

extern "C" int ssu_scan_backward(const rssm_scan_dims* dims, const void* dy, const void* x,
                                 const void* dt, const float* A, const void* B, const void* C,
                                 const float* D, const float* dt_bias, const int32_t* cu_seqlens,
                                 const void* initial_state, const uint8_t* has_initial,
                                 const int32_t* slot_idx, const float* dfinal_state, void* dx,
                                 void* ddt, void* dB, void* dC, float* dA, float* dD,
                                 float* ddt_bias, float* dinitial_state, void* workspace,
                                 size_t workspace_bytes, int32_t* status, hipStream_t stream) {
  int rc = scan_check(dims);
  if (rc) return rc;
  const rssm_scan_dims& d = *dims;
  if (d.seqs == 0 && d.tokens > 0) return RSSM_EINVAL;
  if (!A || !dA) return RSSM_EINVAL;
  if (d.tokens > 0 && (!dy || !x || !dt || !B || !C || !dx || !ddt || !dB || !dC))
    return RSSM_EINVAL;
  if (!cu_seqlens && d.seqs > 1) return RSSM_EINVAL;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(dx) ||
      !aligned16(dB) || !aligned16(dC) || !aligned16(initial_state) || !aligned16(dfinal_state) ||
      !aligned16(dinitial_state) || !aligned16(workspace))
    return RSSM_EINVAL;
  const BwdLayout l = bwd_layout(d);
  if (l.end && (!workspace || workspace_bytes < l.end)) return RSSM_EINVAL;
  char* const ws = static_cast<char*>(workspace);
  ScanBwdArgs b{};
  ScanArgs& a = b.f;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.B = B;
  a.C = C;
  a.D = D;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.init = initial_state;
  a.has_init = has_initial;
  a.slot_idx = slot_idx;
  a.status = status;
  fill_dims(a, d);
  a.seg = bwd_seg(d);
  a.vheads = d.nheads * (d.headdim / kPT);
  a.vpg = a.vheads / d.ngroups;
  a.seg_state = reinterpret_cast<float*>(ws + l.seg_state);
  a.seg_decay = reinterpret_cast<float*>(ws + l.seg_decay);
  b.dy = dy;
  b.dfinal = dfinal_state;
  b.dx = dx;
  b.ddt = ddt;
  b.dB = dB;
  b.dC = dC;
  b.dA = dA;
  b.dD = dD;
  b.ddt_bias = ddt_bias;
  b.dinit = dinitial_state;
  a.dec = reinterpret_cast<f32x4*>(ws + l.dec);
  a.chunk_state = ws + l.chunk_state;
  b.grad_state = reinterpret_cast<float*>(ws + l.grad_state);
  b.seg_grad = reinterpret_cast<float*>(ws + l.seg_grad);
  b.grad_decay = reinterpret_cast<float*>(ws + l.grad_decay);
  b.ddt_part = reinterpret_cast<float*>(ws + l.ddt);
  b.dB_part = reinterpret_cast<float*>(ws + l.dB);
  b.dC_part = reinterpret_cast<float*>(ws + l.dC);
  b.head_part = reinterpret_cast<float*>(ws + l.head);
  b.dy_stride = d.dy_stride ? d.dy_stride : (long)d.nheads * d.headdim;
  b.slots = scan_slots(d.tokens, d.seqs, a.seg);
  b.cslots = scan_slots(d.tokens, d.seqs, kQ);
  a.upg = l.upg;
  a.upb = l.upb;
  a.hb = l.hb;
  const bool f32 = d.io_dtype == RSSM_F32;
  const long sgrid = b.slots * d.ngroups * ((a.vpg + 3) / 4);
  const long mgrid = b.cslots * d.ngroups * a.hb;
  const long dgrid = b.cslots * ((d.nheads + 3) / 4);
  const long cgrid = ((long)kPT * d.dstate / 4 + 255) / 256 * a.vheads * d.seqs;
  const long nbc = ((long)d.tokens * d.ngroups * d.dstate / 8 + 255) / 256;
  const long nd = ((long)d.tokens + 63) / 64 * ((d.nheads + 15) / 16);
  const long jgrid = 2 * nbc + nd + (d.nheads + 3) / 4;
  const long most = 1L << 23;  // 2^32 threads of up to 512
  if (2 * sgrid >= most || mgrid >= most || dgrid >= most || 2 * cgrid >= most || jgrid >= most)
    return RSSM_ESHAPE;
  const auto go = [&](int which, long grid, int threads) {
    const void* fn = f32 ? pick_bwd<float>(which, d) : pick_bwd<bf16>(which, d);
    return launch_kernel(fn, (unsigned)grid, threads, 0, stream, b);
  };
  if (d.seqs > 0) {
    if (d.tokens > 0)
      rc = f32 ? launch_decay<float>(a, b.cslots, stream) : launch_decay<bf16>(a, b.cslots, stream);
    if (!rc && d.tokens > a.seg) {
      b.dir_blocks = (int32_t)sgrid;
      rc = go(kSegments, 2 * sgrid, 256);
      b.dir_blocks = (int32_t)cgrid;
      if (!rc)
        rc = launch_kernel(reinterpret_cast<const void*>(&scan_combine_both_kernel),
                           (unsigned)(2 * cgrid), 256, 0, stream, b);
    }
    b.dir_blocks = (int32_t)sgrid;
    if (!rc) rc = go(kStates, 2 * sgrid, 256);
    if (!rc) rc = go(kMain, mgrid, 64 * bwd_waves(f32, d.dstate));
    if (rc) return rc;
  }
  int inbc = (int)nbc, ind = (int)nd;
  void* kargs[] = {&b, &inbc, &ind};
  const void* fn = f32 ? reinterpret_cast<const void*>(&scan_bwd_join_kernel<float>)
                       : reinterpret_cast<const void*>(&scan_bwd_join_kernel<bf16>);
  return hipLaunchKernel(fn, dim3((unsigned)jgrid), dim3(256), kargs, 0, stream) == hipSuccess
             ? RSSM_OK
             : RSSM_ELAUNCH;
}
