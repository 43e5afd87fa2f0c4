// Selective scan over packed sequences, backward.
//
// With S_t the states, L_t = sum_{u>=t} e^{a_u-a_t} dy_u C_u^T + (what comes
// from later chunks) their gradients, and dS the gradient of a chunk's end
// state (forward form: scan_common.hpp):
//   dx_t = D dy_t + dt_t L_t B_t
//        = D dy_t + dt_t [ sum_{u>=t} e^{a_u-a_t} (C_u.B_t) dy_u + e^{a_Q-a_t} dS B_t ]
//   dB_t = dt_t sum_heads [ sum_{u>=t} e^{a_u-a_t} (dy_u.x_t) C_u + e^{a_Q-a_t} dS^T x_t ]
//   dC_t = sum_heads [ sum_{s<=t} e^{a_t-a_s} dt_s (dy_t.x_s) B_s + e^{a_t} S_in^T dy_t ]
//   dS' = e^{a_Q} dS + sum_t e^{a_t} dy_t C_t^T      (the chunk before's)
// and for the decay exponent alpha_t = dt_t A, with w_ut = e^{a_u-a_t} dt_t
// (C_u.B_t)(dy_u.x_t) for u > t, i_t = e^{a_t} dy_t^T S_in C_t and
// e_t = e^{a_Q-a_t} x_t^T dS B_t:
//   dalpha_t = sum_{s<t<=u} w_us + sum_{k>=t} i_k + sum_{s<t} dt_s e_s
//            + e^{a_Q} <S_in, dS>
// (each sum over one chunk).  The first is summed as it stands, from the tiles'
// rows, columns and totals, and not as the difference of the rows' and the
// columns' running sums, whose rounding would not cancel.
// ddt_t = x_t.L_t B_t + A dalpha_t, times the softplus's derivative.
//
// Everything that reaches an fp32 output (dA, ddt_bias, dinitial_state, and
// ddt through dalpha) takes its state products with the state as three bf16
// terms; what only reaches an output in the io type rounds one factor once
// (dx) or takes two terms (dB, dC, which are sums over heads).
//
// A wave owns 32 rows of one head's state.  The states S_in come from a
// forward launch that leaves every chunk's in the workspace in the layout of
// the accumulators; the main launch walks a segment's chunks backwards with dS
// in registers.  dB and dC are joined over a workgroup's waves in LDS and over
// workgroups by a last launch, in a fixed order.
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
  float* chunk_state;  // [chunk slots][V][tiles][64][4]
  float* seg_grad;     // [slots][V][32][N]
  float* grad_decay;   // [slots][V], log2
  float* ddt_part;     // [V][T]
  float* dB_part;      // [hb][T][G][N]
  float* dC_part;
  double* head_part;   // [slots][V][3]: dA, ddt_bias, dD
  long dy_stride, slots;
  int32_t hb;
};

// Waves of a workgroup: what the tiles leave room for in 160 KB of LDS.
constexpr int bwd_waves(bool f32, int n) { return f32 ? (n == 256 ? 1 : 2) : (n == 256 ? 4 : 8); }

// The state tile pair of column tile nt, rows tile_col(pt, 4g + r), column
// 16 nt + l%16, from natural [32][N] memory.
template <int N>
__device__ static inline long row_at(int nt, int pt, int r, int lane) {
  return (long)(pair_base(pt) + 8 * (lane >> 4) + r) * N + 16 * nt + (lane & 15);
}

// GRAD false: forward over a segment from its starting state, leaving each
// chunk's S_in in the workspace.  GRAD true: backward over a segment from a
// zero dS, leaving the gradient of its start (what the segment adds).
template <typename T, int N, bool GRAD>
__global__ void __launch_bounds__(256) scan_states_kernel(const ScanBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  constexpr int W = 4;
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad, NT = N / 16;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sX[W][kQ * LX];
  __shared__ __attribute__((aligned(16))) float sW[W][kQ];
  const ScanArgs& a = b.f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hb = (a.vpg + W - 1) / W;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  if (sg.len == 0 || (GRAD && sg.first)) return;
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!GRAD && live) {
    const int pool = sg.first && a.init ? scan_slot(a, sg.seq) : -1;
    const bool from_pool = pool >= 0 && (!a.has_init || a.has_init[sg.seq]);
    if (!sg.first || from_pool) {
      const void* src = sg.first ? a.init : a.seg_state;
      const long base = ((long)(sg.first ? pool : slot) * a.vheads + v) * (kPT * N);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const long e = base + row_at<N>(n, p, r, lane);
            S[n][p][r] = sg.first && a.state_bf16 ? Elt<bf16>::load1(src, e)
                                                  : Elt<float>::load1(src, e);
          }
    }
  }
  const long cbase = seg_base(a.cu, sg.seq, kQ, a.tokens) + (long)sg.k * (a.seg / kQ);
  const int chunks = (sg.len + kQ - 1) / kQ;
  double total = 0.0;
  for (int ci = 0; ci < chunks; ++ci) {
    const int c = GRAD ? chunks - 1 - ci : ci;
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    const long t0 = sg.tok + c * kQ;
    if (!GRAD && live) {
      f32x4* dst = reinterpret_cast<f32x4*>(b.chunk_state) +
                   ((cbase + c) * a.vheads + v) * (NT * 2 * 64) + lane;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) dst[(n * 2 + p) * 64] = S[n][p];
    }
    if (!GRAD && c + 1 == chunks) break;  // the last chunk's end state is not read
    __syncthreads();
    const void* nsrc = GRAD ? a.C : a.B;
    const long nstride = GRAD ? a.C_stride : a.B_stride;
    stage_tile<T, N, NP, 64 * W>(sB, LN,
                                 static_cast<const E*>(nsrc) + t0 * nstride + (long)grp * N,
                                 nstride, rows, threadIdx.x);
    const void* psrc = GRAD ? b.dy : a.x;
    const long pstride = GRAD ? b.dy_stride : a.x_stride;
    stage_tile<T, kPT, kPT, 64>(sX[wave], LX,
                                static_cast<const E*>(psrc) + t0 * pstride +
                                    (long)h * a.headdim + p0,
                                pstride, live ? rows : 0, lane);
    const ChunkDt q = chunk_dt<T>(a, h, bias, A2, t0, rows, lane);
    total += q.all;
    sW[wave][lane] = GRAD ? exp2_f32((float)q.cum) : q.dt * exp2_f32((float)(q.all - q.cum));
    const float decay = exp2_f32((float)q.all);
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
  if (GRAD && live) {
    const long base = ((long)slot * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) b.seg_grad[base + row_at<N>(n, p, r, lane)] = S[n][p][r];
    if (lane == 0) b.grad_decay[(long)slot * a.vheads + v] = (float)total;
  }
}

// Each sequence's segments from the last to the first: what a segment adds is
// replaced by the gradient of its end state (the last one's is dfinal).
__global__ void __launch_bounds__(256) scan_combine_grad_kernel(const ScanBwdArgs b) {
  const ScanArgs& a = b.f;
  const int elems = kPT * a.dstate;
  const int per = (elems / 4 + 255) / 256;
  const long id = blockIdx.x;
  const int e = ((int)(id % per) * 256 + (int)threadIdx.x) * 4;
  const int v = (int)(id / per % a.vheads), i = (int)(id / per / a.vheads);
  if (e >= elems) return;
  const SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  f32x4 g = {0.f, 0.f, 0.f, 0.f};
  if (b.dfinal)
    g = *reinterpret_cast<const f32x4*>(b.dfinal + ((long)i * a.vheads + v) * elems + e);
  const long base = seg_base(a.cu, i, a.seg, a.tokens);
  for (int k = segs - 1; k >= 0; --k) {
    const long at = (base + k) * a.vheads + v;
    f32x4* const p = reinterpret_cast<f32x4*>(b.seg_grad + at * elems + e);
    f32x4 own = {0.f, 0.f, 0.f, 0.f};
    float d = 0.f;
    if (k) {
      own = *p;
      d = exp2_f32(b.grad_decay[at]);
    }
    *p = g;
#pragma unroll
    for (int r = 0; r < 4; ++r) g[r] = fmaf(d, g[r], own[r]);
  }
}

// Nothing is scheduled across this point: fully unrolled, the compiler would
// start every tile's products at once and spill what they leave.
__device__ static inline void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// The value is unknown from here on: what was computed from it is computed
// again where it is next needed, instead of being kept in registers (the three
// passes over the chunk's tiles share their products and decays, 80 registers).
__device__ static inline void forget(float& v) { asm volatile("" : "+v"(v)); }
__device__ static inline void forget(u32x4& v) { asm volatile("" : "+v"(v)); }
__device__ static inline void forget(Mat<float>::Frag& f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) forget(f.v[e]);
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
__device__ static inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <typename T, int N>
__global__ void __launch_bounds__(64 * bwd_waves(sizeof(typename Mat<T>::E) == 4, N))
    scan_bwd_kernel(const ScanBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int W = bwd_waves(sizeof(E) == 4, N), TH = 64 * W;
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad;
  constexpr int NT = N / 16, KB = NP / 32, T2 = M::kTerms == 1 ? 1 : 2;
  constexpr int LE = kPT + M::kPad;
  constexpr int kRed = W * 4 * 64 * 16;              // one n-tile of every wave
  constexpr int kEx = W * 32 * LE * (int)sizeof(E);  // 32 state columns of every wave
  constexpr int kShare = 2 * kRed > kEx ? 2 * kRed : kEx;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sC[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sY[W][kQ * LX];
  __shared__ f32x4 sCB[10][64];
  __shared__ __attribute__((aligned(16))) char share[kShare];
  __shared__ float2 sA[W][kQ];
  __shared__ __attribute__((aligned(16))) float sD[W][kQ];
  __shared__ __attribute__((aligned(16))) float sE[W][kQ];  // e^{a_t}

  const ScanArgs& a = b.f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g = lane >> 4;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * b.hb), rest = id % (a.ngroups * b.hb);
  const int grp = rest / b.hb, hblk = rest % b.hb, vl = hblk * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  double* const hp = b.head_part + ((long)slot * a.vheads + v) * 3;
  if (threadIdx.x == 0 && rest == 0 && sg.first && a.status) {
    if (sg.bad) atomicOr(a.status, RSSM_ST_BAD_SEQ);
    if (a.init && scan_slot(a, sg.seq) < 0) atomicOr(a.status, RSSM_ST_BAD_SLOT);
  }
  const long sbase = ((long)sg.seq * a.vheads + v) * (kPT * N);
  const bool has = a.init && scan_slot(a, sg.seq) >= 0 && (!a.has_init || a.has_init[sg.seq]);
  if (sg.len == 0) {
    if (live && lane < 3) hp[lane] = 0.0;
    if (live && sg.empty && b.dinit) {  // the state passes through
      for (int e = lane; e < kPT * N; e += 64)
        b.dinit[sbase + e] = has && b.dfinal ? b.dfinal[sbase + e] : 0.f;
    }
    return;
  }
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const float Ah = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

  // dS: rows tile_col(pt, 4g + r), columns 16 nt + i16
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (live && (!sg.last || b.dfinal)) {
    const float* src = sg.last ? b.dfinal + sbase
                               : b.seg_grad + ((long)slot * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] = src[row_at<N>(n, p, r, lane)];
  }
  double sum_a = 0.0, sum_b = 0.0, sum_d = 0.0;
  const long cbase = seg_base(a.cu, sg.seq, kQ, a.tokens) + (long)sg.k * (a.seg / kQ);

  for (int c = (sg.len + kQ - 1) / kQ - 1; c >= 0; --c) {
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    const long t0 = sg.tok + c * kQ;
    __syncthreads();
    stage_tile<T, N, NP, TH>(sB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N,
                             a.B_stride, rows, threadIdx.x);
    stage_tile<T, N, NP, TH>(sC, LN, static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N,
                             a.C_stride, rows, threadIdx.x);
    // x and dy rows 16 j + i16, elements 8g.. (order D of the state's rows)
    Frag xf[4], yf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 16 * j + i16;
      float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      xf[j] = yf[j] = M::pack(z);
      if (live && t < rows) {
        const long col = (long)h * a.headdim + p0 + 8 * g;
        xf[j] = M::rows_c(static_cast<const E*>(a.x) + (t0 + t) * a.x_stride + col);
        yf[j] = M::rows_c(static_cast<const E*>(b.dy) + (t0 + t) * b.dy_stride + col);
      }
      *reinterpret_cast<Frag*>(&sY[wave][t * LX + 8 * g]) = yf[j];
    }
    const ChunkDt q = chunk_dt<T>(a, h, bias, A2, t0, rows, lane);
    {
      const float hi = (float)q.cum;
      sA[wave][lane] = make_float2(hi, (float)(q.cum - (double)hi));
      sD[wave][lane] = q.dt;
      sE[wave][lane] = exp2_f32((float)q.cum);
    }
    const float decay = exp2_f32((float)q.all);
    const float ahi = (float)q.all, alo = (float)(q.all - (double)ahi);
    __syncthreads();
    // C_u.B_t for the ten tiles on and below the diagonal, shared by the heads
    for (int k = wave; k < 10; k += W) {
      const int iu = k < 1 ? 0 : (k < 3 ? 1 : (k < 6 ? 2 : 3)), j = k - iu * (iu + 1) / 2;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = M::mma(M::rows_c(sC + (16 * iu + i16) * LN + 32 * kb + 8 * g),
                     M::rows_c(sB + (16 * j + i16) * LN + 32 * kb + 8 * g), acc);
      sCB[k][lane] = acc;
    }
    __syncthreads();

    // ---- this head's products inside the chunk, rows u, columns t
    float2 at[4];
    float dt_t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at[j] = sA[wave][16 * j + i16];
      dt_t[j] = sD[wave][16 * j + i16];
    }
    const auto forget_all = [&]() {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        forget(xf[j]);
        forget(yf[j]);
        forget(at[j].x);
        forget(at[j].y);
        forget(dt_t[j]);
      }
    };
    float my_w = 0.f, my_q = 0.f, my_i = 0.f, my_e = 0.f;
    float tot[2] = {0.f, 0.f};  // w over (u, s) tiles {2,3} x {0} and {3} x {0,1}
    {
      f32x4 X[4][2];  // dx^T: rows tile_col(p, 4g + r), column t
#pragma unroll
      for (int j = 0; j < 4; ++j) X[j][0] = X[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      // e^{a_Q - a_t} dS B_t: dS goes through LDS (32 columns at a time) to
      // turn its rows into operand rows, rounded to the io type as dx is
      E* const ex = reinterpret_cast<E*>(share) + wave * 32 * LE;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int n = 2 * kb + q2;
            E* const d = ex + (16 * q2 + i16) * LE + pair_base(p) + 8 * g;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              Elt<T>::store1(d, r, n < NT ? S[n < NT ? n : 0][p][r] : 0.f);
          }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_s_waitcnt(0xc07f);  // the wave's own LDS writes are in
        __builtin_amdgcn_wave_barrier();
        Frag sf[2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
          sf[p] = M::cols(cols_at<T, true>(ex, LE, 0, pair_base(p), lane), LE);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Frag bt = M::rows_d(sB + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
          for (int p = 0; p < 2; ++p) X[j][p] = M::mma(sf[p], bt, X[j][p]);
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_s_waitcnt(0xc07f);  // and read before the next columns land
        __builtin_amdgcn_wave_barrier();
        keep_order();
      }
      float racc[4][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float et = exp2_f32((ahi - at[j].x) + (alo - at[j].y));
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) X[j][p][r] *= et;
        float col = 0.f, in = 0.f, diag = 0.f, dd = 0.f;
#pragma unroll
        for (int kb = j / 2; kb < 2; ++kb) {
          float m1[8];
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const int iu = 2 * kb + q2;
#pragma unroll
            for (int r = 0; r < 4; ++r) m1[4 * q2 + r] = 0.f;
            if (iu < j) continue;
            const f32x4 dxt = M::mma(yf[iu], xf[j], f32x4{0.f, 0.f, 0.f, 0.f});
            const f32x4 cb = sCB[iu * (iu + 1) / 2 + j][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int u = 16 * iu + 4 * g + r, t = 16 * j + i16;
              const float e = exp2_f32(gap2(sA[wave][u], at[j]));
              const float m = u >= t ? e * cb[r] : 0.f;
              const float s = m * dxt[r];
              m1[4 * q2 + r] = m;
              if (iu > j) {
                const float w = s * dt_t[j];
                col += s;
                racc[iu][r] += w;
                if (j == 0 && iu >= 2) tot[0] += w;
                if (j <= 1 && iu == 3) tot[1] += w;
              } else {
                // within the tile: sum of w_us over s < t <= u, for this t
                const float p = before16(u > t ? s * dt_t[j] : 0.f);
                in += u >= t ? p : 0.f;
                diag += u >= t ? s : 0.f;
                dd += u == t ? dxt[r] : 0.f;
              }
            }
          }
          const Frag mf = M::pack(m1);
#pragma unroll
          for (int p = 0; p < 2; ++p)
            X[j][p] = M::mma(M::cols(cols_at<T, true>(sY[wave], LX, 32 * kb, pair_base(p), lane),
                                     LX), mf, X[j][p]);
        }
        // u >= t in this tile's rows, u in later tiles
        col = sum_g(col);
        const float w = before16(col * dt_t[j]) + sum_g(in);
        const float qq = col + sum_g(diag);
        if (g == j) {
          my_w = w;
          my_q = qq;
        }
        sum_d += (double)dd;
        const int t = 16 * j + i16;
        if (live && t < rows) {
          float o[8], yv[8];
          M::unpack(yf[j], yv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r] = fmaf(Dh, yv[r], dt_t[j] * X[j][0][r]);
            o[4 + r] = fmaf(Dh, yv[4 + r], dt_t[j] * X[j][1][r]);
          }
          Vec8<T>::store(b.dx, (t0 + t) * (long)a.nheads * a.headdim + (long)h * a.headdim + p0 +
                                   8 * g, o);
        }
        keep_order();
      }
      // rows' sums over the columns of earlier tiles, u at and after t: token
      // 16 iu + 4g + r is in the lanes of g, and goes to lane 4g + r first
#pragma unroll
      for (int iu = 1; iu < 4; ++iu) {
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float got = __shfl(sum16(racc[iu][r]), 16 * (i16 >> 2), 64);
          mine = (i16 & 3) == r ? got : mine;
        }
        mine = from16(mine);
        if (g == iu) my_w += mine;
      }
      const float t1 = sum_g(sum16(tot[0])), t2 = sum_g(sum16(tot[1]));
      my_w += g == 1 ? t1 : (g == 2 ? t2 : 0.f);
    }
    __syncthreads();  // the exchange's memory becomes the joining buffers
    forget_all();

    // ---- dC, then dB: a column tile of 16 at a time over all tokens, joined
    // over the waves (two buffers: one barrier a tile)
    f32x4(*const red)[W][4][64] = reinterpret_cast<f32x4(*)[W][4][64]>(share);
    double k0 = 0.0;
    const auto join = [&](int buf, int nt, float* part) {
      for (int e = threadIdx.x; e < 256; e += TH) {
        const int j = e >> 6, l = e & 63;
        f32x4 s = red[buf][0][j][l];
#pragma unroll
        for (int w = 1; w < W; ++w) {
          const f32x4 o = red[buf][w][j][l];
#pragma unroll
          for (int r = 0; r < 4; ++r) s[r] += o[r];
        }
        const int t = 16 * j + (l & 15);
        if (t < rows)
          *reinterpret_cast<f32x4*>(part + (((long)hblk * a.tokens + t0 + t) * a.ngroups + grp) * N +
                                    16 * nt + 4 * (l >> 4)) = s;
      }
    };
    {
      Split<T, T2> m3[4][2];  // e^{a_t - a_s} dt_s (x_s.dy_t): rows s, columns t
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int kb = 0; kb <= j / 2; ++kb) {
          float m[8];
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const int is = 2 * kb + q2;
#pragma unroll
            for (int r = 0; r < 4; ++r) m[4 * q2 + r] = 0.f;
            if (is > j) continue;
            const f32x4 dxt = M::mma(xf[is], yf[j], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int s = 16 * is + 4 * g + r, t = 16 * j + i16;
              const float e = exp2_f32(gap2(at[j], sA[wave][s])) * sD[wave][s];
              m[4 * q2 + r] = s <= t ? e * dxt[r] : 0.f;
            }
          }
          m3[j][kb].set(m);
          keep_order();
        }
      float dot[4] = {0.f, 0.f, 0.f, 0.f};
      const f32x4* src = reinterpret_cast<const f32x4*>(b.chunk_state) +
                         ((cbase + c) * a.vheads + v) * (NT * 2 * 64) + lane;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const f32x4 s0 = live ? src[nt * 128] : f32x4{0.f, 0.f, 0.f, 0.f};
        const f32x4 s1 = live ? src[nt * 128 + 64] : f32x4{0.f, 0.f, 0.f, 0.f};
        float f[8], ks = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = s0[r];
          f[4 + r] = s1[r];
          ks = fmaf(s0[r], S[nt][0][r], fmaf(s1[r], S[nt][1][r], ks));
        }
        k0 += (double)ks;
        Split<T, M::kTerms> ss;
        ss.set(f);
        Frag bc[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          bc[kb] = M::cols(cols_at<T, false>(sB, LN, 32 * kb, 16 * nt, lane), LN);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = ss.a_times(yf[j], f32x4{0.f, 0.f, 0.f, 0.f});
          const E* cp = sC + (16 * j + i16) * LN + 16 * nt + 4 * g;
          const float et = sE[wave][16 * j + i16];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            dot[j] = fmaf(acc[r], Elt<T>::load1(cp, r), dot[j]);
            acc[r] *= et;
          }
#pragma unroll
          for (int kb = 0; kb <= j / 2; ++kb) acc = m3[j][kb].b_times(bc[kb], acc);
          red[nt & 1][wave][j][lane] = acc;
          keep_order();
        }
        __syncthreads();
        join(nt & 1, nt, b.dC_part);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = sum_g(dot[j]) * sE[wave][16 * j + i16];
        if (g == j) my_i = s;
      }
    }
    __syncthreads();
    forget_all();
    {
      Split<T, T2> m2[4][2];  // e^{a_u - a_t} (dy_u.x_t): rows u, columns t
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int kb = j / 2; kb < 2; ++kb) {
          float m[8];
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const int iu = 2 * kb + q2;
#pragma unroll
            for (int r = 0; r < 4; ++r) m[4 * q2 + r] = 0.f;
            if (iu < j) continue;
            const f32x4 dxt = M::mma(yf[iu], xf[j], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int u = 16 * iu + 4 * g + r, t = 16 * j + i16;
              const float e = exp2_f32(gap2(sA[wave][u], at[j]));
              m[4 * q2 + r] = u >= t ? e * dxt[r] : 0.f;
            }
          }
          m2[j][kb].set(m);
          keep_order();
        }
      float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = S[nt][0][r];
          f[4 + r] = S[nt][1][r];
        }
        Split<T, M::kTerms> ss;
        ss.set(f);
        Frag cc[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          cc[kb] = M::cols(cols_at<T, false>(sC, LN, 32 * kb, 16 * nt, lane), LN);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = ss.a_times(xf[j], f32x4{0.f, 0.f, 0.f, 0.f});
          const E* bp = sB + (16 * j + i16) * LN + 16 * nt + 4 * g;
          const float et = exp2_f32((ahi - at[j].x) + (alo - at[j].y));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            dot[j] = fmaf(acc[r], Elt<T>::load1(bp, r), dot[j]);
            acc[r] *= et;
          }
#pragma unroll
          for (int kb = j / 2; kb < 2; ++kb) acc = m2[j][kb].b_times(cc[kb], acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] *= dt_t[j];
          red[nt & 1][wave][j][lane] = acc;
          keep_order();
        }
        __syncthreads();
        join(nt & 1, nt, b.dB_part);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = sum_g(dot[j]) * exp2_f32((ahi - at[j].x) + (alo - at[j].y));
        if (g == j) my_e = s;
      }
    }
    // ---- the decay's gradient, one token per lane
    k0 = wave_sum(k0) * (double)decay;
    {
      const double back = (double)my_i;
      const double ahead = (double)q.dt * (double)my_e;
      const double sb = wave_cumsum(back, lane), sf = wave_cumsum(ahead, lane);
      const double dal = k0 + (double)my_w + (__shfl(sb, 63, 64) - sb + back) + (sf - ahead);
      const double sig = a.dt_softplus ? 1.0 / (1.0 + (double)expf(-q.raw)) : 1.0;
      const double dd = ((double)my_q + (double)my_e + (double)Ah * dal) * sig;
      if (lane < rows) {
        sum_a += dal * (double)q.dt;
        sum_b += dd;
        if (live) b.ddt_part[(long)v * a.tokens + t0 + lane] = (float)dd;
      }
    }
    // ---- the gradient of the chunk before's end state
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] *= decay;
    rank_update<T, NT, LX, LN, true>(S, sY[wave], sC, sE[wave], rows, lane);
  }
  if (!live) return;
  sum_a = wave_sum(sum_a);
  sum_b = wave_sum(sum_b);
  sum_d = wave_sum(sum_d);
  if (lane == 0) {
    hp[0] = sum_a;
    hp[1] = sum_b;
    hp[2] = sum_d;
  }
  if (sg.first && b.dinit) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          b.dinit[sbase + row_at<N>(n, p, r, lane)] = has ? S[n][p][r] : 0.f;
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
    for (int k = 0; k < b.hb; ++k) {
      float o[8];
      Vec8<float>::load(part + k * tgn, e, o);
#pragma unroll
      for (int r = 0; r < 8; ++r) s[r] += o[r];
    }
    Vec8<T>::store(dst, e, s);
    return;
  }
  id -= 2 * nbc;
  const int slices = a.headdim / kPT;
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
  for (long k = lane; k < b.slots * slices; k += 64) {
    const double* p = b.head_part + ((k / slices) * a.vheads + (long)h * slices + k % slices) * 3;
#pragma unroll
    for (int r = 0; r < 3; ++r) s[r] += p[r];
  }
#pragma unroll
  for (int r = 0; r < 3; ++r) s[r] = wave_sum(s[r]);
  if (lane == 0) {
    b.dA[h] = (float)s[0];
    if (b.ddt_bias) b.ddt_bias[h] = (float)s[1];
    if (b.dD) b.dD[h] = (float)s[2];
  }
}

// Tokens of a backward segment.
static int bwd_seg(const rssm_scan_dims& d) {
  const long vheads = (long)d.nheads * (d.headdim / kPT);
  const long want = (d.tokens * vheads + 2047) / 2048;
  long seg = (want + kQ - 1) / kQ * kQ;
  if (seg < 4 * kQ) seg = 4 * kQ;
  if (seg > 64 * kQ) seg = 64 * kQ;
  return (int)seg;
}

// The workspace, in order; every part a multiple of 16 bytes.
struct BwdLayout {
  size_t chunk_state, seg_state, seg_grad, seg_decay, grad_decay, ddt, dB, dC, head, end;
};
static BwdLayout bwd_layout(const rssm_scan_dims& d) {
  const size_t T = d.tokens, n = d.seqs, seg = bwd_seg(d);
  const size_t V = (size_t)d.nheads * (d.headdim / kPT), hpn = (size_t)d.nheads * d.headdim * d.dstate;
  const size_t slots = T / seg + n, cslots = T / kQ + n;
  const size_t waves = bwd_waves(d.io_dtype == RSSM_F32, d.dstate);
  const size_t hb = (V / d.ngroups + waves - 1) / waves;
  const bool many = T > seg;
  const auto up = [](size_t b) { return (b + 15) / 16 * 16; };
  BwdLayout l;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t p = at;
    at += up(bytes);
    return p;
  };
  l.chunk_state = take(cslots * hpn * 4);
  l.seg_state = take(many ? slots * hpn * 4 : 0);
  l.seg_grad = take(many ? slots * hpn * 4 : 0);
  l.seg_decay = take(many ? slots * V * 4 : 0);
  l.grad_decay = take(many ? slots * V * 4 : 0);
  l.ddt = take(V * T * 4);
  l.dB = take(hb * T * d.ngroups * d.dstate * 4);
  l.dC = take(hb * T * d.ngroups * d.dstate * 4);
  l.head = take(slots * V * 3 * 8);
  l.end = at;
  return l;
}

enum { kStates, kGrads, kMain };
template <typename T>
static const void* pick_bwd(int which, int n) {
#define RSSM_SCAN_BWD(N)                                                                    \
  if (n == N)                                                                               \
  return which == kStates  ? reinterpret_cast<const void*>(&scan_states_kernel<T, N, false>) \
         : which == kGrads ? reinterpret_cast<const void*>(&scan_states_kernel<T, N, true>)  \
                           : reinterpret_cast<const void*>(&scan_bwd_kernel<T, N>)
  RSSM_SCAN_BWD(16);
  RSSM_SCAN_BWD(32);
  RSSM_SCAN_BWD(64);
  RSSM_SCAN_BWD(128);
  RSSM_SCAN_BWD(256);
  return nullptr;
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
  b.chunk_state = reinterpret_cast<float*>(ws + l.chunk_state);
  b.seg_grad = reinterpret_cast<float*>(ws + l.seg_grad);
  b.grad_decay = reinterpret_cast<float*>(ws + l.grad_decay);
  b.ddt_part = reinterpret_cast<float*>(ws + l.ddt);
  b.dB_part = reinterpret_cast<float*>(ws + l.dB);
  b.dC_part = reinterpret_cast<float*>(ws + l.dC);
  b.head_part = reinterpret_cast<double*>(ws + l.head);
  b.dy_stride = d.dy_stride ? d.dy_stride : (long)d.nheads * d.headdim;
  b.slots = scan_slots(d.tokens, d.seqs, a.seg);
  const bool f32 = d.io_dtype == RSSM_F32;
  const int waves = bwd_waves(f32, d.dstate);
  b.hb = (a.vpg + waves - 1) / waves;
  const long sgrid = b.slots * d.ngroups * ((a.vpg + 3) / 4);
  const long mgrid = b.slots * d.ngroups * b.hb;
  const long cgrid = ((long)kPT * d.dstate / 4 + 255) / 256 * a.vheads * d.seqs;
  const long nbc = ((long)d.tokens * d.ngroups * d.dstate / 8 + 255) / 256;
  const long nd = ((long)d.tokens + 63) / 64 * ((d.nheads + 15) / 16);
  const long jgrid = 2 * nbc + nd + (d.nheads + 3) / 4;
  if (sgrid > 0x7fffffffL || mgrid > 0x7fffffffL || cgrid > 0x7fffffffL || jgrid > 0x7fffffffL)
    return RSSM_ESHAPE;
  const auto go = [&](int which, long grid, int threads) {
    const void* fn = f32 ? pick_bwd<float>(which, d.dstate) : pick_bwd<bf16>(which, d.dstate);
    return launch_kernel(fn, (unsigned)grid, threads, 0, stream, b);
  };
  if (d.seqs > 0) {
    if (d.tokens > a.seg) {
      rc = scan_segment_states(a, d, stream);
      if (!rc) rc = go(kGrads, sgrid, 256);
      if (!rc)
        rc = launch_kernel(reinterpret_cast<const void*>(&scan_combine_grad_kernel),
                           (unsigned)cgrid, 256, 0, stream, b);
    }
    if (!rc && d.tokens > 0) rc = go(kStates, sgrid, 256);
    if (!rc) rc = go(kMain, mgrid, 64 * waves);
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
