// Selective scan over packed sequences, forward (see scan_common.hpp for the
// chunked form).
//
// Long calls: (1) dt and the decays' running sums of every chunk and head; (2)
// the recurrence over the chunks, a wave for 32 rows of one head's state, which
// leaves the state before every chunk in the workspace, in fp32 (with two
// launches in front where sequences are longer than a segment: what each segment
// adds from zero, then their running combination); (3) the outputs, a workgroup
// for one chunk and several heads.
// Short calls (up to kShort tokens) are one launch, in which a wave walks a
// sequence's chunks with the state in registers.
//
// Both factors of y that are fp32, the state and dt e^{a_t-a_s} C_t.B_s, enter
// its products as three bf16 terms (fp32 inputs: as they are), so nothing is
// rounded to the io type but y itself.  One term would take y's error without D
// from 1.0 to 1.4 times that of rounding y.
#include "scan_common.hpp"

namespace rssm {

// Waves of a workgroup: four, or two where fp32 tiles of dstate 256 would not
// fit four heads' x beside them in 160 KB.
constexpr int scan_waves(bool f32, int n) { return f32 && n == 256 ? 2 : 4; }

// A short call in one launch: y and the final states, a wave for 32 rows of one
// head's state and one sequence.  Two workgroups a compute unit: 256 registers a
// lane.  61 fp32 tokens of 8 heads (dstate 16): 13 us, a serial chain.
template <typename T, int N>
__global__ void __launch_bounds__(64 * scan_waves(sizeof(typename Mat<T>::E) == 4, N),
                                  sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    scan_short_kernel(const ScanArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int W = scan_waves(sizeof(E) == 4, N), TH = 64 * W;
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad;
  constexpr int NT = N / 16, KB = NP / 32;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sC[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sX[W][kQ * LX];
  __shared__ f32x4 sCB[10][64];
  __shared__ float2 sA[W][kQ];
  __shared__ __attribute__((aligned(16))) float sD[W][kQ];  // dt
  __shared__ __attribute__((aligned(16))) float sW[W][kQ];  // weight of x in the state

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g = lane >> 4;
  const int hb = (a.vpg + W - 1) / W;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  if (sg.len == 0 && !sg.empty) return;
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

  // state tiles S^T: rows n = 16 nt + 4g + r, columns tile_col(p, i16)
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int pool = a.init || a.final_state ? scan_slot(a, sg.seq) : -1;
  if (threadIdx.x == 0 && rest == 0 && a.status) {
    if (sg.bad) atomicOr(a.status, RSSM_ST_BAD_SEQ);
    if ((a.init || a.final_state) && pool < 0) atomicOr(a.status, RSSM_ST_BAD_SLOT);
  }
  if (live && a.init && pool >= 0 && (!a.has_init || a.has_init[sg.seq])) {
    const long base = ((long)pool * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        S[n][p] = load_state4(a.init, base + tile_col(p, i16) * N + 16 * n + 4 * g, a.state_bf16);
  }

  for (int c0 = 0; c0 < sg.len; c0 += kQ) {
    const int rows = sg.len - c0 < kQ ? sg.len - c0 : kQ;
    const long t0 = sg.tok + c0;
    __syncthreads();  // the previous chunk's tiles are no longer read
    stage_tile<T, N, NP, TH>(sB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N,
                             a.B_stride, rows, threadIdx.x);
    stage_tile<T, N, NP, TH>(sC, LN,
                               static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N,
                               a.C_stride, rows, threadIdx.x);
    stage_tile<T, kPT, kPT, 64>(sX[wave], LX,
                                static_cast<const E*>(a.x) + t0 * a.x_stride +
                                    (long)h * a.headdim + p0,
                                a.x_stride, live ? rows : 0, lane);
    const ChunkDt q = chunk_dt<T>(a, h, bias, A2, t0, rows, lane);
    {
      const float hi = (float)q.cum;
      sA[wave][lane] = make_float2(hi, (float)(q.cum - (double)hi));
      sD[wave][lane] = q.dt;
      sW[wave][lane] = q.dt * exp2_f32((float)(q.all - q.cum));
    }
    const float decay = exp2_f32((float)q.all);
    __syncthreads();

    {
      // C_t.B_s for the ten tiles on and above the diagonal (rows s, columns
      // t), shared by the workgroup's heads
      for (int k = wave; k < 10; k += W) {
        const int j = k < 1 ? 0 : (k < 3 ? 1 : (k < 6 ? 2 : 3)), i = k - j * (j + 1) / 2;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          acc = M::mma(M::rows_c(sB + (16 * i + i16) * LN + 32 * kb + 8 * g),
                       M::rows_c(sC + (16 * j + i16) * LN + 32 * kb + 8 * g), acc);
        sCB[k][lane] = acc;
      }
      f32x4 Y[4][2];  // y^T: rows tile_col(p, 4g + r), column t = 16 j + i16
#pragma unroll
      for (int j = 0; j < 4; ++j) Y[j][0] = Y[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      // e^{a_t} S C_t
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Split<T, M::kTerms> sf[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float f[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            f[r] = S[2 * kb][p][r];
            f[4 + r] = 2 * kb + 1 < NT ? S[2 * kb + 1 < NT ? 2 * kb + 1 : 0][p][r] : 0.f;
          }
          sf[p].set(f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Frag c = M::rows_d(sC + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][p] = sf[p].a_times(c, Y[j][p]);
        }
      }
      float2 at[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        at[j] = sA[wave][16 * j + i16];
        const float et = exp2_f32(at[j].x + at[j].y);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) Y[j][p][r] *= et;
      }
      __syncthreads();  // sCB
      // the chunk's own tokens
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        Frag xf[2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
          xf[p] = M::cols(cols_at<T, true>(sX[wave], LX, 32 * sb, pair_base(p), lane), LX);
#pragma unroll
        for (int j = 2 * sb; j < 4; ++j) {
          float w[8];
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const int i = 2 * sb + q2;
#pragma unroll
            for (int r = 0; r < 4; ++r) w[4 * q2 + r] = 0.f;
            if (i > j) continue;
            const f32x4 cb = sCB[j * (j + 1) / 2 + i][lane];
            const f32x4 ds = *reinterpret_cast<const f32x4*>(&sD[wave][16 * i + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float m = cb[r] * ds[r] * exp2_f32(gap2(at[j], sA[wave][16 * i + 4 * g + r]));
              w[4 * q2 + r] = i < j || 4 * g + r <= i16 ? m : 0.f;
            }
          }
          Split<T, M::kTerms> wf;
          wf.set(w);
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][p] = wf.b_times(xf[p], Y[j][p]);
          keep_order();
        }
      }
      // D x, the gate, and 8 neighbours of token t to memory
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 16 * j + i16;
        if (live && t < rows) {
          float o[8], xv[8];
          M::unpack(M::rows_c(sX[wave] + t * LX + 8 * g), xv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r] = fmaf(Dh, xv[r], Y[j][0][r]);
            o[4 + r] = fmaf(Dh, xv[4 + r], Y[j][1][r]);
          }
          const long col = (long)h * a.headdim + p0 + 8 * g;
          if (a.z) {
            float zv[8];
            Vec8<T>::load(a.z, (t0 + t) * a.z_stride + col, zv);
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] *= zv[r] * sigmoid_f32(zv[r]);
          }
          Vec8<T>::store(a.y, (t0 + t) * (long)a.nheads * a.headdim + col, o);
        }
      }
    }
    // S' = e^{a_Q} S + sum_t (w_t x_t) B_t
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] *= decay;
    rank_update<T, NT, LX, LN, false>(S, sX[wave], sB, sW[wave], rows, lane);
  }

  if (live && a.final_state && pool >= 0) {
    const long base = ((long)pool * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        store_state4(a.final_state, base + tile_col(p, i16) * N + 16 * n + 4 * g, a.state_bf16,
                     S[n][p]);
  }
}

// The recurrence over the chunks of a segment.  STORE: from the state it starts
// from, leaving the state before every chunk (the tiles as the lanes hold them)
// and the final one in its pool; otherwise from zero, leaving what the segment
// adds.  The next chunk's tiles are on their way while one is worked on.
// Slots without a segment lie in runs, so blocks go to the dies in turn.
// 16383 tokens of 80 heads: 218 us storing (0.84 GB: 3.8 TB/s), 110 us not.
template <typename T, int N, bool STORE>
__global__ void __launch_bounds__(256, sizeof(typename Mat<T>::E) == 4 ? 1 : (N == 256 ? 2 : 3))
    scan_fwd_states_kernel(const ScanArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  constexpr int W = 4, TH = 64 * W, V = 16 / sizeof(E);
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad, NT = N / 16;
  constexpr int PN = N / V, QN = (kQ * PN + TH - 1) / TH;  // 16-byte pieces of a row, a thread's
  constexpr int PX = kPT / V, QX = kQ * PX / 64;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sX[W][kQ * LX];
  __shared__ __attribute__((aligned(16))) float sW[W][kQ];
  int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hb = (a.vpg + W - 1) / W;
  const int id = blockIdx.x;
  // here and not in the first launch, whose many small workgroups it slows (16383
  // tokens of 80 heads: 16.9 us instead of 13.6)
  if (STORE && id == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  if (STORE ? sg.len == 0 && !sg.empty : sg.len == 0 || sg.last) return;
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  const int pool = a.init || a.final_state ? scan_slot(a, sg.seq) : -1;
  if (STORE && threadIdx.x == 0 && rest == 0 && sg.first && a.status && (a.init || a.final_state) && pool < 0)
    atomicOr(a.status, RSSM_ST_BAD_SLOT);
  // S^T: rows n = 16 nt + 4g + r, columns tile_col(p, l%16)
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto place = [&](int n, int p) { return tile_col(p, lane & 15) * N + 16 * n + 4 * (lane >> 4); };
  // The pool is read here only by a sequence of one segment, whose wave also
  // writes it: a longer one's first segment takes the copy that the combining
  // launch left, since its last segment may already have stored the final
  // state over the initial one.
  const bool whole = sg.first && sg.last;
  const bool from_pool = whole && a.init && pool >= 0 && (!a.has_init || a.has_init[sg.seq]);
  if (STORE && live && (from_pool || !whole)) {
    const void* src = whole ? a.init : a.seg_state;
    const long base = ((long)(whole ? pool : slot) * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) S[n][p] = load_state4(src, base + place(n, p), whole ? a.state_bf16 : 0);
  }
  const E* const nsrc = static_cast<const E*>(a.B) + (long)grp * N;
  const E* const psrc = static_cast<const E*>(a.x) + (long)h * a.headdim + p0;
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
      if (r < rows) rn[q] = *reinterpret_cast<const u32x4*>(nsrc + (t0 + r) * a.B_stride + (e % PN) * V);
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * 64 + lane, r = e / PX;
      rx[q] = u32x4{0, 0, 0, 0};
      if (live && r < rows) rx[q] = *reinterpret_cast<const u32x4*>(psrc + (t0 + r) * a.x_stride + (e % PX) * V);
    }
    rq = a.dec[((cbase + c) * a.nheads + h) * kQ + lane];
  };
  float total = 0.f;
  if (chunks) fetch(0);
  for (int c = 0; c < chunks; ++c) {
    tid = threadIdx.x;
    forget(tid);
    lane = tid & 63;
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    if (STORE && live) {
      f32x4* dst = static_cast<f32x4*>(a.chunk_state) + ((cbase + c) * a.vheads + v) * (NT * 2 * 64) + lane;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) dst[(n * 2 + p) * 64] = S[n][p];
    }
    if (STORE && c + 1 == chunks && !(sg.last && a.final_state)) break;  // the end is not read
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
    sW[wave][lane] = rq[2] * exp2_f32(gap2(all, rq));
    if (c + 1 < chunks) fetch(c + 1);
    __syncthreads();
    if (!live) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] *= decay;
    rank_update<T, NT, LX, LN, false>(S, sX[wave], sB, sW[wave], rows, lane);
  }
  if (!live) return;
  if (!STORE) {
    const long base = ((long)slot * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) store_state4(a.seg_state, base + place(n, p), 0, S[n][p]);
    if (lane == 0) a.seg_decay[(long)slot * a.vheads + v] = total;
  } else if (sg.last && a.final_state && pool >= 0) {
    const long base = ((long)pool * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        store_state4(a.final_state, base + place(n, p), a.state_bf16, S[n][p]);
  }
}

// The outputs of one chunk.  C and the tiles of C.B, the same for all heads of
// the group, are in LDS; each wave then works alone, a unit (PB state rows of one
// head) at a time, without a barrier: the waves are at different points, and one's
// loads pass behind the others' products.  16383 tokens of 80 heads: 283 us, 1.0 GB
// (3.6 TB/s), two thirds of it the states.
template <typename T, int N, int PB>
__global__ void __launch_bounds__(256, sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    scan_fwd_out_kernel(const ScanArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int W = 4, TH = 64 * W, V = 16 / sizeof(E);
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = PB + M::kPad;
  constexpr int NT = N / 16, KB = NP / 32, SL = PB / 32;
  constexpr int PX = PB / V, QX = kQ * PX / 64;
  constexpr int kX = W * kQ * LX > kQ * LN ? W * kQ * LX : kQ * LN;
  __shared__ __attribute__((aligned(16))) E sC[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sXB[kX];  // B at first, then each wave's x
  __shared__ f32x4 sCB[10][64];
  __shared__ f32x4 sQ[W][kQ];
  int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * a.hb), rest = id % (a.ngroups * a.hb);
  const int grp = rest / a.hb, u0 = (rest % a.hb) * a.upb;
  const int u1 = u0 + a.upb < a.upg ? u0 + a.upb : a.upg, per = a.headdim / PB;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, kQ, slot);
  if (sg.len == 0) return;
  const int rows = sg.len;
  const long t0 = sg.tok;
  {
    const int i16 = lane & 15, g = lane >> 4;
    stage_tile<T, N, NP, TH>(sXB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N,
                             a.B_stride, rows, threadIdx.x);
    stage_tile<T, N, NP, TH>(sC, LN, static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N,
                             a.C_stride, rows, threadIdx.x);
    __syncthreads();
    // C_t.B_s for the ten tiles on and above the diagonal (rows s, columns t)
    for (int k = wave; k < 10; k += W) {
      const int j = k < 1 ? 0 : (k < 3 ? 1 : (k < 6 ? 2 : 3)), i = k - j * (j + 1) / 2;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = M::mma(M::rows_c(sXB + (16 * i + i16) * LN + 32 * kb + 8 * g),
                     M::rows_c(sC + (16 * j + i16) * LN + 32 * kb + 8 * g), acc);
      sCB[k][lane] = acc;
    }
    __syncthreads();
  }
  E* const sX = sXB + wave * kQ * LX;
#pragma unroll 1
  for (int u = u0 + wave; u < u1; u += W) {
    const int hu = grp * a.upg + u, h = hu / per, p0 = (hu % per) * PB;
    lane = threadIdx.x & 63;
    forget(lane);
    const int i16 = lane & 15, g = lane >> 4;
    u32x4 rx[QX];
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * 64 + lane, r = e / PX;
      rx[q] = u32x4{0, 0, 0, 0};
      if (r < rows)
        rx[q] = *reinterpret_cast<const u32x4*>(static_cast<const E*>(a.x) + (t0 + r) * a.x_stride +
                                                (long)h * a.headdim + p0 + (e % PX) * V);
    }
    sQ[wave][lane] = a.dec[((long)slot * a.nheads + h) * kQ + lane];
    // e^{a_t} S C_t: y^T, rows tile_col(p, 4g + r) of a slice, column t = 16 j + i16
    f32x4 Y[4][SL][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < SL; ++s) Y[j][s][0] = Y[j][s][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    const f32x4* const st = static_cast<const f32x4*>(a.chunk_state) +
        ((long)slot * a.vheads + (long)hu * SL) * (NT * 2 * 64) + lane;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Split<T, M::kTerms> sf[SL][2];
#pragma unroll
      for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const f32x4 lo = st[((s * NT + 2 * kb) * 2 + p) * 64];
          const f32x4 hi = 2 * kb + 1 < NT ? st[((s * NT + 2 * kb + 1) * 2 + p) * 64] : f32x4{0.f, 0.f, 0.f, 0.f};
          const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          sf[s][p].set(f);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Frag c = M::rows_d(sC + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
        for (int s = 0; s < SL; ++s)
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][s][p] = sf[s][p].a_times(c, Y[j][s][p]);
      }
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int e = q * 64 + lane;
      *reinterpret_cast<u32x4*>(sX + (e / PX) * LX + (e % PX) * V) = rx[q];
    }
    wave_sync();
    f32x4 at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at[j] = sQ[wave][16 * j + i16];
      const float et = exp2_f32(at[j][0] + at[j][1]);
#pragma unroll
      for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) Y[j][s][p][r] *= et;
    }
    // the chunk's own tokens
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      Frag xf[SL][2];
#pragma unroll
      for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          xf[s][p] = M::cols(cols_at<T, true>(sX, LX, 32 * sb, 32 * s + pair_base(p), lane), LX);
#pragma unroll
      for (int j = 2 * sb; j < 4; ++j) {
        float w[8];
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          const int i = 2 * sb + q2;
#pragma unroll
          for (int r = 0; r < 4; ++r) w[4 * q2 + r] = 0.f;
          if (i > j) continue;
          const f32x4 cb = sCB[j * (j + 1) / 2 + i][lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f32x4 qs = sQ[wave][16 * i + 4 * g + r];
            const float m = cb[r] * qs[2] * exp2_f32(gap2(at[j], qs));
            w[4 * q2 + r] = i < j || 4 * g + r <= i16 ? m : 0.f;
          }
        }
        Split<T, M::kTerms> wf;
        wf.set(w);
#pragma unroll
        for (int s = 0; s < SL; ++s)
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][s][p] = wf.b_times(xf[s][p], Y[j][s][p]);
        keep_order();
      }
    }
    // D x, the gate, and 8 neighbours of token t to memory
    const float Dh = a.D ? a.D[h] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 16 * j + i16;
      if (t < rows) {
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          float o[8], xv[8];
          M::unpack(M::rows_c(sX + t * LX + 32 * s + 8 * g), xv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r] = fmaf(Dh, xv[r], Y[j][s][0][r]);
            o[4 + r] = fmaf(Dh, xv[4 + r], Y[j][s][1][r]);
          }
          const long col = (long)h * a.headdim + p0 + 32 * s + 8 * g;
          if (a.z) {
            float zv[8];
            Vec8<T>::load(a.z, (t0 + t) * a.z_stride + col, zv);
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] *= zv[r] * sigmoid_f32(zv[r]);
          }
          Vec8<T>::store(a.y, (t0 + t) * (long)a.nheads * a.headdim + col, o);
        }
      }
    }
    wave_sync();  // the next unit's x comes over this one's
  }
}

// Each sequence's segments in order: a segment's end-from-zero is replaced by
// the state the segment starts from.  Grid: quads of state elements x heads'
// slices x sequences.
__global__ void __launch_bounds__(256) scan_combine_kernel(const ScanArgs a) {
  const int elems = kPT * a.dstate;
  const int per = (elems / 4 + 255) / 256;
  const long id = blockIdx.x;
  const int e = ((int)(id % per) * 256 + (int)threadIdx.x) * 4;
  const int v = (int)(id / per % a.vheads), i = (int)(id / per / a.vheads);
  if (e >= elems) return;
  const SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  const int pool = a.init ? scan_slot(a, i) : -1;
  if (pool >= 0 && (!a.has_init || a.has_init[i]))
    S = load_state4(a.init, ((long)pool * a.vheads + v) * elems + e, a.state_bf16);
  const long base = seg_base(a.cu, i, a.seg, a.tokens);
  // eight segments' loads at a time: one after another they would take a
  // memory latency each
  constexpr int U = 8;
  for (int k0 = 0; k0 < segs; k0 += U) {
    f32x4 own[U];
    float d[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k = k0 + q;
      own[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      d[q] = 0.f;
      if (k + 1 < segs) {
        const long at = (base + k) * a.vheads + v;
        own[q] = *reinterpret_cast<const f32x4*>(a.seg_state + at * elems + e);
        d[q] = a.seg_decay[at];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (k0 + q >= segs) break;
      *reinterpret_cast<f32x4*>(a.seg_state + ((base + k0 + q) * a.vheads + v) * elems + e) = S;
      const float w = exp2_f32(d[q]);
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = fmaf(w, S[r], own[q][r]);
    }
  }
}

// Calls of up to this many tokens take one launch, a chain of two chunks at most;
// the other way is three launches.  The lengths are on the device, so the total has
// to do for the worst that it can stand for, one long sequence.  80 heads, dstate
// 128, one launch (the other way in brackets), bf16: 128 tokens 25 us (32), 256
// 41 (39), 512 74 (63); fp32: 42 (49), 75 (64), 148 (101).  1024 bf16 tokens would
// gain in 16 sequences of 64, 42 us (68), and lose in one of 1009 and 15 of one
// token, 192 (96).
constexpr int kShort = 128;

// Tokens of a segment: enough segments to give every one of the 1024 SIMDs two
// waves, but no shorter than four chunks (a segment's state crosses memory
// four times, 16 bytes an element, beside 64 tokens' x and y of 256).
static int scan_seg(const rssm_scan_dims& d) {
  const long vheads = (long)d.nheads * (d.headdim / kPT);
  const long want = (d.tokens * vheads + 2047) / 2048;
  long seg = (want + kQ - 1) / kQ * kQ;
  if (seg < 4 * kQ) seg = 4 * kQ;
  if (seg > 64 * kQ) seg = 64 * kQ;
  return (int)seg;
}

// The workspace, in order; every part a multiple of 16 bytes.
struct FwdLayout {
  size_t dec, chunk_state, seg_state, seg_decay, end;
};
static FwdLayout fwd_layout(const rssm_scan_dims& d) {
  FwdLayout l{};
  if (d.tokens <= kShort) return l;
  const size_t T = d.tokens, n = d.seqs, seg = scan_seg(d), cslots = T / kQ + n, slots = T / seg + n;
  const size_t V = (size_t)d.nheads * (d.headdim / kPT);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  l.dec = take(cslots * d.nheads * kQ * 16);
  l.chunk_state = take(cslots * V * kPT * d.dstate * 4);
  l.seg_state = take(T > seg ? slots * V * kPT * d.dstate * 4 : 0);
  l.seg_decay = take(T > seg ? slots * V * 4 : 0);
  l.end = at;
  return l;
}

enum { kFwdShort, kFwdSegments, kFwdStates, kFwdOut };
template <typename T, int N>
static const void* pick_fwd_n(int which, int headdim) {
  switch (which) {
    case kFwdShort: return reinterpret_cast<const void*>(&scan_short_kernel<T, N>);
    case kFwdSegments: return reinterpret_cast<const void*>(&scan_fwd_states_kernel<T, N, false>);
    case kFwdStates: return reinterpret_cast<const void*>(&scan_fwd_states_kernel<T, N, true>);
    default:
      return headdim == 32 ? reinterpret_cast<const void*>(&scan_fwd_out_kernel<T, N, 32>)
                           : reinterpret_cast<const void*>(&scan_fwd_out_kernel<T, N, 64>);
  }
}
template <typename T>
static const void* pick_fwd(int which, const rssm_scan_dims& d) {
  switch (d.dstate) {
    case 16: return pick_fwd_n<T, 16>(which, d.headdim);
    case 32: return pick_fwd_n<T, 32>(which, d.headdim);
    case 64: return pick_fwd_n<T, 64>(which, d.headdim);
    case 128: return pick_fwd_n<T, 128>(which, d.headdim);
    default: return pick_fwd_n<T, 256>(which, d.headdim);
  }
}

}  // namespace rssm

using namespace rssm;

extern "C" size_t ssu_scan_forward_workspace(const rssm_scan_dims* dims) {
  return scan_check(dims) ? 0 : fwd_layout(*dims).end;
}

extern "C" int ssu_scan_forward(const rssm_scan_dims* dims, const void* x, const void* dt,
                                const float* A, const void* B, const void* C, const float* D,
                                const void* z, const float* dt_bias, const int32_t* cu_seqlens,
                                const void* initial_state, const uint8_t* has_initial,
                                const int32_t* slot_idx, void* final_state, void* y,
                                void* workspace, size_t workspace_bytes, int32_t* status,
                                hipStream_t stream) {
  int rc = scan_check(dims);
  if (rc) return rc;
  const rssm_scan_dims& d = *dims;
  if (d.seqs == 0) return d.tokens == 0 ? RSSM_OK : RSSM_EINVAL;
  if (!A || (d.tokens > 0 && (!x || !dt || !B || !C || !y))) return RSSM_EINVAL;
  if (!cu_seqlens && d.seqs != 1) return RSSM_EINVAL;
  if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(z) || !aligned16(y) ||
      !aligned16(initial_state) || !aligned16(final_state) || !aligned16(workspace))
    return RSSM_EINVAL;
  const size_t need = ssu_scan_forward_workspace(dims);
  if (need && (!workspace || workspace_bytes < need)) return RSSM_EINVAL;
  ScanArgs a{};
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.B = B;
  a.C = C;
  a.D = D;
  a.z = z;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.init = initial_state;
  a.has_init = has_initial;
  a.slot_idx = slot_idx;
  a.final_state = final_state;
  a.y = y;
  a.status = status;
  fill_dims(a, d);
  a.vheads = d.nheads * (d.headdim / kPT);
  a.vpg = a.vheads / d.ngroups;
  const bool f32 = d.io_dtype == RSSM_F32;
  const long most = 1L << 24;  // 2^32 threads of 256
  const auto go = [&](int which, long grid, int threads) {
    const void* fn = f32 ? pick_fwd<float>(which, d) : pick_fwd<bf16>(which, d);
    return launch_kernel(fn, (unsigned)grid, threads, 0, stream, a);
  };
  if (d.tokens <= kShort) {
    a.seg = kShort + kQ;  // every sequence is one segment
    const int waves = scan_waves(f32, d.dstate);
    const long grid = (long)d.seqs * d.ngroups * ((a.vpg + waves - 1) / waves);
    return grid < most ? go(kFwdShort, grid, 64 * waves) : RSSM_ESHAPE;
  }
  const FwdLayout l = fwd_layout(d);
  char* const ws = static_cast<char*>(workspace);
  a.dec = reinterpret_cast<f32x4*>(ws + l.dec);
  a.chunk_state = ws + l.chunk_state;
  a.seg_state = reinterpret_cast<float*>(ws + l.seg_state);
  a.seg_decay = reinterpret_cast<float*>(ws + l.seg_decay);
  a.seg = scan_seg(d);
  const long cslots = scan_slots(d.tokens, d.seqs, kQ);
  // Units of a workgroup of the output launch: up to four a wave, which share
  // the chunk's C.B, but so few that there is a workgroup for every compute unit.
  // 16383 tokens of 80 heads: 16 units 613 us, 8 615, 32 655; 4096: 168 us with each.
  a.upg = d.nheads / d.ngroups * (d.headdim == 32 ? 1 : d.headdim / 64);
  a.upb = 16;
  while (a.upb > 4 && cslots * d.ngroups * ((a.upg + a.upb - 1) / a.upb) < 256) a.upb >>= 1;
  a.hb = (a.upg + a.upb - 1) / a.upb;
  const long dgrid = cslots * ((d.nheads + 3) / 4);
  const long sgrid = scan_slots(d.tokens, d.seqs, a.seg) * d.ngroups * ((a.vpg + 3) / 4);
  const long cgrid = ((long)kPT * d.dstate / 4 + 255) / 256 * a.vheads * d.seqs;
  const long ogrid = cslots * d.ngroups * a.hb;
  if (dgrid >= most || sgrid >= most || cgrid >= most || ogrid >= most) return RSSM_ESHAPE;
  rc = f32 ? launch_decay<float>(a, cslots, stream) : launch_decay<bf16>(a, cslots, stream);
  if (!rc && d.tokens > a.seg) {
    rc = go(kFwdSegments, sgrid, 256);
    if (!rc)
      rc = launch_kernel(reinterpret_cast<const void*>(&scan_combine_kernel), (unsigned)cgrid, 256,
                         0, stream, a);
  }
  if (!rc) rc = go(kFwdStates, sgrid, 256);
  return rc ? rc : go(kFwdOut, ogrid, 256);
}
