// Selective scan over packed sequences, forward (see scan_common.hpp for the
// chunked form).
//
// A wave owns 32 rows of one head's state and keeps it in
// registers as it walks the chunks of a segment; the four waves of a workgroup
// share the group's B and C tiles in LDS.  Sequences longer than a segment take
// two more launches in front: the segments' end states from zero (the state
// part alone), then each sequence's running combination of them, which leaves
// every segment the state it starts from.
#include "scan_common.hpp"

namespace rssm {

// Waves of a workgroup: four, or two where fp32 tiles of dstate 256 would not
// fit four heads' x beside them in 160 KB.
constexpr int scan_waves(bool f32, int n) { return f32 && n == 256 ? 2 : 4; }

// OUT: y and the final states; otherwise the segments' end states from zero.
// Two workgroups a compute unit: 256 registers a lane.
template <typename T, int N, bool OUT>
__global__ void __launch_bounds__(64 * scan_waves(sizeof(typename Mat<T>::E) == 4, N),
                                  sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    scan_fwd_kernel(const ScanArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int W = scan_waves(sizeof(E) == 4, N), TH = 64 * W;
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = kPT + M::kPad;
  constexpr int NT = N / 16, KB = NP / 32;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sC[OUT ? kQ * LN : 16];
  __shared__ __attribute__((aligned(16))) E sX[W][kQ * LX];
  __shared__ f32x4 sCB[OUT ? 10 : 1][64];
  __shared__ float2 sA[W][kQ];
  __shared__ __attribute__((aligned(16))) float sD[W][kQ];  // dt
  __shared__ __attribute__((aligned(16))) float sW[W][kQ];  // weight of x in the state

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g = lane >> 4;
  const int hb = (a.vpg + W - 1) / W;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * W + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  if (sg.len == 0 && !(OUT && sg.empty)) return;
  if (!OUT && sg.last) return;  // nothing starts from its end
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / kPT, h = v / slices, p0 = (v % slices) * kPT;
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

  // state tiles S^T: rows n = 16 nt + 4g + r, columns tile_col(p, i16)
  f32x4 S[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  int pool = -1;
  if constexpr (OUT) {
    if (a.init || a.final_state) pool = scan_slot(a, sg.seq);
    if (threadIdx.x == 0 && rest == 0 && sg.first && a.status) {
      if (sg.bad) atomicOr(a.status, RSSM_ST_BAD_SEQ);
      if ((a.init || a.final_state) && pool < 0) atomicOr(a.status, RSSM_ST_BAD_SLOT);
    }
    // The pool is read here only by a sequence of one segment, whose wave also
    // writes it: a longer one's first segment takes the copy that the combining
    // launch left, since its last segment may already have stored the final
    // state over the initial one.
    const bool whole = sg.first && sg.last;
    const bool from_pool = whole && a.init && pool >= 0 && (!a.has_init || a.has_init[sg.seq]);
    if (live && (from_pool || !whole)) {
      const void* src = whole ? a.init : a.seg_state;
      const int bf = whole ? a.state_bf16 : 0;
      const long base = ((long)(whole ? pool : slot) * a.vheads + v) * (kPT * N);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          S[n][p] = load_state4(src, base + tile_col(p, i16) * N + 16 * n + 4 * g, bf);
    }
  }

  double total = 0.0;
  for (int c0 = 0; c0 < sg.len; c0 += kQ) {
    const int rows = sg.len - c0 < kQ ? sg.len - c0 : kQ;
    const long t0 = sg.tok + c0;
    __syncthreads();  // the previous chunk's tiles are no longer read
    stage_tile<T, N, NP, TH>(sB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N,
                             a.B_stride, rows, threadIdx.x);
    if constexpr (OUT)
      stage_tile<T, N, NP, TH>(sC, LN,
                               static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N,
                               a.C_stride, rows, threadIdx.x);
    stage_tile<T, kPT, kPT, 64>(sX[wave], LX,
                                static_cast<const E*>(a.x) + t0 * a.x_stride +
                                    (long)h * a.headdim + p0,
                                a.x_stride, live ? rows : 0, lane);
    const ChunkDt q = chunk_dt<T>(a, h, bias, A2, t0, rows, lane);
    total += q.all;
    {
      const float hi = (float)q.cum;
      sA[wave][lane] = make_float2(hi, (float)(q.cum - (double)hi));
      sD[wave][lane] = q.dt;
      sW[wave][lane] = q.dt * exp2_f32((float)(q.all - q.cum));
    }
    const float decay = exp2_f32((float)q.all);
    __syncthreads();

    if constexpr (OUT) {
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
      // e^{a_t} S C_t.  The state enters y rounded to the io type: y is
      // rounded to it too, and D x usually outweighs it
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Frag sf[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float f[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            f[r] = S[2 * kb][p][r];
            f[4 + r] = 2 * kb + 1 < NT ? S[2 * kb + 1 < NT ? 2 * kb + 1 : 0][p][r] : 0.f;
          }
          sf[p] = M::pack(f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Frag c = M::rows_d(sC + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][p] = M::mma(sf[p], c, Y[j][p]);
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
          const Frag wf = M::pack(w);
#pragma unroll
          for (int p = 0; p < 2; ++p) Y[j][p] = M::mma(xf[p], wf, Y[j][p]);
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

  if (!live) return;
  if constexpr (OUT) {
    if (sg.last && a.final_state && pool >= 0) {
      const long base = ((long)pool * a.vheads + v) * (kPT * N);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          store_state4(a.final_state, base + tile_col(p, i16) * N + 16 * n + 4 * g, a.state_bf16,
                       S[n][p]);
    }
  } else {
    const long base = ((long)slot * a.vheads + v) * (kPT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        store_state4(a.seg_state, base + tile_col(p, i16) * N + 16 * n + 4 * g, 0, S[n][p]);
    if (lane == 0) a.seg_decay[(long)slot * a.vheads + v] = (float)total;
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
  for (int k = 0; k < segs; ++k) {
    const long at = (base + k) * a.vheads + v;
    f32x4* const p = reinterpret_cast<f32x4*>(a.seg_state + at * elems + e);
    f32x4 own = {0.f, 0.f, 0.f, 0.f};
    float d = 0.f;
    if (k + 1 < segs) {
      own = *p;
      d = exp2_f32(a.seg_decay[at]);
    }
    *p = S;
#pragma unroll
    for (int r = 0; r < 4; ++r) S[r] = fmaf(d, S[r], own[r]);
  }
}

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

static size_t scan_states(const rssm_scan_dims& d) {
  return (size_t)scan_slots(d.tokens, d.seqs, scan_seg(d)) * d.nheads * d.headdim * d.dstate;
}
static size_t scan_decays(const rssm_scan_dims& d) {
  return (size_t)scan_slots(d.tokens, d.seqs, scan_seg(d)) * d.nheads * (d.headdim / kPT);
}

template <typename T, bool OUT>
static const void* pick_fwd(int n) {
#define RSSM_SCAN_FWD(N) if (n == N) return reinterpret_cast<const void*>(&scan_fwd_kernel<T, N, OUT>)
  RSSM_SCAN_FWD(16);
  RSSM_SCAN_FWD(32);
  RSSM_SCAN_FWD(64);
  RSSM_SCAN_FWD(128);
  RSSM_SCAN_FWD(256);
  return nullptr;
}

// The segments' end states from zero, then each segment's starting state (the
// backward pass recomputes the states from them).
int scan_segment_states(const ScanArgs& a, const rssm_scan_dims& d, hipStream_t stream) {
  const int waves = scan_waves(d.io_dtype == RSSM_F32, d.dstate);
  const long hb = (a.vpg + waves - 1) / waves;
  const long grid = scan_slots(d.tokens, d.seqs, a.seg) * d.ngroups * hb;
  const long cgrid = ((long)kPT * d.dstate / 4 + 255) / 256 * a.vheads * d.seqs;
  if (grid > 0x7fffffffL || cgrid > 0x7fffffffL) return RSSM_ESHAPE;
  const void* fn = d.io_dtype == RSSM_F32 ? pick_fwd<float, false>(d.dstate)
                                          : pick_fwd<bf16, false>(d.dstate);
  const int rc = launch_kernel(fn, (unsigned)grid, 64 * waves, 0, stream, a);
  if (rc) return rc;
  return launch_kernel(reinterpret_cast<const void*>(&scan_combine_kernel), (unsigned)cgrid, 256,
                       0, stream, a);
}

}  // namespace rssm

using namespace rssm;

extern "C" size_t ssu_scan_forward_workspace(const rssm_scan_dims* dims) {
  if (scan_check(dims) || dims->tokens <= scan_seg(*dims)) return 0;
  return sizeof(float) * (scan_states(*dims) + scan_decays(*dims));
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
  a.seg_state = static_cast<float*>(workspace);
  a.seg_decay = need ? a.seg_state + scan_states(d) : nullptr;
  a.status = status;
  fill_dims(a, d);
  a.seg = scan_seg(d);
  a.vheads = d.nheads * (d.headdim / kPT);
  a.vpg = a.vheads / d.ngroups;
  const int waves = scan_waves(d.io_dtype == RSSM_F32, d.dstate);
  const long hb = (a.vpg + waves - 1) / waves;
  const long grid = scan_slots(d.tokens, d.seqs, a.seg) * d.ngroups * hb;
  if (grid > 0x7fffffffL) return RSSM_ESHAPE;
  const bool f32 = d.io_dtype == RSSM_F32;
  if (need) {
    rc = scan_segment_states(a, d, stream);
    if (rc) return rc;
  }
  const void* fn = f32 ? pick_fwd<float, true>(d.dstate) : pick_fwd<bf16, true>(d.dstate);
  return launch_kernel(fn, (unsigned)grid, 64 * waves, 0, stream, a);
}
