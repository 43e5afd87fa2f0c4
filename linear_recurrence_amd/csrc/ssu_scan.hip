// Selective scan over packed sequences, forward (see scan_common.hpp for the
// chunked form).
//
// A wave owns one head's slice of PT rows of the state and keeps it in
// registers as it walks the chunks of a segment; the four waves of a workgroup
// share the group's B and C tiles in LDS.  Sequences longer than a segment take
// two more launches in front: the segments' end states from zero (the state
// part alone), then each sequence's running combination of them, which leaves
// every segment the state it starts from.
#include "scan_common.hpp"

namespace rssm {

struct ScanArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  const int32_t* cu;
  const void* init;
  const uint8_t* has_init;
  const int32_t* slot_idx;
  void* final_state;
  void* y;
  float* seg_state;  // [slots][V][PT][N]
  float* seg_decay;  // [slots][V], log2
  int32_t* status;
  long x_stride, dt_stride, B_stride, C_stride, z_stride;
  int32_t tokens, seqs, nheads, headdim, dstate, ngroups, num_slots, state_bf16, dt_softplus;
  int32_t seg, vheads, vpg, split;
};

// Waves of a workgroup: four, or two where fp32 tiles of dstate 256 would not
// fit four heads' x beside them in 160 KB.
constexpr int scan_waves(bool f32, int n) { return f32 && n == 256 ? 2 : 4; }

__device__ static inline int scan_slot(const ScanArgs& a, int i) {
  const int s = a.slot_idx ? a.slot_idx[i] : i;
  return s >= 0 && s < a.num_slots ? s : -1;
}

__device__ static inline f32x4 load_state4(const void* p, long i, int bf) {
  f32x4 f;
  if (bf) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    f[0] = __uint_as_float(v[0] << 16);
    f[1] = __uint_as_float(v[0] & 0xffff0000u);
    f[2] = __uint_as_float(v[1] << 16);
    f[3] = __uint_as_float(v[1] & 0xffff0000u);
  } else {
    f = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  }
  return f;
}
__device__ static inline void store_state4(void* p, long i, int bf, f32x4 f) {
  if (bf) {
    const u32x2 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) = v;
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f;
  }
}

// OUT: y and the final states; otherwise the segments' end states from zero.
template <typename T, int PT, int N, bool OUT>
__global__ void __launch_bounds__(64 * scan_waves(sizeof(typename Mat<T>::E) == 4, N))
    scan_fwd_kernel(const ScanArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int kScanWaves = scan_waves(sizeof(E) == 4, N);
  constexpr int NP = N < 32 ? 32 : N, LN = NP + M::kPad, LX = PT + M::kPad;
  constexpr int NT = (N + 15) / 16, PTT = PT / 16, KB = NP / 32;
  __shared__ __attribute__((aligned(16))) E sB[kQ * LN];
  __shared__ __attribute__((aligned(16))) E sC[OUT ? kQ * LN : 16];
  __shared__ __attribute__((aligned(16))) E sX[kScanWaves][kQ * LX];
  __shared__ float2 sA[kScanWaves][kQ];
  __shared__ __attribute__((aligned(16))) float sD[kScanWaves][kQ];  // dt
  __shared__ __attribute__((aligned(16))) float sW[kScanWaves][kQ];  // weight of x in the state

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g = lane >> 4;
  const int hb = (a.vpg + kScanWaves - 1) / kScanWaves;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int slot = id / (a.ngroups * hb), rest = id % (a.ngroups * hb);
  const int grp = rest / hb, vl = (rest % hb) * kScanWaves + wave;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
  if (sg.len == 0 && !(OUT && sg.empty)) return;
  if (!OUT && sg.last) return;  // nothing starts from its end
  const bool live = vl < a.vpg;
  const int v = grp * a.vpg + (live ? vl : 0);
  const int slices = a.headdim / PT, h = v / slices, p0 = (v % slices) * PT;
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

  // state tiles S^T: rows n = 16 nt + 4g + r, columns tile_col(pt, i16)
  f32x4 S[NT][PTT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int p = 0; p < PTT; ++p) S[n][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  int pool = -1;
  if constexpr (OUT) {
    if (a.init || a.final_state) pool = scan_slot(a, sg.seq);
    if (threadIdx.x == 0 && rest == 0 && sg.first && a.status) {
      if (sg.bad) atomicOr(a.status, RSSM_ST_BAD_SEQ);
      if ((a.init || a.final_state) && pool < 0) atomicOr(a.status, RSSM_ST_BAD_SLOT);
    }
    const bool from_pool = sg.first && a.init && pool >= 0 && (!a.has_init || a.has_init[sg.seq]);
    if (live && (from_pool || !sg.first)) {
      const void* src = sg.first ? a.init : a.seg_state;
      const int bf = sg.first ? a.state_bf16 : 0;
      const long base = ((long)(sg.first ? pool : slot) * a.vheads + v) * (PT * N);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < PTT; ++p)
          S[n][p] = load_state4(src, base + tile_col(p, i16) * N + 16 * n + 4 * g, bf);
    }
  }

  double total = 0.0;
  for (int c0 = 0; c0 < sg.len; c0 += kQ) {
    const int rows = sg.len - c0 < kQ ? sg.len - c0 : kQ;
    const long t0 = sg.tok + c0;
    __syncthreads();  // the previous chunk's tiles are no longer read
    stage_tile<T, N, NP, 64 * kScanWaves>(
        sB, LN, static_cast<const E*>(a.B) + t0 * a.B_stride + (long)grp * N, a.B_stride, rows,
        threadIdx.x);
    if constexpr (OUT)
      stage_tile<T, N, NP, 64 * kScanWaves>(
          sC, LN, static_cast<const E*>(a.C) + t0 * a.C_stride + (long)grp * N, a.C_stride, rows,
          threadIdx.x);
    stage_tile<T, PT, PT, 64>(sX[wave], LX,
                              static_cast<const E*>(a.x) + t0 * a.x_stride +
                                  (long)h * a.headdim + p0,
                              a.x_stride, live ? rows : 0, lane);
    float d = 0.f;
    if (lane < rows) {
      d = Elt<T>::load1(a.dt, (t0 + lane) * a.dt_stride + h) + bias;
      if (a.dt_softplus) d = softplus_f32(d);
    }
    const double cum = wave_cumsum((double)d * A2, lane);
    const double all = __shfl(cum, 63, 64);
    total += all;
    const float hi = (float)cum;
    sA[wave][lane] = make_float2(hi, (float)(cum - (double)hi));
    sD[wave][lane] = d;
    sW[wave][lane] = d * exp2_f32((float)(all - cum));
    const float decay = exp2_f32((float)all);
    __syncthreads();
    if (!live) continue;

    if constexpr (OUT) {
#pragma unroll 1
      for (int j = 0; j < kQ / 16; ++j) {
        if (16 * j >= rows) break;
        f32x4 Y[PTT];
#pragma unroll
        for (int p = 0; p < PTT; ++p) Y[p] = f32x4{0.f, 0.f, 0.f, 0.f};
        // e^{a_t} S C_t
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const Frag c = M::rows_d(sC + (16 * j + i16) * LN + 32 * kb + 4 * g);
#pragma unroll
          for (int p = 0; p < PTT; ++p) {
            // the state enters y rounded to the io type: y is rounded to it too
            float f[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              f[r] = S[2 * kb][p][r];
              f[4 + r] = 2 * kb + 1 < NT ? S[2 * kb + 1 < NT ? 2 * kb + 1 : 0][p][r] : 0.f;
            }
            Y[p] = M::mma(M::pack(f), c, Y[p]);
          }
        }
        const float2 at = sA[wave][16 * j + i16];
        const float et = exp2_f32(at.x + at.y);
#pragma unroll
        for (int p = 0; p < PTT; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) Y[p][r] *= et;
        // the chunk's own tokens
        Frag ct[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          ct[kb] = M::rows_c(sC + (16 * j + i16) * LN + 32 * kb + 8 * g);
#pragma unroll 1
        for (int sb = 0; 2 * sb <= j; ++sb) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int si = 2 * sb + q;
            f32x4 cb = {0.f, 0.f, 0.f, 0.f};
            if (si <= j) {
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
                cb = M::mma(M::rows_c(sB + (16 * si + i16) * LN + 32 * kb + 8 * g), ct[kb], cb);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int s = 16 * si + 4 * g + r;
              const float m = cb[r] * sD[wave][s] * exp2_f32(gap2(at, sA[wave][s]));
              w[4 * q + r] = s <= 16 * j + i16 ? m : 0.f;
            }
          }
          const Frag wf = M::pack(w);
#pragma unroll
          for (int p = 0; p < PTT; ++p)
            Y[p] = M::mma(M::cols(cols_at<T, true>(sX[wave], LX, 32 * sb, pair_base(p), lane), LX),
                          wf, Y[p]);
        }
        // D x, the gate, and 8 neighbours of token t to memory
        const int t = 16 * j + i16;
        if (t < rows) {
#pragma unroll
          for (int q = 0; q < PTT / 2; ++q) {
            float o[8], xv[8];
            M::unpack(M::rows_c(sX[wave] + t * LX + 32 * q + 8 * g), xv);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              o[r] = fmaf(Dh, xv[r], Y[2 * q][r]);
              o[4 + r] = fmaf(Dh, xv[4 + r], Y[2 * q + 1][r]);
            }
            const long col = (long)h * a.headdim + p0 + 32 * q + 8 * g;
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
    }
    // S' = e^{a_Q} S + sum_t (w_t x_t) B_t
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < PTT; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][p][r] *= decay;
#pragma unroll 1
    for (int kb = 0; kb < kQ / 32; ++kb) {
      if (32 * kb >= rows) break;
      Split<T, M::kTerms> xs[PTT];
      const float* w0 = &sW[wave][32 * kb + 4 * g];
#pragma unroll
      for (int p = 0; p < PTT; ++p) {
        float f[8];
        M::unpack(M::cols(cols_at<T, true>(sX[wave], LX, 32 * kb, pair_base(p), lane), LX), f);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] *= w0[r];
          f[4 + r] *= w0[16 + r];
        }
        xs[p].set(f);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const Frag b = M::cols(cols_at<T, false>(sB, LN, 32 * kb, 16 * n, lane), LN);
#pragma unroll
        for (int p = 0; p < PTT; ++p) S[n][p] = xs[p].b_times(b, S[n][p]);
      }
    }
  }

  if (!live) return;
  if constexpr (OUT) {
    if (sg.last && a.final_state && pool >= 0) {
      const long base = ((long)pool * a.vheads + v) * (PT * N);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < PTT; ++p)
          store_state4(a.final_state, base + tile_col(p, i16) * N + 16 * n + 4 * g, a.state_bf16,
                       S[n][p]);
    }
  } else {
    const long base = ((long)slot * a.vheads + v) * (PT * N);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < PTT; ++p)
        store_state4(a.seg_state, base + tile_col(p, i16) * N + 16 * n + 4 * g, 0, S[n][p]);
    if (lane == 0) a.seg_decay[(long)slot * a.vheads + v] = (float)total;
  }
}

// Each sequence's segments in order: a segment's end-from-zero is replaced by
// the state the segment starts from.  Grid: quads of state elements x heads'
// slices x sequences.
__global__ void __launch_bounds__(256) scan_combine_kernel(const ScanArgs a) {
  const int elems = a.headdim * a.dstate * a.nheads / a.vheads;  // PT * N
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
    if (k) *p = S;
#pragma unroll
    for (int r = 0; r < 4; ++r) S[r] = fmaf(d, S[r], own[r]);
  }
}

static int scan_check(const rssm_scan_dims* d) {
  if (!d) return RSSM_EINVAL;
  if (d->tokens < 0 || d->seqs < 0 || d->nheads < 1 || d->ngroups < 1 ||
      d->nheads % d->ngroups || d->num_slots < 0)
    return RSSM_EINVAL;
  if (!valid_dtype(d->io_dtype) || !valid_dtype(d->state_dtype)) return RSSM_EDTYPE;
  const int P = d->headdim, N = d->dstate;
  if (!(P == 32 || P == 64 || P == 128)) return RSSM_ESHAPE;
  if (!(N == 16 || N == 32 || N == 64 || N == 128 || N == 256)) return RSSM_ESHAPE;
  const long es = d->io_dtype == RSSM_F32 ? 4 : 2;
  const long hp = (long)d->nheads * P, gn = (long)d->ngroups * N;
  const int64_t rows[5] = {d->x_stride, d->z_stride, d->dy_stride, d->B_stride, d->C_stride};
  for (int k = 0; k < 5; ++k)
    if (rows[k] != 0 && (rows[k] < (k < 3 ? hp : gn) || rows[k] * es % 16)) return RSSM_EINVAL;
  if (d->dt_stride != 0 && d->dt_stride < d->nheads) return RSSM_EINVAL;
  return RSSM_OK;
}

// State rows a wave owns.  A wave's tile is at most 64 x 128 (128 registers a
// lane), so dstate 256 takes 32 rows.
static int scan_pt(const rssm_scan_dims& d) {
  return d.headdim == 32 || d.dstate == 256 ? 32 : 64;
}

// Tokens of a segment: enough segments to give every one of the 1024 SIMDs two
// waves, but no shorter than four chunks (a segment's state crosses memory
// four times, 16 bytes an element, beside 64 tokens' x and y of 256).
static int scan_seg(const rssm_scan_dims& d) {
  const long vheads = (long)d.nheads * (d.headdim / scan_pt(d));
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
  return (size_t)scan_slots(d.tokens, d.seqs, scan_seg(d)) * d.nheads * (d.headdim / scan_pt(d));
}

template <typename T, bool OUT>
static const void* pick_fwd(int pt, int n) {
#define RSSM_SCAN_FWD(P, N) \
  if (pt == P && n == N) return reinterpret_cast<const void*>(&scan_fwd_kernel<T, P, N, OUT>)
  RSSM_SCAN_FWD(32, 16);
  RSSM_SCAN_FWD(32, 32);
  RSSM_SCAN_FWD(32, 64);
  RSSM_SCAN_FWD(32, 128);
  RSSM_SCAN_FWD(32, 256);
  RSSM_SCAN_FWD(64, 16);
  RSSM_SCAN_FWD(64, 32);
  RSSM_SCAN_FWD(64, 64);
  RSSM_SCAN_FWD(64, 128);
  return nullptr;
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
  const int pt = scan_pt(d);
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
  a.x_stride = d.x_stride ? d.x_stride : (long)d.nheads * d.headdim;
  a.dt_stride = d.dt_stride ? d.dt_stride : d.nheads;
  a.B_stride = d.B_stride ? d.B_stride : (long)d.ngroups * d.dstate;
  a.C_stride = d.C_stride ? d.C_stride : (long)d.ngroups * d.dstate;
  a.z_stride = d.z_stride ? d.z_stride : (long)d.nheads * d.headdim;
  a.tokens = d.tokens;
  a.seqs = d.seqs;
  a.nheads = d.nheads;
  a.headdim = d.headdim;
  a.dstate = d.dstate;
  a.ngroups = d.ngroups;
  a.num_slots = d.num_slots;
  a.state_bf16 = d.state_dtype == RSSM_BF16;
  a.dt_softplus = d.dt_softplus;
  a.seg = scan_seg(d);
  a.vheads = d.nheads * (d.headdim / pt);
  a.vpg = a.vheads / d.ngroups;
  const int waves = scan_waves(d.io_dtype == RSSM_F32, d.dstate);
  const long hb = (a.vpg + waves - 1) / waves;
  const long grid = scan_slots(d.tokens, d.seqs, a.seg) * d.ngroups * hb;
  const long elems = (long)pt * d.dstate;
  const long cgrid = (elems / 4 + 255) / 256 * a.vheads * d.seqs;
  if (grid > 0x7fffffffL || cgrid > 0x7fffffffL) return RSSM_ESHAPE;
  const bool f32 = d.io_dtype == RSSM_F32;
  if (need) {
    const void* fn =
        f32 ? pick_fwd<float, false>(pt, d.dstate) : pick_fwd<bf16, false>(pt, d.dstate);
    rc = launch_kernel(fn, (unsigned)grid, 64 * waves, 0, stream, a);
    if (rc) return rc;
    rc = launch_kernel(reinterpret_cast<const void*>(&scan_combine_kernel), (unsigned)cgrid, 256,
                       0, stream, a);
    if (rc) return rc;
  }
  const void* fn = f32 ? pick_fwd<float, true>(pt, d.dstate) : pick_fwd<bf16, true>(pt, d.dstate);
  return launch_kernel(fn, (unsigned)grid, 64 * waves, 0, stream, a);
}
