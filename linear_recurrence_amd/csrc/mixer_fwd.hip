// Linear attention and the gated delta rule over packed sequences, forward (the
// chunked form: mixer_common.hpp).
//
// The delta rule's T of every chunk is independent of the state and comes from a
// launch in front (mix_inverse_kernel).  Then a workgroup walks the chunks of one
// sequence and 64 columns of one value head's state, a wave 16 of them, with the
// state in registers; the next chunk's tiles are on their way while one is worked on.
//
// The states, X and D are fp32 values and enter the products that make states as
// three bf16 terms (24 bits).  What only the output reads goes in as two terms: the
// decayed q.k, D and S in o's products, 2^-17 of each term where o, rounded to bf16,
// is off by 2^-9 of itself.  fp32 inputs stay fp32 everywhere.
#include "mixer_states.hpp"

namespace rssm {

template <typename T>
constexpr int out_terms() { return Mat<T>::kTerms > 2 ? 2 : Mat<T>::kTerms; }

template <typename T, int TA, int TB>
__device__ static inline Split<T, TB> cut(const Split<T, TA>& s) {  // the leading terms
  Split<T, TB> r;
#pragma unroll
  for (int k = 0; k < TB; ++k) r.t[k] = s.t[k];
  return r;
}

template <typename T, int K, bool DELTA>
__global__ void __launch_bounds__(256, sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    mix_forward_kernel(const MixArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  constexpr int TS = M::kTerms, TO = out_terms<T>();
  constexpr int LK = K + M::kPad, LV = 64 + M::kPad, KT = K / 16, KB = K / 32;
  constexpr int TF = 6 * TS * 64 * sizeof(Frag) / 16;  // 16-byte pieces of T
  constexpr int QT = DELTA ? (TF + 255) / 256 : 1;
  __shared__ __attribute__((aligned(16))) E sK[kQ * LK];
  __shared__ __attribute__((aligned(16))) E sQ[kQ * LK];
  __shared__ __attribute__((aligned(16))) E sV[kQ * LV];
  __shared__ __attribute__((aligned(16))) u32x4 sT[DELTA ? TF : 1];
  __shared__ __attribute__((aligned(16))) u32x4 sP[6 * TO * 64 * sizeof(Frag) / 16];
  __shared__ ChunkGates sg;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const MixUnit un = mix_unit(a, blockIdx.x, a.vpk * a.slices);
  if (blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if (!un.live) return;
  const int hv = un.hk * a.vpk + un.rest / a.slices, v0 = (un.rest % a.slices) * 64;
  const Segment sp = find_segment(a.cu, a.seqs, a.tokens, a.seg, un.slot);
  if (sp.len == 0 && !sp.empty) return;
  const int pool = a.init || a.final_state ? mix_slot(a, sp.seq) : -1;
  if (tid == 0 && sp.first && un.rest == 0 && un.hk == 0 && a.status && (a.init || a.final_state) && pool < 0)
    atomicOr(a.status, RSSM_ST_BAD_SLOT);
  // S: rows k = 16 kt + 4g + r, column v0 + 16 wave + i16
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto place = [&](long n) {
    return ((n * a.v_heads + hv) * a.dv + v0 + 16 * wave + (lane & 15)) * K + 4 * (lane >> 4);
  };
  // The pool is read here only by a sequence of one segment, whose wave also writes it:
  // a longer one's first segment takes the copy that the combining launch left, since
  // its last segment may already have stored the final state over the initial one.
  const bool whole = sp.first && sp.last;
  if (!whole || (a.init && pool >= 0 && (!a.has_init || a.has_init[sp.seq]))) {
    const float* p = whole ? a.init + place(pool) : a.seg_state + place(un.slot);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(p + 16 * kt);
  }
  const long cbase = seg_base(a.cu, sp.seq, kQ, a.tokens) + (long)sp.k * (a.seg / kQ);
  const int chunks = (sp.len + kQ - 1) / kQ;
  const int i16 = lane & 15, g = lane >> 4;
  TileLoad<T, K, 256> rk, rq;
  TileLoad<T, 64, 256> rv;
  GateLoad rg;
  u32x4 rt[QT];
  const u32x4* tsrc = static_cast<const u32x4*>(a.tinv) + (cbase * a.v_heads + hv) * TF + tid;
  rk.start(static_cast<const E*>(a.k) + sp.tok * a.k_stride + (long)un.hk * K, a.k_stride, tid);
  rq.start(static_cast<const E*>(a.q) + sp.tok * a.q_stride + (long)un.hk * K, a.q_stride, tid);
  rv.start(static_cast<const E*>(a.v) + sp.tok * a.v_stride + (long)hv * a.dv + v0, a.v_stride, tid);
  rg.start(a, sp.tok, hv, lane, DELTA);
  E* out = static_cast<E*>(a.o) + ((long)(sp.tok + i16) * a.v_heads + hv) * a.dv + v0 + 16 * wave + 4 * g;
  const long orow = (long)a.v_heads * a.dv;
  const auto fetch = [&](int c) {
    const int rows = sp.len - c * kQ < kQ ? sp.len - c * kQ : kQ;
    rk.fetch(rows, tid);
    rq.fetch(rows, tid);
    rv.fetch(rows, tid);
    rg.fetch(rows, lane);
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
        if (TF % 256 == 0 || i * 256 + tid < TF) rt[i] = tsrc[i * 256];
    }
    rk.step(1);
    rq.step(1);
    rv.step(1);
    rg.step(1);
    tsrc += (long)a.v_heads * TF;
  };
  if (chunks) fetch(0);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const int rows = sp.len - c * kQ < kQ ? sp.len - c * kQ : kQ;
    __syncthreads();  // the previous chunk's tiles are no longer read
    rk.put(sK, LK, tid);
    rq.put(sQ, LK, tid);
    rv.put(sV, LV, tid);
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
        if (TF % 256 == 0 || i * 256 + tid < TF) sT[i * 256 + tid] = rt[i];
    }
    if (wave == 3) sg.set(rg.rg, rg.rb, lane);
    if (c + 1 < chunks) fetch(c + 1);
    __syncthreads();
    f32x4 R[4], O[4];  // K S, rows t; (Q S)^T, columns t
    f32x4 P[3];        // this wave's tiles of k_j.q_i, rows j
#pragma unroll
    for (int it = 0; it < 4; ++it) R[it] = O[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    P[0] = P[1] = P[2] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      float f[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = S[2 * b][r];
        f[4 + r] = S[2 * b + 1][r];
      }
      Split<T, DELTA ? TS : TO> sf;
      sf.set(f);
      const auto so = cut<T, DELTA ? TS : TO, TO>(sf);
      Frag kf[4], qf[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        kf[it] = M::rows_d(sK + (16 * it + i16) * LK + 32 * b + 4 * g);
        qf[it] = M::rows_d(sQ + (16 * it + i16) * LK + 32 * b + 4 * g);
      }
      if constexpr (DELTA) {
#pragma unroll
        for (int k = TS - 1; k >= 0; --k)
#pragma unroll
          for (int it = 0; it < 4; ++it) R[it] = M::mma(kf[it], sf.t[k], R[it]);
      }
#pragma unroll
      for (int k = TO - 1; k >= 0; --k)
#pragma unroll
        for (int it = 0; it < 4; ++it) O[it] = M::mma(so.t[k], qf[it], O[it]);
      if (wave == 0) {
        P[0] = M::mma(kf[0], qf[3], P[0]);
        P[1] = M::mma(kf[1], qf[3], P[1]);
        P[2] = M::mma(kf[0], qf[0], P[2]);
      } else if (wave == 1) {
        P[0] = M::mma(kf[2], qf[3], P[0]);
        P[1] = M::mma(kf[3], qf[3], P[1]);
      } else if (wave == 2) {
        P[0] = M::mma(kf[0], qf[2], P[0]);
        P[1] = M::mma(kf[1], qf[2], P[1]);
      } else {
        P[0] = M::mma(kf[0], qf[1], P[0]);
        P[1] = M::mma(kf[1], qf[1], P[1]);
        P[2] = M::mma(kf[2], qf[2], P[2]);
      }
    }
    {
      // scale e^{G_i-G_j} q_i.k_j of the lower triangle as fragments: (3, 0) and (0, 0);
      // (3, 1); (2, 0); (1, 0) and (2, 1)
      const int it = wave < 2 ? 3 : (wave == 2 ? 2 : 1), kb = wave == 1, ie = wave ? 2 : 0, ke = wave != 0;
      const auto weigh = [&](int i, int j, const f32x4& p, float* f) {  // of one tile
        const float2 gi = sg.G[16 * i + i16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = a.scale * exp2_f32(gap2(gi, sg.G[16 * j + 4 * g + r])) * p[r];
          f[r] = j < i || 4 * g + r <= i16 ? w : 0.f;
        }
      };
      float f[8];
      Split<T, TO> s;
      weigh(it, 2 * kb, P[0], f);
      weigh(it, 2 * kb + 1, P[1], f + 4);
      s.set(f);
      put_split<T, TO>(sP, low_frag(it, kb), s, lane);
      if (wave == 0 || wave == 3) {
        weigh(ie, 2 * ke, P[2], f);
        f[4] = f[5] = f[6] = f[7] = 0.f;
        s.set(f);
        put_split<T, TO>(sP, low_frag(ie, ke), s, lane);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const float e = a.scale * sg.eg[16 * it + i16];
#pragma unroll
      for (int r = 0; r < 4; ++r) O[it][r] *= e;
    }
    float d[2][8];  // D, token 32 kb + (4g + r, 16 + 4g + r), this lane's column
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      M::unpack(M::cols(cols_at<T, false>(sV, LV, 32 * kb, 16 * wave, lane), LV), d[kb]);
      if (DELTA) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 e = *reinterpret_cast<const f32x4*>(&sg.eg[32 * kb + 16 * h + 4 * g]);
          const f32x4 b = *reinterpret_cast<const f32x4*>(&sg.beta[32 * kb + 16 * h + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) d[kb][4 * h + r] = b[r] * fmaf(-e[r], R[2 * kb + h][r], d[kb][4 * h + r]);
        }
      }
    }
    if (DELTA) {
      f32x4 acc[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Split<T, TS> xf;
        xf.set(d[kb]);
#pragma unroll
        for (int it = 2 * kb; it < 4; ++it)
          acc[it] = mma_split<T, TS, TS>(split_at<T, TS>(sT, low_frag(it, kb), lane), xf, acc[it]);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) d[it >> 1][4 * (it & 1) + r] = acc[it][r];
    }
    __syncthreads();  // sP
    // o^T += D^T P^T, and S' = e^{G_Q} S + K^T (e^{G_Q - G} D)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      Split<T, DELTA ? TO : 1> df;
      df.set(d[kb]);
#pragma unroll
      for (int it = 2 * kb; it < 4; ++it)
        O[it] = mma_split<T, DELTA ? TO : 1, TO>(df, split_at<T, TO>(sP, low_frag(it, kb), lane), O[it]);
    }
    const float all = sg.all;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[kt][r] *= all;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (32 * kb >= rows) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 e = *reinterpret_cast<const f32x4*>(&sg.et[32 * kb + 16 * h + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) d[kb][4 * h + r] *= e[r];
      }
      Split<T, TS> wf;
      wf.set(d[kb]);
#pragma unroll
      for (int k4 = 0; k4 < KT; k4 += 4) {
        Frag kf[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) kf[q] = M::cols(cols_at<T, false>(sK, LK, 32 * kb, 16 * (k4 + q), lane), LK);
#pragma unroll
        for (int k = TS - 1; k >= 0; --k)
#pragma unroll
          for (int q = 0; q < 4; ++q) S[k4 + q] = M::mma(kf[q], wf.t[k], S[k4 + q]);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const float f[4] = {O[it][0], O[it][1], O[it][2], O[it][3]};
      if (16 * it + i16 < rows) *reinterpret_cast<typename M::Four*>(out + 16 * it * orow) = M::pack4(f);
    }
    out += kQ * orow;
  }
  if (sp.last && a.final_state && pool >= 0) {
    float* p = a.final_state + place(pool);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + 16 * kt) = S[kt];
  }
}

struct FwdLayout {
  size_t tinv, end;
  SegLayout seg;
};
static FwdLayout fwd_layout(const rssm_mixer_dims& d, bool delta) {
  FwdLayout l{};
  MixTake take;
  const size_t units = (size_t)scan_slots(d.tokens, d.seqs, kQ) * d.v_heads;
  l.tinv = take(delta ? units * mix_inverse_bytes(d.io_dtype == RSSM_F32, false) : 0);
  l.seg = seg_layout(d, delta, false, take);
  l.end = take.at;
  return l;
}
static size_t mix_forward_bytes(const rssm_mixer_dims* dims, bool delta) {
  return mix_check(dims, delta) || dims->tokens == 0 ? 0 : fwd_layout(*dims, delta).end;
}

template <typename T, bool DELTA>
static const void* pick_forward(int dk) {
  return dk == 64 ? reinterpret_cast<const void*>(&mix_forward_kernel<T, 64, DELTA>)
                  : reinterpret_cast<const void*>(&mix_forward_kernel<T, 128, DELTA>);
}

static int mix_forward(const rssm_mixer_dims* dims, bool delta, const void* q, const void* k, const void* v,
                       const float* g, const float* beta, const int32_t* cu_seqlens,
                       const float* initial_state, const uint8_t* has_initial, const int32_t* slot_idx,
                       float* final_state, void* o, void* workspace, size_t workspace_bytes,
                       int32_t* status, hipStream_t stream) {
  int rc = mix_check(dims, delta);
  if (rc) return rc;
  const rssm_mixer_dims& d = *dims;
  if (d.seqs == 0) return d.tokens == 0 ? RSSM_OK : RSSM_EINVAL;
  if (!cu_seqlens && d.seqs != 1) return RSSM_EINVAL;
  if (d.tokens > 0 && (!q || !k || !v || !o || (d.decay && !g) || (delta && !beta))) return RSSM_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(initial_state) ||
      !aligned16(final_state) || !aligned16(workspace))
    return RSSM_EINVAL;
  const size_t need = mix_forward_bytes(dims, delta);
  if (need && (!workspace || workspace_bytes < need)) return RSSM_EINVAL;
  MixArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.cu = cu_seqlens;
  a.init = initial_state;
  a.has_init = has_initial;
  a.slot_idx = slot_idx;
  a.final_state = final_state;
  a.o = o;
  a.status = status;
  mix_fill(a, d);
  const bool f32 = d.io_dtype == RSSM_F32;
  const FwdLayout l = fwd_layout(d, delta);
  a.tinv = static_cast<char*>(workspace) + l.tinv;
  seg_fill(a, d, l.seg, workspace);
  a.seg_grad = nullptr;  // no gradients to combine
  const long cslots = scan_slots(d.tokens, d.seqs, kQ);
  const long grid = mix_grid(a.slots, d.k_heads, (long)a.vpk * a.slices);
  if (!segments_fit(a, d.dk) || (delta && !grid_fits(cslots * ((d.v_heads + 3) / 4), 256))) return RSSM_ESHAPE;
  if (delta && d.tokens > 0) {
    rc = f32 ? launch_inverse<float, false>(a, d.dk, cslots, stream)
             : launch_inverse<bf16, false>(a, d.dk, cslots, stream);
    if (rc) return rc;
  }
  if (d.tokens > a.seg) {
    MixBwdArgs b{};
    b.m = a;
    rc = f32 ? (delta ? launch_segments<float, true, false>(b, d.dk, stream)
                      : launch_segments<float, false, false>(b, d.dk, stream))
             : (delta ? launch_segments<bf16, true, false>(b, d.dk, stream)
                      : launch_segments<bf16, false, false>(b, d.dk, stream));
    if (rc) return rc;
  }
  const void* fn = f32 ? (delta ? pick_forward<float, true>(d.dk) : pick_forward<float, false>(d.dk))
                       : (delta ? pick_forward<bf16, true>(d.dk) : pick_forward<bf16, false>(d.dk));
  return launch_kernel(fn, (unsigned)grid, 256, 0, stream, a);
}

}  // namespace rssm

using namespace rssm;

extern "C" size_t linear_attention_forward_workspace(const rssm_mixer_dims* dims) {
  return mix_forward_bytes(dims, false);
}

extern "C" int linear_attention_forward(const rssm_mixer_dims* dims, const void* q, const void* k,
                                        const void* v, const float* log_decay, const int32_t* cu_seqlens,
                                        const float* initial_state, const uint8_t* has_initial,
                                        const int32_t* slot_idx, float* final_state, void* o,
                                        void* workspace, size_t workspace_bytes, int32_t* status,
                                        hipStream_t stream) {
  return mix_forward(dims, false, q, k, v, log_decay, nullptr, cu_seqlens, initial_state, has_initial,
                     slot_idx, final_state, o, workspace, workspace_bytes, status, stream);
}

extern "C" size_t gdn_scan_forward_workspace(const rssm_mixer_dims* dims) {
  return mix_forward_bytes(dims, true);
}

extern "C" int gdn_scan_forward(const rssm_mixer_dims* dims, const void* q, const void* k, const void* v,
                                const float* log_g, const float* beta, const int32_t* cu_seqlens,
                                const float* initial_state, const uint8_t* has_initial,
                                const int32_t* slot_idx, float* final_state, void* o, void* workspace,
                                size_t workspace_bytes, int32_t* status, hipStream_t stream) {
  return mix_forward(dims, true, q, k, v, log_g, beta, cu_seqlens, initial_state, has_initial, slot_idx,
                     final_state, o, workspace, workspace_bytes, status, stream);
}
