// The recurrences over the chunks without their outputs: states and their gradients for
// the backward pass, and the segments of long sequences for both passes (the chunked
// form: mixer_common.hpp; the backward formulas: mixer_bwd.hip).
#pragma once

#include "mixer_common.hpp"

namespace rssm {

struct MixBwdArgs {
  MixArgs m;
  const void* dout;
  const float* dfinal;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dbeta;
  float* dinit;
  float* state;  // [chunk slots][v_heads][V][K]: before the chunk
  float* grad;   // dS', the same
  float* D;      // [chunk slots][v_heads][64][V]
  float* dX;     // the same
  float* part;   // [chunk slots][v_heads]: dg summed over the chunk
  long do_stride, cslots;
  int32_t dir_blocks;  // blocks of one direction
  int32_t elems;       // of a state
};

template <typename T, int K, bool DELTA, bool BOTH>
struct StatesLds {
  typedef typename Mat<T>::E E;
  static constexpr int kFrag = sizeof(typename Mat<T>::Frag), TS = Mat<T>::kTerms;
  static constexpr int LK = K + Mat<T>::kPad;
  static constexpr int TF = 6 * TS * 64 * kFrag / 16;  // 16-byte pieces of T or its transpose
  __attribute__((aligned(16))) E k[kQ * LK];
  __attribute__((aligned(16))) E v[kQ * 64];  // V forward, dO backward
  __attribute__((aligned(16))) u32x4 t[DELTA ? TF : 1];
  __attribute__((aligned(16))) E q[BOTH ? kQ * LK : 1];
  __attribute__((aligned(16))) u32x4 p[BOTH ? TF : 1];
  ChunkGates g;
};

// One of the two recurrences over the chunks of a segment, a workgroup for 64 columns of
// one value head's state (mix_forward_kernel without the outputs).  Blocks: forward;
// BOTH: backward, last chunk first; the delta rule's transition.
// STORE: from the segment's start, leaving the states before all chunks, D and dX (or
// dV) and the gradient of the initial state.  Otherwise from zero, leaving what the
// segment adds and, as columns that start from the identity without V, the matrix that
// its starting state is multiplied by, as first operands: rows of it and (BOTH) of its
// transpose, which gradients go through.
template <typename T, int K, bool DELTA, bool STORE, bool BOTH>
static __global__ void __launch_bounds__(256, sizeof(typename Mat<T>::E) == 4 ? 1 : 2)
    mix_states_kernel(const MixBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  typedef StatesLds<T, K, DELTA, BOTH> L;
  constexpr int TS = M::kTerms, LK = L::LK, KT = K / 16, KB = K / 32, TF = L::TF;
  constexpr int QT = DELTA ? (TF + 255) / 256 : 1;
  __shared__ L s;
  const MixArgs& a = b.m;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool back = BOTH && (int)blockIdx.x >= b.dir_blocks && (int)blockIdx.x < 2 * b.dir_blocks;
  const bool trans = !STORE && DELTA && (int)blockIdx.x >= (BOTH ? 2 : 1) * b.dir_blocks;
  const int slices = trans ? K / 64 : a.slices;
  const MixUnit un = mix_unit(a, blockIdx.x - (trans ? (BOTH ? 2 : 1) : back) * b.dir_blocks, a.vpk * slices);
  if (STORE && blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if (!un.live) return;
  const int hv = un.hk * a.vpk + un.rest / slices, v0 = (un.rest % slices) * 64;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, un.slot);
  if (sg.len == 0 && !(STORE && sg.empty)) return;
  const bool whole = sg.first && sg.last;
  // what no other segment starts from (the matrix of a last one: only gradients)
  if (!STORE && (whole || (trans ? sg.last && !BOTH : (back ? sg.first : sg.last)))) return;
  const int pool = STORE && a.init ? mix_slot(a, sg.seq) : -1;
  if (STORE && tid == 0 && !back && sg.first && un.rest == 0 && un.hk == 0 && a.status && a.init && pool < 0)
    atomicOr(a.status, RSSM_ST_BAD_SLOT);
  const bool has = pool >= 0 && (!a.has_init || a.has_init[sg.seq]);
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this lane's first element in state number n
  const auto place = [&](long n) {
    return ((n * a.v_heads + hv) * a.dv + v0 + 16 * wave + (lane & 15)) * K + 4 * (lane >> 4);
  };
  if (STORE) {
    const float* src = back ? b.dfinal : (has ? a.init : nullptr);
    if (!whole) src = back ? a.seg_grad : a.seg_state;
    if (src) {
      src += place(!whole ? un.slot : (back ? sg.seq : pool));
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(src + 16 * kt);
    }
  } else if (trans) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[kt][r] = 16 * kt + 4 * (lane >> 4) + r == v0 + 16 * wave + (lane & 15) ? 1.f : 0.f;
  }
  float total = 1.f;
  const long vstride = back ? b.do_stride : a.v_stride;
  const long cbase = seg_base(a.cu, sg.seq, kQ, a.tokens) + (long)sg.k * (a.seg / kQ);
  const int chunks = (sg.len + kQ - 1) / kQ, way = back ? -1 : 1;
  const int i16 = lane & 15, g = lane >> 4;
  const long first = chunks && back ? chunks - 1 : 0, tok = sg.tok + first * kQ;
  TileLoad<T, K, 256> rk, rq;
  TileLoad<T, 64, 256> rv;
  GateLoad rg;
  u32x4 rt[QT];
  const u32x4* tsrc = static_cast<const u32x4*>(a.tinv) +
      (((cbase + first) * a.v_heads + hv) * (BOTH ? 2 : 1) + back) * TF + tid;
  rk.start(static_cast<const E*>(a.k) + tok * a.k_stride + (long)un.hk * K, a.k_stride, tid);
  if (BOTH) rq.start(static_cast<const E*>(a.q) + tok * a.q_stride + (long)un.hk * K, a.q_stride, tid);
  rv.start(static_cast<const E*>(back ? b.dout : a.v) + tok * vstride + (long)hv * a.dv + v0, vstride, tid);
  rg.start(a, tok, hv, lane, DELTA);
  const auto fetch = [&](int c) {
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    rk.fetch(rows, tid);
    if (back) rq.fetch(rows, tid);
    rv.fetch(trans ? 0 : rows, tid);
    rg.fetch(rows, lane);
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
        if (TF % 256 == 0 || i * 256 + tid < TF) rt[i] = tsrc[i * 256];
    }
    rk.step(way);
    if (BOTH) rq.step(way);
    rv.step(way);
    rg.step(way);
    tsrc += way * (long)a.v_heads * ((BOTH ? 2 : 1) * TF);
  };
  float* const keep = back ? b.grad : b.state;
  float* const rowmat = back ? b.dX : b.D;
  if (chunks) fetch(back ? chunks - 1 : 0);
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    const int c = back ? chunks - 1 - n : n;
    const int rows = sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ;
    const long t0 = sg.tok + (long)c * kQ;
    if (STORE) {
      float* p = keep + place(cbase + c);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + 16 * kt) = S[kt];
    }
    __syncthreads();  // the previous chunk's tiles are no longer read
    rk.put(s.k, LK, tid);
    if (back) rq.put(s.q, LK, tid);
    rv.put(s.v, 64, tid);
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
        if (TF % 256 == 0 || i * 256 + tid < TF) s.t[i * 256 + tid] = rt[i];
    }
    if (wave == 3) s.g.set(rg.rg, rg.rb, lane);
    if (n + 1 < chunks) fetch(back ? c - 1 : c + 1);
    __syncthreads();
    if (back) {
      // P^T by rows j, fragments (0, 1); (0, 0) and (3, 1); (1, 1); (2, 1) and (1, 0)
      const auto make = [&](int jt, int kb) {
        f32x4 acc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < KB; ++x) {
          const Frag kf = M::rows_c(s.k + (16 * jt + i16) * LK + 32 * x + 8 * g);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (2 * kb + h >= jt)
              acc[h] = M::mma(M::rows_c(s.q + (16 * (2 * kb + h) + i16) * LK + 32 * x + 8 * g), kf, acc[h]);
        }
        const int j = 16 * jt + i16;
        const float2 gj = s.g.G[j];
        float f[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * (2 * kb + h) + 4 * g + r;
            const float w = a.scale * exp2_f32(gap2(s.g.G[i], gj)) * acc[h][r];
            f[4 * h + r] = i >= j ? w : 0.f;
          }
        Split<T, TS> sp3;
        sp3.set(f);
        put_split<T, TS>(s.p, up_frag(jt, kb), sp3, lane);
      };
      if (wave == 0) {
        make(0, 1);
      } else if (wave == 1) {
        make(0, 0);
        make(3, 1);
      } else if (wave == 2) {
        make(1, 1);
      } else {
        make(2, 1);
        make(1, 0);
      }
    }
    // K S (or K dS'), rows t
    f32x4 R[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) R[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (DELTA || back) {
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = S[2 * x][r];
          f[4 + r] = S[2 * x + 1][r];
        }
        Split<T, TS> sf;
        sf.set(f);
        Frag kf[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) kf[it] = M::rows_d(s.k + (16 * it + i16) * LK + 32 * x + 4 * g);
#pragma unroll
        for (int k = TS - 1; k >= 0; --k)
#pragma unroll
          for (int it = 0; it < 4; ++it) R[it] = M::mma(kf[it], sf.t[k], R[it]);
      }
    }
    if (back) __syncthreads();  // s.p
    float d[2][8];  // tokens 32 kb + (4g + r, 16 + 4g + r), this lane's column
    Frag vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      vf[kb] = M::cols(cols_at<T, false>(s.v, 64, 32 * kb, 16 * wave, lane), 64);
      M::unpack(vf[kb], d[kb]);
    }
    if (back) {  // dD
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 e = *reinterpret_cast<const f32x4*>(&s.g.et[16 * it + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[it][r] *= e[r];
#pragma unroll
        for (int kb = it / 2; kb < 2; ++kb) {
          const auto pf = split_at<T, TS>(s.p, up_frag(it, kb), lane);
          R[it] = pf.a_times(vf[kb], R[it]);
        }
      }
    } else if (DELTA) {  // X
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 e = *reinterpret_cast<const f32x4*>(&s.g.eg[16 * it + 4 * g]);
        const f32x4 be = *reinterpret_cast<const f32x4*>(&s.g.beta[16 * it + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[it][r] = be[r] * fmaf(-e[r], R[it][r], d[it >> 1][4 * (it & 1) + r]);
      }
    }
    if (DELTA) {  // D = T X, or dX = T^T dD
      f32x4 acc[4];
      Split<T, TS> xf[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = R[2 * kb][r];
          f[4 + r] = R[2 * kb + 1][r];
        }
        xf[kb].set(f);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (back) {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int kb = it / 2; kb < 2; ++kb)
            acc[it] = mma_split<T, TS, TS>(split_at<T, TS>(s.t, up_frag(it, kb), lane), xf[kb], acc[it]);
      } else {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int kb = 0; kb <= it / 2; ++kb)
            acc[it] = mma_split<T, TS, TS>(split_at<T, TS>(s.t, low_frag(it, kb), lane), xf[kb], acc[it]);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) R[it] = acc[it];
      if (STORE) {
        float* p = rowmat + ((cbase + c) * a.v_heads + hv) * (long)(kQ * a.dv) + v0 + 16 * wave + i16;
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r) p[(16 * it + 4 * g + r) * a.dv] = acc[it][r];
      }
    } else if (STORE && back) {  // linear attention: dV
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * it + 4 * g + r;
          if (t < rows) Elt<T>::store1(b.dv, ((t0 + t) * a.v_heads + hv) * a.dv + v0 + 16 * wave + i16, R[it][r]);
        }
    }
    if (STORE && !back && n + 1 == chunks) break;  // the end is not read
    const float all = s.g.all;
    total *= all;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[kt][r] *= all;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (32 * kb >= rows) break;
      float f[8];  // the weighted rows that go with K (D; backward: dX), and with Q (dO)
      float o[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = 32 * kb + 16 * h + 4 * g;
        const f32x4 e = *reinterpret_cast<const f32x4*>(back ? &s.g.eg[at] : &s.g.et[at]);
        const f32x4 be = *reinterpret_cast<const f32x4*>(&s.g.beta[at]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          o[4 * h + r] = a.scale * e[r] * d[kb][4 * h + r];
          f[4 * h + r] = back ? -be[r] * e[r] * R[2 * kb + h][r]
                              : e[r] * (DELTA ? R[2 * kb + h][r] : d[kb][4 * h + r]);
        }
      }
      Split<T, TS> wf;
      if (DELTA || !back) {
        wf.set(f);
#pragma unroll
        for (int k4 = 0; k4 < KT; k4 += 4) {
          Frag kf[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) kf[x] = M::cols(cols_at<T, false>(s.k, LK, 32 * kb, 16 * (k4 + x), lane), LK);
#pragma unroll
          for (int k = TS - 1; k >= 0; --k)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[k4 + x] = M::mma(kf[x], wf.t[k], S[k4 + x]);
        }
      }
      if (back) {
        wf.set(o);
#pragma unroll
        for (int k4 = 0; k4 < KT; k4 += 4) {
          Frag qf[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) qf[x] = M::cols(cols_at<T, false>(s.q, LK, 32 * kb, 16 * (k4 + x), lane), LK);
#pragma unroll
          for (int k = TS - 1; k >= 0; --k)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[k4 + x] = M::mma(qf[x], wf.t[k], S[k4 + x]);
        }
      }
    }
  }
  if (!STORE) {
    if (!trans) {
      float* p = (back ? a.seg_grad : a.seg_state) + place(un.slot);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + 16 * kt) = S[kt];
      // once, so that the same call gives the same bits: forward but for a last segment
      if (!DELTA && tid == 0 && v0 == 0 && back == sg.last) a.seg_decay[(long)un.slot * a.v_heads + hv] = total;
      return;
    }
    if constexpr (DELTA) {
    // fragments (rows kt, columns jb) of the matrix, then (rows jt, columns kb) of its transpose
    constexpr int NF = KT * KB, LM = K + 4;
    char* const out = static_cast<char*>(a.trans) +
        ((long)un.slot * a.v_heads + hv) * ((BOTH ? 2 : 1) * NF * TS * 64 * sizeof(Frag));
    if (BOTH) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = S[2 * kb][r];
          f[4 + r] = S[2 * kb + 1][r];
        }
        Split<T, TS> x;
        x.set(f);
        put_split<T, TS>(out, NF + (v0 / 16 + wave) * KB + kb, x, lane);
      }
    }
    float* const sm = reinterpret_cast<float*>(&s);  // [64 columns][LM]
    static_assert(sizeof(L) >= 64 * LM * 4, "the matrix's columns fit");
    __syncthreads();
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(sm + (16 * wave + i16) * LM + 16 * kt + 4 * g) = S[kt];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < KT / 2; ++n) {
      const int id = wave * (KT / 2) + n, kt = id >> 1, jl = id & 1;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sm[(32 * jl + 4 * g + (e < 4 ? e : 12 + e)) * LM + 16 * kt + i16];
      Split<T, TS> x;
      x.set(f);
      put_split<T, TS>(out, kt * KB + v0 / 32 + jl, x, lane);
    }
    }
    return;
  }
  if (back && sg.first && b.dinit) {
    float* p = b.dinit + place(sg.seq);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      *reinterpret_cast<f32x4*>(p + 16 * kt) = has ? S[kt] : f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// Each sequence's segments in order (backward: from the last): what a segment adds is
// replaced by the state (the gradient) it starts from, S <- M S + N.  The delta rule:
// a wave for 16 columns, as in the recurrence.
template <typename T, int K>
static __global__ void __launch_bounds__(256) mix_combine_kernel(const MixBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::Frag Frag;
  constexpr int TS = M::kTerms, KT = K / 16, KB = K / 32, NF = KT * KB;
  const MixArgs& a = b.m;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool back = (int)blockIdx.x >= b.dir_blocks, both = a.seg_grad != nullptr;
  const int id = back ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int hv = id / a.slices % a.v_heads, v0 = id % a.slices * 64, seq = id / a.slices / a.v_heads;
  const SeqSpan sp = seq_span(a.cu, seq, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  const auto place = [&](long n) {
    return ((n * a.v_heads + hv) * a.dv + v0 + 16 * wave + (lane & 15)) * K + 4 * (lane >> 4);
  };
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int pool = a.init ? mix_slot(a, seq) : -1;
  const bool has = pool >= 0 && (!a.has_init || a.has_init[seq]);
  const float* src = back ? b.dfinal : (has ? a.init : nullptr);
  if (src) {
    src += place(back ? seq : pool);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(src + 16 * kt);
  }
  const long base = seg_base(a.cu, seq, a.seg, a.tokens);
#pragma unroll 1
  for (int n = 0; n < segs; ++n) {
    const long slot = base + (back ? segs - 1 - n : n);
    float* const p = (back ? a.seg_grad : a.seg_state) + place(slot);
    f32x4 add[KT];
    if (n + 1 < segs) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) add[kt] = *reinterpret_cast<const f32x4*>(p + 16 * kt);
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + 16 * kt) = S[kt];
    if (n + 1 == segs) break;
    const char* const tr = static_cast<const char*>(a.trans) +
        ((slot * a.v_heads + hv) * (both ? 2 : 1) + back) * (NF * TS * 64 * sizeof(Frag));
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float f[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = S[2 * kb][r];
        f[4 + r] = S[2 * kb + 1][r];
      }
      Split<T, TS> x;
      x.set(f);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        add[kt] = mma_split<T, TS, TS>(split_at<T, TS>(tr, kt * KB + kb, lane), x, add[kt]);
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = add[kt];
  }
}

// Linear attention: M is the segment's decay, so a thread for four elements.
static __global__ void __launch_bounds__(256) mix_combine_decay_kernel(const MixBwdArgs b) {
  const MixArgs& a = b.m;
  const bool back = (int)blockIdx.x >= b.dir_blocks;
  const int id = back ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int elems = b.elems, per = elems / 1024;
  const int e = (id % per * 256 + (int)threadIdx.x) * 4, hv = id / per % a.v_heads, seq = id / per / a.v_heads;
  const SeqSpan sp = seq_span(a.cu, seq, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  const int pool = a.init ? mix_slot(a, seq) : -1;
  const bool has = pool >= 0 && (!a.has_init || a.has_init[seq]);
  const float* src = back ? b.dfinal : (has ? a.init : nullptr);
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (src) S = *reinterpret_cast<const f32x4*>(src + ((long)(back ? seq : pool) * a.v_heads + hv) * elems + e);
  const long base = seg_base(a.cu, seq, a.seg, a.tokens);
  float* const mat = back ? a.seg_grad : a.seg_state;
  // eight segments' loads at a time: one after another they would take a memory
  // latency each
  constexpr int U = 8;
  for (int n0 = 0; n0 < segs; n0 += U) {
    f32x4 add[U];
    float d[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int n = n0 + q;
      add[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      d[q] = 0.f;
      if (n + 1 < segs) {
        const long at = (base + (back ? segs - 1 - n : n)) * a.v_heads + hv;
        add[q] = *reinterpret_cast<const f32x4*>(mat + at * elems + e);
        d[q] = a.seg_decay[at];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int n = n0 + q;
      if (n >= segs) break;
      *reinterpret_cast<f32x4*>(mat + ((base + (back ? segs - 1 - n : n)) * a.v_heads + hv) * elems + e) = S;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = fmaf(d[q], S[r], add[q][r]);
    }
  }
}

// Whether those launches hold fewer than 2^32 threads each.
static inline bool segments_fit(const MixArgs& a, int dk) {
  const long dir = mix_grid(a.slots, a.k_heads, (long)a.vpk * a.slices);
  const long tr = mix_grid(a.slots, a.k_heads, (long)a.vpk * (dk / 64));
  return grid_fits(2 * dir + tr, 256) && grid_fits(2L * a.seqs * a.v_heads * (dk * a.dv / 1024), 256);
}

// The launches in front of a call whose tokens may take several segments.
template <typename T, bool DELTA, bool BOTH>
static int launch_segments(MixBwdArgs b, int dk, hipStream_t stream) {
  const MixArgs& a = b.m;
  const long dir = mix_grid(a.slots, a.k_heads, (long)a.vpk * a.slices);
  const long tr = DELTA ? mix_grid(a.slots, a.k_heads, (long)a.vpk * (dk / 64)) : 0;
  const long cdir = DELTA ? (long)a.seqs * a.v_heads * a.slices : (long)a.seqs * a.v_heads * (dk * a.dv / 1024);
  const long grid = (BOTH ? 2 : 1) * dir + tr, cgrid = (BOTH ? 2 : 1) * cdir;
  b.dir_blocks = (int)dir;
  b.elems = dk * a.dv;
  const void* fn = dk == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 64, DELTA, false, BOTH>)
                            : reinterpret_cast<const void*>(&mix_states_kernel<T, 128, DELTA, false, BOTH>);
  const int rc = launch_kernel(fn, (unsigned)grid, 256, 0, stream, b);
  if (rc) return rc;
  b.dir_blocks = (int)cdir;
  if (DELTA)
    fn = dk == 64 ? reinterpret_cast<const void*>(&mix_combine_kernel<T, 64>)
                  : reinterpret_cast<const void*>(&mix_combine_kernel<T, 128>);
  else
    fn = reinterpret_cast<const void*>(&mix_combine_decay_kernel);
  return launch_kernel(fn, (unsigned)cgrid, 256, 0, stream, b);
}

}  // namespace rssm
