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
  int32_t* new_order;  // of the first launch (MixArgs::order), of all_slots segments
  int32_t all_slots;
  long do_stride, cslots;
  int32_t dir_blocks;  // blocks of one direction
  int32_t elems;       // of a state
};

template <typename T, int K, int V, bool DELTA, bool BOTH>
struct StatesLds {
  typedef typename Mat<T>::E E;
  static constexpr int kFrag = sizeof(typename Mat<T>::Frag), TS = Mat<T>::kTerms;
  static constexpr int TF = 6 * TS * 64 * kFrag / 16;  // 16-byte pieces of T or its transpose
  // fp32 with both directions' tiles twice would not fit 160 KB
  static constexpr int B = BOTH && sizeof(E) == 2 ? 2 : 1;
  __attribute__((aligned(16))) E k[B][Tile<T, K>::SIZE];
  __attribute__((aligned(16))) E v[B][Tile<T, V>::SIZE];  // V forward, dO backward
  __attribute__((aligned(16))) u32x4 t[DELTA ? B : 1][DELTA ? TF : 1];
  __attribute__((aligned(16))) E q[BOTH ? B : 1][BOTH ? Tile<T, K>::SIZE : 1];
  __attribute__((aligned(16))) u32x4 p[BOTH ? TF : 1];
  ChunkGates g[B];
};

// The segment slots by length, the longest first and those without a segment last, by one
// workgroup (64 classes of length; the order within one does not matter to any result):
// uneven sequences otherwise leave the longest to the end (16383 tokens of 13 sequences,
// delta rule: the outputs' launch takes a sixth less).
__device__ static inline void order_segments(const MixArgs& a, int slots, int32_t* order) {
  __shared__ int count[65];
  for (int i = threadIdx.x; i < 65; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const auto rank = [&](int slot) {
    const Segment sg = find_segment(a.cu, a.seqs, a.tokens, a.seg, slot);
    return sg.len == 0 ? 64 : 63 - (int)((sg.len - 1L) * 64 / a.seg);
  };
  for (int i = threadIdx.x; i < slots; i += blockDim.x) atomicAdd(&count[rank(i)], 1);
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = 0;
    for (int i = 0; i < 65; ++i) {
      const int n = count[i];
      count[i] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += blockDim.x) order[atomicAdd(&count[rank(i)], 1)] = i;
}

// One of the two recurrences over the chunks of a segment, a workgroup for one value
// head's state (mix_forward_kernel without the outputs).  Blocks: forward; BOTH:
// backward, last chunk first; the delta rule's transition.
// STORE: from the segment's start, leaving the states before all chunks, D and dX (or
// dV) and the gradient of the initial state.  Otherwise from zero, leaving what the
// segment adds and, as columns that start from the identity without V, the matrix that
// its starting state is multiplied by, as first operands: rows of it and (BOTH) of its
// transpose, which gradients go through.
// With STORE memory bounds it more than products do: 8 x 1024 tokens of 32 heads of the
// delta rule write 0.8 GB (and read 0.2) and take 288 us, three quarters of that with the
// products taken out and five eighths with the loads and stores taken out.  Without,
// products and what splits their factors bound it: 8 chunks a segment take 71 us, two
// workgroups a compute unit (four waves a SIMD; two take a tenth longer).
template <typename T, int K, int V, bool DELTA, bool STORE, bool BOTH>
static __global__ void __launch_bounds__(4 * V, BOTH || sizeof(typename Mat<T>::E) == 4 ? 2 : 4) mix_states_kernel(const MixBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  typedef StatesLds<T, K, V, DELTA, BOTH> L;
  typedef Tile<T, K> TK;
  typedef Tile<T, V> TV;
  static_assert(!DELTA || K == V, "the transition's columns are as many as V's");
  constexpr int TS = M::kTerms, KT = K / 16, KB = K / 32, TF = L::TF, W = V / 16, TH = 64 * W, B = L::B;
  constexpr bool kAhead = BOTH || !DELTA || sizeof(E) == 4;
  __shared__ union {
    L t;
    float m[STORE || !DELTA ? 1 : K * (K + 4)];
  } u;
  L& s = u.t;
  const MixArgs& a = b.m;
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (!STORE && blockIdx.x + 1 == gridDim.x) {
    order_segments(a, b.all_slots, b.new_order);
    return;
  }
  // Batches without a sequence of several segments: found by one look at the table (the
  // blocks' searches, one a compute unit at a time, took 13 us for 8 sequences of 32
  // heads; this takes 5 to 7).
  if (!STORE && a.seqs > 1 && a.seqs <= 64 &&
      !__any(lane < a.seqs && seq_span(a.cu, lane, a.seqs, a.tokens).len > a.seg)) return;
  // The kinds of a segment's block stand side by side: in parts of the grid of their own,
  // the second's live blocks met the first's on some units and left others idle, or did
  // not, by the time that empty blocks took (16383 tokens of 13 sequences: 175 us or 260).
  constexpr int KINDS = STORE ? 1 : 1 + BOTH + DELTA;
  const int second = STORE && (int)blockIdx.x >= b.dir_blocks;
  const int turn = blockIdx.x >> 3, kind = STORE ? second : turn % KINDS;  // (the lowest bits: the die)
  const bool back = BOTH && kind == 1, trans = !STORE && DELTA && kind == KINDS - 1;
  const MixUnit un = mix_unit(a, STORE ? blockIdx.x - second * b.dir_blocks
                                       : turn / KINDS * 8 + (blockIdx.x & 7), a.vpk);
  if (STORE && blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if (!un.live) return;
  const int hv = un.hk * a.vpk + un.rest;
  const Segment sg = STORE ? find_segment(a.cu, a.seqs, a.tokens, a.seg, un.slot)
                           : find_long(a.cu, a.seqs, a.tokens, a.seg, a.few, un.slot);
  if (sg.len == 0 && !(STORE && sg.empty)) return;
  const bool whole = sg.first && sg.last;
  const long kept = STORE ? long_base(a.cu, sg.seq, a.seg, a.tokens, a.few) + sg.k : un.slot;  // (not of a whole one)
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
  const auto place = [&](long n) { return ((n * a.v_heads + hv) * V + 16 * wave + i16) * K + 8 * g; };
  if (STORE) {
    const float* src = back ? b.dfinal : (has ? a.init : nullptr);
    if (!whole) src = back ? a.seg_grad : a.seg_state;
    if (src) {
      src += place(!whole ? kept : (back ? sg.seq : pool));
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(src + mix_row(kt, 0));
    }
  } else if (trans) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[kt][r] = mix_row(kt, 4 * g + r) == mix_row(wave, i16) ? 1.f : 0.f;
  }
  float total = 1.f;
  const long vstride = back ? b.do_stride : a.v_stride;
  const long cbase = seg_base(a.cu, sg.seq, kQ, a.tokens) + (long)sg.k * (a.seg / kQ);
  const int chunks = (sg.len + kQ - 1) / kQ, way = back ? -1 : 1;
  const long first = chunks && back ? chunks - 1 : 0, tok = sg.tok + first * kQ;
  TileLoad<T, K, TH> rk, rq;
  TileLoad<T, V, TH> rv;
  GateLoad rg;
  FragLoad<TF, TH> rt;
  rt.p = static_cast<const u32x4*>(a.tinv) + (((cbase + first) * a.v_heads + hv) * (BOTH ? 2 : 1) + back) * TF;
  rk.start(static_cast<const E*>(a.k) + tok * a.k_stride + (long)un.hk * K, a.k_stride, tid);
  if (BOTH) rq.start(static_cast<const E*>(a.q) + tok * a.q_stride + (long)un.hk * K, a.q_stride, tid);
  rv.start(static_cast<const E*>(back ? b.dout : a.v) + tok * vstride + (long)hv * V, vstride, tid);
  rg.start(a, tok, hv, DELTA);
  const Minus minus;
  const auto rows_of = [&](int c) { return sg.len - c * kQ < kQ ? sg.len - c * kQ : kQ; };
  const auto fetch = [&](int c) {
    const int rows = rows_of(c);
    rk.fetch(rows, tid);
    if (back) rq.fetch(rows, tid);
    rv.fetch(rows, tid);
    rg.fetch(rows, lane);
    if (DELTA) rt.fetch(tid);
    rk.step(way);
    if (BOTH) rq.step(way);
    rv.step(way);
    rg.step(way);
    rt.p += way * (long)a.v_heads * ((BOTH ? 2 : 1) * TF);
  };
  const auto put = [&](int n) {
    const int rows = rows_of(back ? chunks - 1 - n : n);
    rk.put(s.k[n % B], rows, tid);
    if (back) rq.put(s.q[BOTH ? n % B : 0], rows, tid);
    rv.put(s.v[n % B], trans ? 0 : rows, tid);
    if (DELTA) rt.put(s.t[DELTA ? n % B : 0], tid);
    if (wave == W - 1) s.g[n % B].set(rg.log_g(rows, lane), rg.beta(rows, lane), lane);
  };
  float* const keep = back ? b.grad : b.state;
  float* const rowmat = back ? b.dX : b.D;
  if (chunks) {
    fetch(back ? chunks - 1 : 0);
    put(0);
  }
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) forget(S[kt]);  // has arrived: see mix_forward_kernel
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    const int c = back ? chunks - 1 - n : n, rows = rows_of(c);
    const long t0 = sg.tok + (long)c * kQ;
    const E *const sK = s.k[n % B], *const sQ = s.q[BOTH ? n % B : 0], *const sV = s.v[n % B];
    const u32x4* const sT = s.t[DELTA ? n % B : 0];
    const ChunkGates& gt = s.g[n % B];
    if (STORE) {
      float* p = keep + place(cbase + c);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + mix_row(kt, 0)) = S[kt];
    }
    __syncthreads();
    if (kAhead && n + 1 < chunks) fetch(back ? c - 1 : c + 1);
    // K S (or K dS'), rows t; backward: this wave's tiles of q_i.k_j, rows i
    f32x4 R[4], P[2], P2[2];
#pragma unroll
    for (int it = 0; it < 4; ++it) R[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    P[0] = P[1] = P2[0] = P2[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // P^T by rows j: fragments (0, 1), (0, 0), (1, 1), (2, 1), then (3, 1) and (1, 0)
    const int jt = wave < 2 ? 0 : (wave == 2 ? 1 : (wave == 3 ? 2 : (wave == 4 ? 3 : 1)));
    const int kp = wave == 0 || wave == 2 || wave == 3 || wave == 4;
    if (DELTA || back) {
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = S[2 * x][r];
          f[4 + r] = S[2 * x + 1][r];
        }
        const auto sf = split<T, TS>(f, minus);
        Frag kf[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) kf[it] = TK::rows_c(sK, it, 32 * x, lane);
#pragma unroll
        for (int k = TS - 1; k >= 0; --k)
#pragma unroll
          for (int it = 0; it < 4; ++it) R[it] = M::mma(kf[it], sf.t[k], R[it]);
        if (back && wave < 6) {
          const Frag kj = TK::rows_c(sK, jt, 32 * x, lane);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (2 * kp + h >= jt) P[h] = M::mma(TK::rows_c(sQ, 2 * kp + h, 32 * x, lane), kj, P[h]);
          if (W == 4 && wave < 2) {  // (1, 0) and (3, 1): one tile each
            const int j2 = wave ? 3 : 1;
            P2[1] = M::mma(TK::rows_c(sQ, j2, 32 * x, lane), TK::rows_c(sK, j2, 32 * x, lane), P2[1]);
          }
        }
      }
    }
    if (back) {
      const auto make = [&](int jb, int kb, const f32x4* acc) {
        const int j = 16 * jb + i16;
        const float2 gj = gt.G[j];
        float f[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * (2 * kb + h) + 4 * g + r;
            const float w = a.scale * exp2_f32(gap2(gt.G[i], gj)) * acc[h][r];
            f[4 * h + r] = i >= j ? w : 0.f;
          }
        const auto x = split<T, TS>(f, minus);
        put_split<T, TS>(s.p, up_frag(jb, kb), x, lane);
      };
      if (wave < 6) make(jt, kp, P);
      if (W == 4 && wave < 2) make(wave ? 3 : 1, wave, P2);
      __syncthreads();
    }
    float d[2][8];  // tokens 32 kb + (4g + r, 16 + 4g + r), this lane's column
    Frag vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      vf[kb] = TV::cols(sV, 32 * kb, 16 * wave, lane);
      M::unpack(vf[kb], d[kb]);
    }
    if (back) {  // dD
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 e = *reinterpret_cast<const f32x4*>(&gt.et[16 * it + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[it][r] *= e[r];
      }
      Split<T, 1> o0, o1;
      o0.t[0] = vf[0];
      o1.t[0] = vf[1];
      mma_many<T, TS, 1, 2>([&](int n, int k) { return frag_at<T>(s.p, up_frag(n, 0) * TS + k, lane); }, o0, R);
      mma_many<T, TS, 1, 4>([&](int n, int k) { return frag_at<T>(s.p, up_frag(n, 1) * TS + k, lane); }, o1, R);
    } else if (DELTA) {  // X
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 e = *reinterpret_cast<const f32x4*>(&gt.eg[16 * it + 4 * g]);
        const f32x4 be = *reinterpret_cast<const f32x4*>(&gt.beta[16 * it + 4 * g]);
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
        xf[kb] = split<T, TS>(f, minus);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (back) {
        mma_many<T, TS, TS, 2>([&](int n, int k) { return frag_at<T>(sT, up_frag(n, 0) * TS + k, lane); }, xf[0], acc);
        mma_many<T, TS, TS, 4>([&](int n, int k) { return frag_at<T>(sT, up_frag(n, 1) * TS + k, lane); }, xf[1], acc);
      } else {
        mma_many<T, TS, TS, 4>([&](int n, int k) { return frag_at<T>(sT, low_frag(n, 0) * TS + k, lane); }, xf[0], acc);
        mma_many<T, TS, TS, 2>([&](int n, int k) { return frag_at<T>(sT, low_frag(2 + n, 1) * TS + k, lane); }, xf[1],
                               acc + 2);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) R[it] = acc[it];
      if (STORE) {
        float* p = rowmat + ((cbase + c) * a.v_heads + hv) * (long)(kQ * V) + 16 * wave + i16;
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r) p[(16 * it + 4 * g + r) * V] = acc[it][r];
      }
    } else if (STORE && back) {  // linear attention: dV
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * it + 4 * g + r;
          if (t < rows) Elt<T>::store1(b.dv, ((t0 + t) * a.v_heads + hv) * V + 16 * wave + i16, R[it][r]);
        }
    }
    if (STORE && !back && n + 1 == chunks) break;  // the end is not read
    if (B == 2 && n + 1 < chunks) put(n + 1);
    const float all = gt.all;
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
        const f32x4 e = *reinterpret_cast<const f32x4*>(back ? &gt.eg[at] : &gt.et[at]);
        const f32x4 be = *reinterpret_cast<const f32x4*>(&gt.beta[at]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          o[4 * h + r] = a.scale * e[r] * d[kb][4 * h + r];
          f[4 * h + r] = back ? -be[r] * e[r] * R[2 * kb + h][r]
                              : e[r] * (DELTA ? R[2 * kb + h][r] : d[kb][4 * h + r]);
        }
      }
      Split<T, TS> wf;
      if (DELTA || !back) {
        wf = split<T, TS>(f, minus);
#pragma unroll
        for (int k4 = 0; k4 < KT; k4 += 4) {
          Frag kf[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) kf[x] = TK::cols_of(sK, 32 * kb, k4 + x, lane);
#pragma unroll
          for (int k = TS - 1; k >= 0; --k)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[k4 + x] = M::mma(kf[x], wf.t[k], S[k4 + x]);
        }
      }
      if (back) {
        wf = split<T, TS>(o, minus);
#pragma unroll
        for (int k4 = 0; k4 < KT; k4 += 4) {
          Frag qf[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) qf[x] = TK::cols_of(sQ, 32 * kb, k4 + x, lane);
#pragma unroll
          for (int k = TS - 1; k >= 0; --k)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[k4 + x] = M::mma(qf[x], wf.t[k], S[k4 + x]);
        }
      }
    }
    if (B == 1) {
      __syncthreads();  // the tiles are no longer read
      if (n + 1 < chunks) {
        if (!kAhead) fetch(back ? c - 1 : c + 1);
        put(n + 1);
      }
    }
  }
  if (!STORE) {
    if (!trans) {
      float* p = (back ? a.seg_grad : a.seg_state) + place(kept);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + mix_row(kt, 0)) = S[kt];
      // once, so that the same call gives the same bits: forward but for a last segment
      if (!DELTA && tid == 0 && back == sg.last) a.seg_decay[kept * a.v_heads + hv] = total;
      return;
    }
    if constexpr (DELTA) {
    // fragments (rows kt, columns jb) of the matrix, then (rows jt, columns kb) of its transpose
    constexpr int NF = KT * KB, LM = K + 4;
    char* const out = static_cast<char*>(a.trans) +
        (kept * a.v_heads + hv) * ((BOTH ? 2 : 1) * NF * TS * 64 * sizeof(Frag));
    if (BOTH) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] = S[2 * kb][r];
          f[4 + r] = S[2 * kb + 1][r];
        }
        const auto x = split<T, TS>(f, minus);
        put_split<T, TS>(out, NF + wave * KB + kb, x, lane);
      }
    }
    float* const sm = u.m;  // [K columns][LM]
    __syncthreads();
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(sm + mix_row(wave, i16) * LM + mix_row(kt, 4 * g)) = S[kt];
    __syncthreads();
#pragma unroll
    for (int jb = 0; jb < KB; ++jb) {  // a wave for 16 rows
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sm[(32 * jb + 8 * g + e) * LM + mix_row(wave, i16)];
      const auto x = split<T, TS>(f, minus);
      put_split<T, TS>(out, wave * KB + jb, x, lane);
    }
    }
    return;
  }
  if (back && sg.first && b.dinit) {
    float* p = b.dinit + place(sg.seq);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      *reinterpret_cast<f32x4*>(p + mix_row(kt, 0)) = has ? S[kt] : f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// The sequence that a combining workgroup takes: the n-th, or, where most are short, the
// one whose segments begin at place n; -1: none.
__device__ static inline int combine_seq(const MixArgs& a, int n) {
  if (a.few) return n;
  const Segment sg = find_long(a.cu, a.seqs, a.tokens, a.seg, false, n);
  return sg.len && sg.first ? sg.seq : -1;
}

// Each sequence's segments in order (backward: from the last): what a segment adds is
// replaced by the state (the gradient) it starts from, S <- M S + N.  The delta rule: a
// workgroup for 32 columns, a wave for 32 rows of them: it reads its rows of M alone, the
// next segment's as this one's are used up, and S is passed on through LDS as terms, with
// one barrier a segment, 3 us.  (With all rows of 16 columns a wave and M through LDS a
// segment took 6 us.)
template <typename T, int K>
static __global__ void __launch_bounds__(2 * K) mix_combine_kernel(const MixBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::Frag Frag;
  constexpr int TS = M::kTerms, KB = K / 32, NF = 2 * KB * KB;
  __shared__ __attribute__((aligned(16))) Frag sS[2][KB * 2 * TS * 64];
  const MixArgs& a = b.m;
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool back = (int)blockIdx.x >= b.dir_blocks, both = a.seg_grad != nullptr;
  const int id = back ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int hv = id / KB % a.v_heads, c0 = id % KB * 32, seq = combine_seq(a, id / KB / a.v_heads);
  if (seq < 0) return;
  const SeqSpan sp = seq_span(a.cu, seq, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  // this lane's first element: rows 32 wave + 8 g + 4 h, column c0 + 16 ct + i16
  const auto place = [&](long n, int h, int ct) {
    return ((n * a.v_heads + hv) * K + c0 + 16 * ct + i16) * K + 32 * wave + 8 * g + 4 * h;
  };
  const int pool = a.init ? mix_slot(a, seq) : -1;
  const bool has = pool >= 0 && (!a.has_init || a.has_init[seq]);
  const long base = long_base(a.cu, seq, a.seg, a.tokens, a.few);
  const auto slot_of = [&](int n) { return base + (back ? segs - 1 - n : n); };
  float* const mat = back ? a.seg_grad : a.seg_state;
  const Minus minus;
  Frag m[KB][2][TS];
  f32x4 S[2][2], add[2][2];  // [h][ct]
  const auto fetch_m = [&](int n, int kb) {
    const char* const p = static_cast<const char*>(a.trans) +
        ((slot_of(n) * a.v_heads + hv) * (both ? 2 : 1) + back) * (NF * TS * 64 * sizeof(Frag));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < TS; ++k) m[kb][h][k] = frag_at<T>(p, ((2 * wave + h) * KB + kb) * TS + k, lane);
  };
  const auto fetch_add = [&](int n) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) add[h][ct] = *reinterpret_cast<const f32x4*>(mat + place(slot_of(n), h, ct));
  };
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) fetch_m(0, kb);
  fetch_add(0);
  const float* src = back ? b.dfinal : (has ? a.init : nullptr);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct)
      S[h][ct] = src ? *reinterpret_cast<const f32x4*>(src + place(back ? seq : pool, h, ct)) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int n = 0;; ++n) {
    const long slot = slot_of(n);
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      float f[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = S[0][ct][r];
        f[4 + r] = S[1][ct][r];
      }
      put_split<T, TS>(sS[n & 1], wave * 2 + ct, split<T, TS>(f, minus), lane);
    }
    f32x4 acc[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) acc[h][ct] = add[h][ct];
    const int next = n + 2 < segs ? n + 1 : n;  // (at the end: the same again)
    fetch_add(next);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) *reinterpret_cast<f32x4*>(mat + place(slot, h, ct)) = S[h][ct];
    if (n + 1 == segs) break;
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Split<T, TS> x[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) x[ct] = split_at<T, TS>(sS[n & 1], kb * 2 + ct, lane);
#pragma unroll
      for (int s = TS - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) acc[h][ct] = M::mma(m[kb][h][i], x[ct].t[s - i], acc[h][ct]);
      fetch_m(next, kb);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) S[h][ct] = acc[h][ct];
  }
}

// Linear attention: M is the segment's decay, so a thread for four elements.
static __global__ void __launch_bounds__(256) mix_combine_decay_kernel(const MixBwdArgs b) {
  const MixArgs& a = b.m;
  const bool back = (int)blockIdx.x >= b.dir_blocks;
  const int id = back ? blockIdx.x - b.dir_blocks : blockIdx.x;
  const int elems = b.elems, per = elems / 1024;
  const int e = (id % per * 256 + (int)threadIdx.x) * 4, hv = id / per % a.v_heads;
  const int seq = combine_seq(a, id / per / a.v_heads);
  if (seq < 0) return;
  const SeqSpan sp = seq_span(a.cu, seq, a.seqs, a.tokens);
  const int segs = (sp.len + a.seg - 1) / a.seg;
  if (segs <= 1) return;
  const int pool = a.init ? mix_slot(a, seq) : -1;
  const bool has = pool >= 0 && (!a.has_init || a.has_init[seq]);
  const float* src = back ? b.dfinal : (has ? a.init : nullptr);
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (src) S = *reinterpret_cast<const f32x4*>(src + ((long)(back ? seq : pool) * a.v_heads + hv) * elems + e);
  const long base = long_base(a.cu, seq, a.seg, a.tokens, a.few);
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

// Blocks of those launches: of the recurrences over the segments, and of one direction's
// combination.
struct SegGrids {
  long states, combine;
};
static inline SegGrids segment_grids(const MixArgs& a, int dk, bool delta, bool both) {
  const long places = long_places(a.tokens, a.seqs, a.seg);
  return {mix_grid(places, a.k_heads, a.vpk) * (1 + both + delta) + 1,
          (a.few ? a.seqs : places) * a.v_heads * (delta ? dk / 32 : dk * a.dv / 1024)};
}
// Whether they hold fewer than 2^32 threads each, where a call has them.
static inline bool segments_fit(const MixArgs& a, int dk, bool delta, bool both) {
  if (a.tokens <= a.seg) return true;
  const SegGrids n = segment_grids(a, dk, delta, both);
  return grid_fits(n.states, 4 * a.dv) && grid_fits((1 + both) * n.combine, delta ? 2 * dk : 256);
}

template <typename T, bool BOTH>
static const void* pick_segments(int dk, int dv, bool delta) {
  if (delta)
    return dk == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 64, true, false, BOTH>)
                    : reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 128, true, false, BOTH>);
  if (dk == 64)
    return dv == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 64, false, false, BOTH>)
                    : reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 128, false, false, BOTH>);
  return dv == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 64, false, false, BOTH>)
                  : reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 128, false, false, BOTH>);
}

// The launches in front of a call whose tokens may take several segments.
template <typename T, bool BOTH>
static int launch_segments(MixBwdArgs b, int dk, bool delta, hipStream_t stream) {
  const MixArgs& a = b.m;
  const SegGrids n = segment_grids(a, dk, delta, BOTH);
  b.elems = dk * a.dv;
  MixBwdArgs first = b;  // its own units are in no order yet: the last block makes it
  first.new_order = const_cast<int32_t*>(b.m.order);
  first.m.order = nullptr;
  first.all_slots = a.slots;
  first.m.slots = (int)long_places(a.tokens, a.seqs, a.seg);
  const int rc = launch_kernel(pick_segments<T, BOTH>(dk, a.dv, delta),
                               (unsigned)n.states, 4 * a.dv, 0, stream, first);
  if (rc) return rc;
  b.dir_blocks = (int)n.combine;
  const void* fn = reinterpret_cast<const void*>(&mix_combine_decay_kernel);
  if (delta)
    fn = dk == 64 ? reinterpret_cast<const void*>(&mix_combine_kernel<T, 64>)
                  : reinterpret_cast<const void*>(&mix_combine_kernel<T, 128>);
  return launch_kernel(fn, (unsigned)((1 + BOTH) * n.combine), delta ? 2 * dk : 256, 0, stream, b);
}

}  // namespace rssm
