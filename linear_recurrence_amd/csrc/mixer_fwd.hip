// Linear attention and the gated delta rule over packed sequences, forward (the
// chunked form: mixer_common.hpp).
//
// The delta rule's T of every chunk is independent of the state and comes from a
// launch in front (mix_inverse_kernel).  Then a workgroup walks the chunks of one
// sequence (or a segment of one) and value head with the state in registers; the next
// chunk's tiles are on their way while one is worked on.
//
// The states, X, D and the decayed q.k are fp32 values and enter all products as three
// bf16 terms (24 bits), so nothing is rounded to the io type but o itself.  Two terms
// in o's products would be 3 to 9% faster (16383 tokens of 32 heads of 128: 529 us
// instead of 547, linear attention 243 instead of 265) and leave twenty times the fp32
// sums' own error in o.  fp32 inputs stay fp32 everywhere.
#include "mixer_states.hpp"

namespace rssm {

template <typename T, int K, int V, bool DELTA>
struct ForwardLds {
  typedef typename Mat<T>::E E;
  static constexpr int kFrag = sizeof(typename Mat<T>::Frag);
  static constexpr int TF = 6 * Mat<T>::kTerms * 64 * kFrag / 16;  // 16-byte pieces of T
  // fp32: nothing is left of 160 KB for the outputs
  static constexpr int kOut = sizeof(E) == 4 ? Tile<T, V>::SIZE / 4 : 1;
  __attribute__((aligned(16))) E k[2][Tile<T, K>::SIZE];
  __attribute__((aligned(16))) E q[Tile<T, K>::SIZE];
  __attribute__((aligned(16))) E v[Tile<T, V>::SIZE];
  __attribute__((aligned(16))) u32x4 t[DELTA ? TF : 1];
  __attribute__((aligned(16))) u32x4 p[TF];
  __attribute__((aligned(16))) E o[Tile<T, V>::SIZE / kOut];
  ChunkGates g[2];
};

// A workgroup for one value head and segment, a wave for 16 columns of its state.  Two
// barriers a chunk: behind the first its tiles are in LDS and the next chunk's loads
// start; at the second the tiles of q, v and T are no longer read, and take the next
// chunk's (K, read to the end, has two).  The outputs cross LDS and go to memory behind
// the next barrier, a row's neighbours together: as the lanes hold them, 32 bytes of a
// row a wave, their stores took a fifth of the time.  A chunk of the delta rule takes 8.1
// us: 3.0 of the matrix units (224 products a wave, 16 cycles each), 2.2 of the vector
// units (splitting and weighing the products' factors) and 2.8 of LDS, a third of it bank
// conflicts; they overlap little in one workgroup a compute unit.  One of linear attention
// takes 5.7: 1.6, 1.5 and 1.9, and its bytes 3.5 at a copy's rate.  4096 tokens of 32 heads
// of 128: 72 us (linear attention 51) for 8 chunks a workgroup; 16383 tokens: 300 and 196.
// Waves of 32 columns, one a SIMD, were slower (a fifth).
template <typename T, int K, int V, bool DELTA>
__global__ void __launch_bounds__(4 * V, 2) mix_forward_kernel(const MixArgs a) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  typedef ForwardLds<T, K, V, DELTA> L;
  typedef Tile<T, K> TK;
  typedef Tile<T, V> TV;
  constexpr bool kBf16 = sizeof(E) == 2;
  constexpr int TS = M::kTerms, W = V / 16, TH = 64 * W;
  constexpr int KT = K / 16, KB = K / 32, TF = L::TF;
  __shared__ L s;
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int dv = V == 128 ? V : a.dv, parts = dv / V;
  const MixUnit un = mix_unit(a, blockIdx.x, a.vpk * parts);
  if (blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if (!un.live) return;
  const int hv = un.hk * a.vpk + un.rest / parts, v0 = un.rest % parts * V;  // the head, its first column
  const Segment sp = find_segment(a.cu, a.seqs, a.tokens, a.seg, un.slot);
  if (sp.len == 0 && !sp.empty) return;
  const int pool = a.init || a.final_state ? mix_slot(a, sp.seq) : -1;
  if (tid == 0 && sp.first && un.rest == 0 && un.hk == 0 && a.status && (a.init || a.final_state) && pool < 0)
    atomicOr(a.status, RSSM_ST_BAD_SLOT);
  // S: rows mix_row(kt, 4g + r), column 16 wave + i16
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto place = [&](long n) { return ((n * a.v_heads + hv) * dv + v0 + 16 * wave + i16) * K + 8 * g; };
  // The pool is read here only by a sequence of one segment, whose wave also writes it:
  // a longer one's first segment takes the copy that the combining launch left, since
  // its last segment may already have stored the final state over the initial one.
  const bool whole = sp.first && sp.last;
  if (!whole || (a.init && pool >= 0 && (!a.has_init || a.has_init[sp.seq]))) {
    const float* p = whole ? a.init + place(pool)
                           : a.seg_state + place(long_base(a.cu, sp.seq, a.seg, a.tokens, a.few) + sp.k);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(p + mix_row(kt, 0));
  }
  const long cbase = seg_base(a.cu, sp.seq, kQ, a.tokens) + (long)sp.k * (a.seg / kQ);
  const int chunks = (sp.len + kQ - 1) / kQ;
  TileLoad<T, K, TH> rk, rq;
  TileLoad<T, V, TH> rv;
  GateLoad rg;
  FragLoad<TF, TH> rt;
  rt.p = static_cast<const u32x4*>(a.tinv) + (cbase * a.v_heads + hv) * TF;
  rk.start(static_cast<const E*>(a.k) + sp.tok * a.k_stride + (long)un.hk * K, a.k_stride, tid);
  rq.start(static_cast<const E*>(a.q) + sp.tok * a.q_stride + (long)un.hk * K, a.q_stride, tid);
  rv.start(static_cast<const E*>(a.v) + sp.tok * a.v_stride + (long)hv * dv + v0, a.v_stride, tid);
  rg.start(a, sp.tok, hv, DELTA);
  const long orow = (long)a.v_heads * dv;
  E* out = static_cast<E*>(a.o) + ((long)sp.tok * a.v_heads + hv) * dv + v0;
  if (kBf16) out += tid / TileLoad<T, V, TH>::PER * orow + tid % TileLoad<T, V, TH>::PER * 8;
  else out += i16 * orow + 16 * wave + 4 * g;
  // 16 bytes of every R-th row of the chunk before
  const auto store = [&](int rows) {
    constexpr int PER = TileLoad<T, V, TH>::PER, R = TileLoad<T, V, TH>::R;
#pragma unroll
    for (int i = 0; i < kQ / R; ++i)
      if (tid / PER + i * R < rows)
        *reinterpret_cast<u32x4*>(out + i * R * orow) =
            *reinterpret_cast<const u32x4*>(s.o + TV::at(tid / PER + i * R, tid % PER * 8));
    out += kQ * orow;
  };
  const Minus minus;
  const auto rows_of = [&](int c) { return sp.len - c * kQ < kQ ? sp.len - c * kQ : kQ; };
  const auto fetch = [&](int c) {
    const int rows = rows_of(c);
    rk.fetch(rows, tid);
    rq.fetch(rows, tid);
    rv.fetch(rows, tid);
    rg.fetch(rows, lane);
    if (DELTA) rt.fetch(tid);
    rk.step(1);
    rq.step(1);
    rv.step(1);
    rg.step(1);
    rt.p += (long)a.v_heads * TF;
  };
  const auto put = [&](int c) {
    const int rows = rows_of(c);
    rk.put(s.k[c & 1], rows, tid);
    rq.put(s.q, rows, tid);
    rv.put(s.v, rows, tid);
    if (DELTA) rt.put(s.t, tid);
    if (wave == W - 1) s.g[c & 1].set(rg.log_g(rows, lane), rg.beta(rows, lane), lane);
  };
  if (chunks) {
    fetch(0);
    put(0);
  }
  // The state has arrived: waited for at its first use, in the loop, it would have every
  // chunk wait for the next one's loads too.
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) forget(S[kt]);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const int rows = rows_of(c);
    const E* const sK = s.k[c & 1];
    const ChunkGates& sg = s.g[c & 1];
    __syncthreads();
    if (c + 1 < chunks) fetch(c + 1);
    if (kBf16 && c) store(kQ);
    f32x4 R[4], O[4];  // K S, rows t; (Q S)^T, columns t
    f32x4 P[2];        // this wave's tiles of k_j.q_i, rows j
#pragma unroll
    for (int it = 0; it < 4; ++it) R[it] = O[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    P[0] = P[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 P2[2];
    P2[0] = P2[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      float f[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = S[2 * b][r];
        f[4 + r] = S[2 * b + 1][r];
      }
      const auto sf = split<T, TS>(f, minus);
      Frag kf[4], qf[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        kf[it] = TK::rows_c(sK, it, 32 * b, lane);
        qf[it] = TK::rows_c(s.q, it, 32 * b, lane);
      }
#pragma unroll
      for (int k = TS - 1; k >= 0; --k)
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          if (DELTA) R[it] = M::mma(kf[it], sf.t[k], R[it]);
          O[it] = M::mma(sf.t[k], qf[it], O[it]);
        }
    }
    // k_j.q_i of the lower triangle's six fragments: a wave each (of four waves, two have a
    // second one)
    const int pi = wave < 2 ? 3 : (wave == 2 || wave == 5 ? 2 : (wave == 3 ? 1 : 0)), pk = wave == 1 || wave == 5;
    if (wave < 6) {
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const Frag qf = TK::rows_c(s.q, pi, 32 * b, lane);
        P[0] = M::mma(TK::rows_c(sK, 2 * pk, 32 * b, lane), qf, P[0]);
        P[1] = M::mma(TK::rows_c(sK, 2 * pk + 1, 32 * b, lane), qf, P[1]);
        if (W == 4 && wave < 2)
          P2[0] = M::mma(TK::rows_c(sK, 2 * wave, 32 * b, lane), TK::rows_c(s.q, 2 * wave, 32 * b, lane), P2[0]);
      }
    }
    {
      // scale e^{G_i-G_j} q_i.k_j as a fragment
      const auto weigh = [&](int i, int j, const f32x4& p, float* f) {  // of one tile
        const float2 gi = sg.G[16 * i + i16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = a.scale * exp2_f32(gap2(gi, sg.G[16 * j + 4 * g + r])) * p[r];
          f[r] = j < i || (j == i && 4 * g + r <= i16) ? w : 0.f;
        }
      };
      const auto make = [&](int it, int kb, const f32x4* p) {
        float f[8];
        weigh(it, 2 * kb, p[0], f);
        weigh(it, 2 * kb + 1, p[1], f + 4);
        put_split<T, TS>(s.p, low_frag(it, kb), split<T, TS>(f, minus), lane);
      };
      if (wave < 6) make(pi, pk, P);
      if (W == 4 && wave < 2) make(wave ? 2 : 0, wave, P2);
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
      M::unpack(TV::cols(s.v, 32 * kb, 16 * wave, lane), d[kb]);
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
        const auto xf = split<T, TS>(d[kb], minus);
        const auto tf = [&](int n, int k) { return frag_at<T>(s.t, low_frag(2 * kb + n, kb) * TS + k, lane); };
        if (kb == 0) mma_many<T, TS, TS, 4>(tf, xf, acc);
        else mma_many<T, TS, TS, 2>(tf, xf, acc + 2);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) d[it >> 1][4 * (it & 1) + r] = acc[it][r];
    }
    __syncthreads();  // P; and q, v and T are no longer read
    if (c + 1 < chunks) put(c + 1);
    // o^T += D^T P^T, and S' = e^{G_Q} S + K^T (e^{G_Q - G} D)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const auto df = split<T, DELTA ? TS : 1>(d[kb], minus);  // (V is an input)
      const auto pf = [&](int n, int k) { return frag_at<T>(s.p, low_frag(2 * kb + n, kb) * TS + k, lane); };
      if (kb == 0) mma_many<T, TS, DELTA ? TS : 1, 4, true>(pf, df, O);
      else mma_many<T, TS, DELTA ? TS : 1, 2, true>(pf, df, O + 2);
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
      const auto wf = split<T, TS>(d[kb], minus);
#pragma unroll
      for (int k4 = 0; k4 < KT; k4 += 4) {
        Frag kf[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) kf[q] = TK::cols_of(sK, 32 * kb, k4 + q, lane);
#pragma unroll
        for (int k = TS - 1; k >= 0; --k)
#pragma unroll
          for (int q = 0; q < 4; ++q) S[k4 + q] = M::mma(kf[q], wf.t[k], S[k4 + q]);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const float f[4] = {O[it][0], O[it][1], O[it][2], O[it][3]};
      if (kBf16)
        *reinterpret_cast<typename M::Four*>(s.o + TV::at(16 * it + i16, 16 * wave + 4 * g)) = M::pack4(f);
      else if (16 * it + i16 < rows)
        *reinterpret_cast<typename M::Four*>(out + 16 * it * orow) = M::pack4(f);
    }
    if (!kBf16) out += kQ * orow;
  }
  if (kBf16 && chunks) {
    __syncthreads();
    store(sp.len - (chunks - 1) * kQ);
  }
  if (sp.last && a.final_state && pool >= 0) {
    float* p = a.final_state + place(pool);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(p + mix_row(kt, 0)) = S[kt];
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

// Columns of a head that a workgroup takes: 64 of 128 while there are compute units for
// both halves' workgroups, since a chunk takes less time with one wave a SIMD than with
// two, and every half does the tokens' products again (delta rule, 32 heads of 128, 512
// tokens: 62 us instead of 74; fp32 122 instead of 170; linear attention 39 instead of 43).
static int forward_columns(const rssm_mixer_dims& d, long slots) {
  return d.dv == 128 && slots * d.v_heads <= 128 ? 64 : d.dv;
}
template <typename T>
static const void* pick_forward(int dk, int columns, bool delta) {
  if (delta) {
    if (dk == 64) return reinterpret_cast<const void*>(&mix_forward_kernel<T, 64, 64, true>);
    return columns == 64 ? reinterpret_cast<const void*>(&mix_forward_kernel<T, 128, 64, true>)
                         : reinterpret_cast<const void*>(&mix_forward_kernel<T, 128, 128, true>);
  }
  if (dk == 64)
    return columns == 64 ? reinterpret_cast<const void*>(&mix_forward_kernel<T, 64, 64, false>)
                         : reinterpret_cast<const void*>(&mix_forward_kernel<T, 64, 128, false>);
  return columns == 64 ? reinterpret_cast<const void*>(&mix_forward_kernel<T, 128, 64, false>)
                       : reinterpret_cast<const void*>(&mix_forward_kernel<T, 128, 128, false>);
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
  const long cslots = scan_slots(d.tokens, d.seqs, kQ), slots = scan_slots(d.tokens, d.seqs, a.seg);
  const int columns = forward_columns(d, slots);
  const long grid = mix_grid(slots, d.k_heads, a.vpk * (d.dv / columns));
  if (!grid_fits(grid, 4 * columns) || !segments_fit(a, d.dk, delta, false) ||
      (delta && !grid_fits(cslots * ((d.v_heads + 3) / 4), 256)))
    return RSSM_ESHAPE;
  if (output_meets(a, d, o) || pools_meet(d, initial_state, final_state)) return RSSM_EINVAL;
  if (delta && d.tokens > 0) {
    rc = f32 ? launch_inverse<float, false>(a, d.dk, cslots, stream)
             : launch_inverse<bf16, false>(a, d.dk, cslots, stream);
    if (rc) return rc;
  }
  if (d.tokens > a.seg) {
    MixBwdArgs b{};
    b.m = a;
    rc = f32 ? launch_segments<float, false>(b, d.dk, delta, stream)
             : launch_segments<bf16, false>(b, d.dk, delta, stream);
    if (rc) return rc;
  }
  return launch_kernel(f32 ? pick_forward<float>(d.dk, columns, delta) : pick_forward<bf16>(d.dk, columns, delta),
                       (unsigned)grid, 4 * columns, 0, stream, a);
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
