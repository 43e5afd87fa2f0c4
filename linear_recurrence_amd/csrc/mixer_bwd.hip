// Linear attention and the gated delta rule over packed sequences, backward.
//
// With the chunk's quantities of mixer_common.hpp, P_ij = scale c_ij q_i.k_j (i >= j),
// dS' the gradient of the state after the chunk (linear attention: dD itself is dV,
// D = V, and what has dX in it is left out):
//   dD = P^T dO + e^{G_Q-G} K dS',  dX = T^T dD,  dV = beta dX
//   dS = e^{G_Q} dS' + (scale e^G Q)^T dO - (beta e^G K)^T dX
//   N_ij = scale c_ij dO_i.d_j (i >= j),  L_ij = -beta_i c_ij dX_i.d_j (i > j)
//   dq = scale e^G dO S^T + N K
//   dk = e^{G_Q-G} D dS'^T - beta e^G dX S^T + N^T Q + (L + L^T) K
//   dbeta_i = dX_i.v_i - e^{G_i} dX_i.(S^T k_i) - sum_{j<i} c_ij (k_i.k_j) (dX_i.d_j)
// and for the decays, with w_ij = (q_i.k_j) N_ij + (k_i.k_j) L_ij (i > j),
//   dG_i = sum_j w_ij - sum_j w_ji + scale e^{G_i} q_i.(dO_i S^T)
//          - beta_i e^{G_i} k_i.(dX_i S^T) - take_i,   take = e^{G_Q-G} k.(D dS'^T)
//   dg_t = sum_{i>=t} dG_i + sum take + e^{G_Q} <S, dS'>    (one chunk's tokens)
// dX_i.d_i / beta_i would be dbeta in a word, and has no value at beta = 0.
//
// Launches: (1) T of every chunk (the delta rule); (2) both recurrences over the
// chunks, the states and D forward, their gradients and dX backward, which leave
// every chunk's in the workspace in fp32; (3) the rest, a workgroup for one chunk and
// key head, which needs nothing from other chunks; (4) decays of a head: its sum.
//
// What is not an input enters the products as three bf16 terms, pairs of such factors
// as the six products that fp32 can hold, so nothing is rounded to the io type but the
// results.  Two terms of N and L, which only dq and dk read, would be 1 to 3% faster (8 x
// 1024 tokens of the delta rule: 688 us instead of 709).  fp32 inputs stay fp32.
#include "mixer_states.hpp"

namespace rssm {

template <typename T, int K, bool DELTA>
struct MainLds {
  typedef typename Mat<T>::E E;
  static constexpr int kFrag = 64 * sizeof(typename Mat<T>::Frag), TS = Mat<T>::kTerms;
  static constexpr int TD = DELTA ? TS : 1, W = K / 16;
  // fragments of 32 columns of dO, D (or V) and dX for the four blocks of 16 tokens
  static constexpr int kStage = 4 * (1 + TD + (DELTA ? TS : 0)) * kFrag;
  static constexpr int oD = 4 * kFrag, oX = oD + 4 * TD * kFrag;
  static constexpr int kTri = TS * Tile<T, 64>::SIZE;  // N, or L, as terms
  static constexpr int kTris = (DELTA ? 2 : 1) * kTri * (int)sizeof(E);
  __attribute__((aligned(16))) E k[Tile<T, K>::SIZE];
  __attribute__((aligned(16))) E q[Tile<T, K>::SIZE];
  __attribute__((aligned(16))) char area[2 * kStage > kTris ? 2 * kStage : kTris];
  ChunkGates g;
  float wrow[10][16], wcol[10][16], brow[10][16];  // by tile i (i + 1) / 2 + j
  float give[W][kQ], back[W][kQ], take[W][kQ];
  float xv[kQ], dot[W], own[kQ], took[kQ], all;
};

// Everything that stays within a chunk.  A wave owns 16 of the K columns of dq and dk;
// the columns of V are taken 32 at a time: each wave splits its share of D and dX for
// all of them and its own columns of S and dS', whose loads (the next 32 columns', or
// the next head's) are on their way during the products.  The 64x64 products dO D^T and
// dX D^T are held by tiles, and cross LDS once as rows of N and L, which then are read
// by rows and, transposing, by columns.  8 x 1024 tokens of 32 value heads of the delta
// rule take 372 us: 0.8 GB are read, 0.6 of them from memory, 170 us at a copy's rate; 75 us
// of the matrix units, 110 of the vector units and 100 of LDS, and five barriers a value head
// behind its columns' loop (without what stands between them it takes a quarter less), in one
// workgroup a compute unit (registers), overlap little.
template <typename T, int K, bool DELTA>
__global__ void __launch_bounds__(4 * K, 2) mix_main_kernel(const MixBwdArgs b) {
  typedef Mat<T> M;
  typedef typename M::E E;
  typedef typename M::Frag Frag;
  typedef MainLds<T, K, DELTA> L;
  typedef Tile<T, K> TK;
  typedef Tile<T, 64> TN;
  constexpr int TS = L::TS, TD = L::TD, KB = K / 32, W = L::W, TH = 64 * W;
  constexpr int JOBS = (10 + W - 1) / W;  // 16x16 tiles of the lower triangle a wave
  constexpr int SETS = 8 / W;             // blocks of rows that a wave splits: of D (V), of dX and dO
  __shared__ L s;
  const MixArgs& a = b.m;
  const int tid = threadIdx.x;
  int lane = tid & 63, i16 = lane & 15, g = lane >> 4;
  // what is worked out from the lane is worked out again, not kept through the loops
  const auto again = [&]() {
    forget(lane);
    i16 = lane & 15;
    g = lane >> 4;
  };
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / a.k_heads, hk = blockIdx.x % a.k_heads;
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, kQ, slot);
  if (sg.len == 0) {
    if (b.part)  // (the value heads of a key head may be more than the threads)
      for (int i = tid; i < a.vpk; i += TH) b.part[(long)slot * a.v_heads + hk * a.vpk + i] = 0.f;
    return;
  }
  const int rows = sg.len;
  const long t0 = sg.tok;
  TileLoad<T, K, TH> x, y;
  {
    x.start(static_cast<const E*>(a.k) + t0 * a.k_stride + (long)hk * K, a.k_stride, tid);
    y.start(static_cast<const E*>(a.q) + t0 * a.q_stride + (long)hk * K, a.q_stride, tid);
    x.fetch(rows, tid);
    y.fetch(rows, tid);
  }
  f32x4 dq[4], dk[4];  // rows t = 16 t + 4g + r, column 16 wave + i16
#pragma unroll
  for (int t = 0; t < 4; ++t) dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const Minus minus;
  const int blocks = a.dv / 32;
  // What the next 32 columns of V need, on its way: this wave's columns of the states, and
  // its rows (set 0: D, or V of linear attention; set 1: dX, dO and V)
  float fs[8], fg[8];
  RawK<float, 8> rx[SETS];
  RawK<T, 8> ro[SETS], rv;
  float rb = 0.f;  // beta of this lane's row
  const auto fetch_states = [&](int hx, int vb) {
    const long at = (long)slot * a.v_heads + hk * a.vpk + hx;
    const long p = (at * a.dv + 32 * vb + 8 * g) * K + 16 * wave + i16;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      fs[e] = b.state[p + e * K];
      fg[e] = b.grad[p + e * K];
    }
  };
  const auto fetch_rows = [&](int hx, int vb) {
    const int trow = 16 * (wave & 3) + i16, vc = 32 * vb + 8 * g;
    const long hv = hk * a.vpk + hx, at = (long)slot * a.v_heads + hv;
    const long tok = t0 + (trow < rows ? trow : 0);
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
      const bool second = W == 4 ? u == 1 : wave >= 4;
      if (DELTA) rx[u].load(second ? b.dX : b.D, (at * kQ + trow) * a.dv + vc, 8);
      ro[u].load(second ? b.dout : a.v, tok * (second ? b.do_stride : a.v_stride) + hv * a.dv + vc, 8);
    }
    if (DELTA) rv.load(a.v, tok * a.v_stride + hv * a.dv + vc, 8);
    if (DELTA) rb = a.beta[tok * a.v_heads + hv];
  };
  fetch_states(0, 0);
  fetch_rows(0, 0);
  x.put(s.k, rows, tid);
  y.put(s.q, rows, tid);
  // q_i.k_j and k_i.k_j of this wave's tiles (i, j), rows j, columns i: the same for all heads
  f32x4 qk[JOBS], kk[JOBS];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < JOBS; ++u) {
    const int n = wave + u * W, ti = n < 1 ? 0 : (n < 3 ? 1 : (n < 6 ? 2 : 3)), tj = n - ti * (ti + 1) / 2;
    qk[u] = kk[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (n < 10) {
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        const Frag kj = TK::rows_c(s.k, tj, 32 * x, lane);
        qk[u] = M::mma(kj, TK::rows_c(s.q, ti, 32 * x, lane), qk[u]);
        if (DELTA) kk[u] = M::mma(kj, TK::rows_c(s.k, ti, 32 * x, lane), kk[u]);
      }
    }
  }
#pragma unroll 1
  for (int hx = 0; hx < a.vpk; ++hx) {
    const int hv = hk * a.vpk + hx;
    const long at = (long)slot * a.v_heads + hv;
    GateLoad ld;
    ld.start(a, t0, hv, DELTA);
    ld.fetch(rows, lane);
    f32x4 into[4], back[4], out[4], dp[JOBS], dx[JOBS];
#pragma unroll
    for (int t = 0; t < 4; ++t) into[t] = back[t] = out[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < JOBS; ++u) dp[u] = dx[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    float xv = 0.f, dot = 0.f;
#pragma unroll 1
    for (int vb = 0; vb < blocks; ++vb) {
      again();
      char* const area = s.area + (vb & 1) * L::kStage;
      const int vc = 32 * vb + 8 * g, trow = 16 * (wave & 3) + i16;
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(fs[e], fg[e], dot);
      const auto ss = split<T, TS>(fs, minus), sd = split<T, TS>(fg, minus);
      const int hn = vb + 1 < blocks ? hx : hx + 1, vn = vb + 1 < blocks ? vb + 1 : 0;
      const bool more = hn < a.vpk;  // (behind the last there is the first again)
      fetch_states(more ? hn : 0, vn);
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
        const bool second = W == 4 ? u == 1 : wave >= 4;
        const int tb = wave & 3;
        float o[8], f[8];
        ro[u].get(o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = trow < rows ? o[e] : 0.f;
        if (DELTA) rx[u].get(f);
        if (second || !DELTA)
          put_split<T, 1>(area + (second ? 0 : L::oD), tb, split<T, 1>(o, minus), lane);
        if (DELTA) put_split<T, TS>(area + (second ? L::oX : L::oD), tb, split<T, TS>(f, minus), lane);
        if (DELTA && second && trow < rows) {
          float v[8], w[8];
          rv.get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xv = fmaf(f[e], v[e], xv);
            w[e] = rb * f[e];
          }
          Vec8<T>::store(b.dv, ((t0 + trow) * a.v_heads + hv) * a.dv + vc, w);
        }
      }
      fetch_rows(more ? hn : 0, vn);
      __syncthreads();
      again();
      mma_many<T, 1, TS, 4>([&](int t, int) { return frag_at<T>(area, t, lane); }, ss, into);
      mma_many<T, TD, TS, 4>([&](int t, int k) { return frag_at<T>(area + L::oD, t * TD + k, lane); }, sd, out);
      if (DELTA)
        mma_many<T, TS, TS, 4>([&](int t, int k) { return frag_at<T>(area + L::oX, t * TS + k, lane); }, ss, back);
      // rows j, columns i of tile (i, j)
#pragma unroll
      for (int u = 0; u < JOBS; ++u) {
        const int n = wave + u * W, ti = n < 1 ? 0 : (n < 3 ? 1 : (n < 6 ? 2 : 3)), tj = n - ti * (ti + 1) / 2;
        if (n < 10) {
          const auto d = split_at<T, TD>(area + L::oD, tj, lane);
          dp[u] = d.a_times(frag_at<T>(area, ti, lane), dp[u]);
          if (DELTA) dx[u] = mma_split<T, TD, TS>(d, split_at<T, TS>(area + L::oX, ti, lane), dx[u]);
        }
      }
    }
    if (DELTA) {
      xv = groups_sum(xv);
      if (wave >= W - 4 && g == 0) s.xv[16 * (wave & 3) + i16] = xv;
    }
    dot = groups_sum(row16_sum(dot));
    if (lane == 0) s.dot[wave] = dot;
    if (wave == W - 1) s.g.set(ld.log_g(rows, lane), ld.beta(rows, lane), lane);
    __syncthreads();  // the stages are no longer read
    again();
    // N and L by rows i, and the sums of w's rows and columns
    E* const sN = reinterpret_cast<E*>(s.area);
    E* const sL = sN + L::kTri;
#pragma unroll
    for (int u = 0; u < JOBS; ++u) {
      const int tile = wave + u * W, ti = tile < 1 ? 0 : (tile < 3 ? 1 : (tile < 6 ? 2 : 3)),
                tj = tile - ti * (ti + 1) / 2;
      if (tile < 10) {
        const int i = 16 * ti + i16;
        const float2 gi = s.g.G[i];
        const float be = s.g.beta[i];
        float n[4], l[4], wc[4], wr = 0.f, br = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * tj + 4 * g + r;
          const float c = exp2_f32(gap2(gi, s.g.G[j]));
          n[r] = i >= j ? a.scale * c * dp[u][r] : 0.f;
          wc[r] = i > j ? qk[u][r] * n[r] : 0.f;
          if (DELTA) {
            const float m = i > j ? c * dx[u][r] : 0.f;
            l[r] = -be * m;
            wc[r] = i > j ? fmaf(kk[u][r], l[r], wc[r]) : 0.f;
            br = i > j ? fmaf(kk[u][r], m, br) : br;
          }
          wr += wc[r];
        }
        wr = groups_sum(wr);
        if (DELTA) br = groups_sum(br);
        if (g == 0) {
          s.wrow[tile][i16] = wr;
          if (DELTA) s.brow[tile][i16] = br;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          wc[r] = row16_sum(wc[r]);
          if (i16 == r) s.wcol[tile][4 * g + r] = wc[r];
        }
        // four neighbours of row i, a term at a time; above the diagonal zeros
        const auto put4 = [&](E* plane, float* v) {
#pragma unroll
          for (int k = 0; k < TS; ++k) {
            const auto p = M::pack4(v);
            *reinterpret_cast<typename M::Four*>(plane + k * TN::SIZE + TN::at(i, 16 * tj + 4 * g)) = p;
            if (k + 1 < TS) {
              float f[4];
              M::unpack4(p, f);
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] -= f[r];
            }
            if (ti != tj) {
              const float z[4] = {0.f, 0.f, 0.f, 0.f};
              *reinterpret_cast<typename M::Four*>(plane + k * TN::SIZE + TN::at(16 * tj + i16, 16 * ti + 4 * g)) =
                  M::pack4(z);
            }
          }
        };
        put4(sN, n);
        if (DELTA) put4(sL, l);
      }
    }
    __syncthreads();
    again();
    {
      Frag kf[2], qf[2];
      float gv[16], bk[16], tk[16];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        kf[kb] = TK::cols(s.k, 32 * kb, 16 * wave, lane);
        qf[kb] = TK::cols(s.q, 32 * kb, 16 * wave, lane);
        float fk[8], fq[8];
        M::unpack(kf[kb], fk);
        M::unpack(qf[kb], fq);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 2 * kb + h;
          const f32x4 eg = *reinterpret_cast<const f32x4*>(&s.g.eg[16 * t + 4 * g]);
          const f32x4 et = *reinterpret_cast<const f32x4*>(&s.g.et[16 * t + 4 * g]);
          const f32x4 be = *reinterpret_cast<const f32x4*>(&s.g.beta[16 * t + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = a.scale * eg[r] * into[t][r], z = et[r] * out[t][r];
            dq[t][r] += x;
            dk[t][r] += z;
            gv[4 * t + r] = x * fq[4 * h + r];
            tk[4 * t + r] = z * fk[4 * h + r];
            if (DELTA) {
              const float y = eg[r] * back[t][r];
              dk[t][r] = fmaf(-be[r], y, dk[t][r]);
              bk[4 * t + r] = y * fk[4 * h + r];
            }
          }
        }
      }
      // sums over the 16 lanes of a group; item 4 t + r is token 16 t + 4g + r
      row16_sums<0>(gv, lane);
      row16_sums<0>(tk, lane);
      if (DELTA) row16_sums<0>(bk, lane);
      const int t16 = 16 * (i16 >> 2) + 4 * g + (i16 & 3);
      s.give[wave][t16] = gv[0];
      s.take[wave][t16] = tk[0];
      if (DELTA) s.back[wave][t16] = bk[0];
#pragma unroll
      for (int k = TS - 1; k >= 0; --k)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const E *const pn = sN + k * TN::SIZE, *const pl = sL + k * TN::SIZE;
            if (kb <= t / 2) {
              dq[t] = M::mma(TN::rows_d(pn, t, 32 * kb, lane), kf[kb], dq[t]);
              if (DELTA) dk[t] = M::mma(TN::rows_d(pl, t, 32 * kb, lane), kf[kb], dk[t]);
            }
            if (kb >= t / 2) {
              dk[t] = M::mma(TN::cols(pn, 32 * kb, 16 * t, lane), qf[kb], dk[t]);
              if (DELTA) dk[t] = M::mma(TN::cols(pl, 32 * kb, 16 * t, lane), kf[kb], dk[t]);
            }
          }
    }
    __syncthreads();
    again();
    // the parts of each token's sums: eight lanes a token (its waves', then its tiles')
    if (b.dg) {
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
        const int p = lane & 7, t = 8 * (wave + u * W) + (lane >> 3), blk = t >> 4, r = t & 15;
        float give = p < W ? s.give[p][t] : 0.f, take = p < W ? s.take[p][t] : 0.f;
        float bk = DELTA && p < W ? s.back[p][t] : 0.f, all = p < W ? s.dot[p] : 0.f;
        float row = p <= blk ? s.wrow[blk * (blk + 1) / 2 + p][r] : 0.f;
        float br = DELTA && p <= blk ? s.brow[blk * (blk + 1) / 2 + p][r] : 0.f;
        row -= p >= blk && p < 4 ? s.wcol[p * (p + 1) / 2 + blk][r] : 0.f;
        const auto sum8 = [](float v) {
          v += dpp_f32<0x141>(v);
          v += dpp_f32<0x4E>(v);
          return v + dpp_f32<0xB1>(v);
        };
        row += give - take;
        if (DELTA) row = fmaf(-s.g.beta[t], bk, row);
        row = sum8(row);
        take = sum8(take);
        all = sum8(all);
        if (DELTA) bk = sum8(bk), br = sum8(br);
        if (p == 0) {
          s.own[t] = row;
          s.took[t] = take;
          if (t == 0) s.all = all;
          if (DELTA && t < rows) b.dbeta[(t0 + t) * a.v_heads + hv] = s.xv[t] - bk - br;
        }
      }
    }
    __syncthreads();  // the next head writes all but what follows needs
    if (wave == W / 2 && b.dg) {  // a wave with the fewest tiles; one token a lane: the sums over i >= t, in double
      const double own = s.own[lane], tot = last_lane(lane_sums((double)s.took[lane])) + (double)s.g.all * s.all;
      const double before = lane_sums(own);  // a difference of sums will do in double
      double dg = last_lane(before) - before + own + tot;
      if (lane >= rows) dg = 0.0;
      if (a.decay == RSSM_DECAY_TOKEN) {
        if (lane < rows) b.dg[(t0 + lane) * a.v_heads + hv] = (float)dg;
      } else {
        dg = last_lane(lane_sums(dg));
        if (lane == 0) b.part[at] = (float)dg;
      }
    }
  }
  // to the io type, and 16 bytes at a time to memory
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int p = TK::at(16 * t + 4 * g + r, 16 * wave + i16);
      Elt<T>::store1(s.q, p, dq[t][r]);
      Elt<T>::store1(s.k, p, dk[t][r]);
    }
  __syncthreads();
  constexpr int V = 16 / sizeof(E), PER = K / V;
  for (int e = tid; e < rows * PER; e += TH) {
    const int t = e / PER, c = (e % PER) * V;
    const long o = ((t0 + t) * a.k_heads + hk) * K + c;
    *reinterpret_cast<u32x4*>(static_cast<E*>(b.dq) + o) = *reinterpret_cast<const u32x4*>(s.q + TK::at(t, c));
    *reinterpret_cast<u32x4*>(static_cast<E*>(b.dk) + o) = *reinterpret_cast<const u32x4*>(s.k + TK::at(t, c));
  }
}

// dg of a head's constant decay: its chunks' sums, in a fixed order.
__global__ void __launch_bounds__(256) mix_decay_sum_kernel(const MixBwdArgs b) {
  __shared__ double sum[256];
  double v = 0.0;
  for (long c = threadIdx.x; c < b.cslots; c += 256) v += b.part[c * b.m.v_heads + blockIdx.x];
  sum[threadIdx.x] = v;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) sum[threadIdx.x] += sum[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) b.dg[blockIdx.x] = (float)sum[0];
}
static int launch_decay_sum(const MixBwdArgs& b, hipStream_t stream) {
  return launch_kernel(reinterpret_cast<const void*>(&mix_decay_sum_kernel), b.m.v_heads, 256, 0, stream, b);
}

struct BwdLayout {
  size_t tinv, state, grad, D, dX, part, end;
  SegLayout seg;
};
static BwdLayout bwd_layout(const rssm_mixer_dims& d, bool delta) {
  BwdLayout l{};
  const size_t units = (size_t)scan_slots(d.tokens, d.seqs, kQ) * d.v_heads;
  MixTake take;
  l.tinv = take(delta ? units * mix_inverse_bytes(d.io_dtype == RSSM_F32, true) : 0);
  l.state = take(units * d.dk * d.dv * 4);
  l.grad = take(units * d.dk * d.dv * 4);
  l.D = take(delta ? units * kQ * d.dv * 4 : 0);
  l.dX = take(delta ? units * kQ * d.dv * 4 : 0);
  l.part = take(units * 4);
  l.seg = seg_layout(d, delta, true, take);
  l.end = take.at;
  return l;
}

template <typename T>
static const void* pick_states(const rssm_mixer_dims& d, bool delta) {
  if (delta)
    return d.dk == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 64, true, true, true>)
                      : reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 128, true, true, true>);
  if (d.dk == 64)
    return d.dv == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 64, false, true, true>)
                      : reinterpret_cast<const void*>(&mix_states_kernel<T, 64, 128, false, true, true>);
  return d.dv == 64 ? reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 64, false, true, true>)
                    : reinterpret_cast<const void*>(&mix_states_kernel<T, 128, 128, false, true, true>);
}
template <typename T>
static const void* pick_main(const rssm_mixer_dims& d, bool delta) {
  if (delta)
    return d.dk == 64 ? reinterpret_cast<const void*>(&mix_main_kernel<T, 64, true>)
                      : reinterpret_cast<const void*>(&mix_main_kernel<T, 128, true>);
  return d.dk == 64 ? reinterpret_cast<const void*>(&mix_main_kernel<T, 64, false>)
                    : reinterpret_cast<const void*>(&mix_main_kernel<T, 128, false>);
}

static size_t mix_backward_bytes(const rssm_mixer_dims* dims, bool delta) {
  return mix_check(dims, delta) || dims->tokens == 0 ? 0 : bwd_layout(*dims, delta).end;
}

static int mix_backward(const rssm_mixer_dims* dims, bool delta, MixBwdArgs b, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  int rc = mix_check(dims, delta);
  if (rc) return rc;
  const rssm_mixer_dims& d = *dims;
  MixArgs& a = b.m;
  if (d.seqs == 0 && d.tokens) return RSSM_EINVAL;
  if (d.decay == RSSM_DECAY_HEAD && !b.dg) return RSSM_EINVAL;
  if (d.seqs == 0) {  // nothing is written but a decay's gradient that has no token's shape
    if (d.decay != RSSM_DECAY_HEAD) return RSSM_OK;
    a.v_heads = d.v_heads;
    return launch_decay_sum(b, stream);
  }
  if (!a.cu && d.seqs != 1) return RSSM_EINVAL;
  if (d.tokens > 0 && (!a.q || !a.k || !a.v || !b.dout || !b.dq || !b.dk || !b.dv ||
                       (d.decay && (!a.g || !b.dg)) || (delta && (!a.beta || !b.dbeta))))
    return RSSM_EINVAL;
  const void* vec[] = {a.q, a.k, a.v, b.dout, b.dq, b.dk, b.dv, a.init, b.dfinal, b.dinit, workspace};
  for (const void* p : vec)
    if (!aligned16(p)) return RSSM_EINVAL;
  const size_t need = mix_backward_bytes(dims, delta);
  if (need && (!workspace || workspace_bytes < need)) return RSSM_EINVAL;
  mix_fill(a, d);
  b.do_stride = d.do_stride ? d.do_stride : (long)d.v_heads * d.dv;
  if (!d.decay) b.dg = nullptr;
  const BwdLayout l = bwd_layout(d, delta);
  char* const ws = static_cast<char*>(workspace);
  a.tinv = ws + l.tinv;
  b.state = reinterpret_cast<float*>(ws + l.state);
  b.grad = reinterpret_cast<float*>(ws + l.grad);
  b.D = reinterpret_cast<float*>(ws + l.D);
  b.dX = reinterpret_cast<float*>(ws + l.dX);
  b.part = d.decay == RSSM_DECAY_HEAD ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  const bool f32 = d.io_dtype == RSSM_F32;
  b.cslots = scan_slots(d.tokens, d.seqs, kQ);
  seg_fill(a, d, l.seg, workspace);
  const long dir = mix_grid(scan_slots(d.tokens, d.seqs, a.seg), d.k_heads, a.vpk), mgrid = b.cslots * d.k_heads;
  if (!grid_fits(2 * dir, 4 * d.dv) || !segments_fit(a, d.dk, delta, true) || !grid_fits(mgrid, 4 * d.dk) ||
      (delta && !grid_fits(b.cslots * ((d.v_heads + 3) / 4), 256)))
    return RSSM_ESHAPE;
  const long es = f32 ? 4 : 2, qk = (long)d.k_heads * d.dk, vw = (long)d.v_heads * d.dv;
  void* const results[] = {b.dq, b.dk, b.dv};
  for (void* p : results) {
    const long columns = p == b.dv ? vw : qk;
    if (mix_meets(a, d, p, columns) || rows_meet(b.dout, b.do_stride * es, vw * es, d.tokens, p, d.tokens * columns * es))
      return RSSM_EINVAL;
  }
  if (b.dinit) {  // by sequence, the pool by slot
    const long state = (long)d.v_heads * d.dv * d.dk * 4;
    if (rows_meet(a.init, state, state, d.num_slots, b.dinit, d.seqs * state)) return RSSM_EINVAL;
  }
  b.dir_blocks = (int)dir;
  if (d.tokens == 0) {  // no chunks, and no gradient of a decay but zero
    b.cslots = 0;
  } else if (delta) {
    rc = f32 ? launch_inverse<float, true>(a, d.dk, b.cslots, stream)
             : launch_inverse<bf16, true>(a, d.dk, b.cslots, stream);
    if (rc) return rc;
  }
  if (d.tokens > a.seg) {
    rc = f32 ? launch_segments<float, true>(b, d.dk, delta, stream)
             : launch_segments<bf16, true>(b, d.dk, delta, stream);
    if (rc) return rc;
  }
  rc = launch_kernel(f32 ? pick_states<float>(d, delta) : pick_states<bf16>(d, delta), (unsigned)(2 * dir),
                     4 * d.dv, 0, stream, b);
  if (!rc && d.tokens > 0)
    rc = launch_kernel(f32 ? pick_main<float>(d, delta) : pick_main<bf16>(d, delta), (unsigned)mgrid, 4 * d.dk, 0,
                       stream, b);
  if (!rc && d.decay == RSSM_DECAY_HEAD) rc = launch_decay_sum(b, stream);
  return rc;
}

}  // namespace rssm

using namespace rssm;

static MixBwdArgs bwd_args(const void* dout, const void* q, const void* k, const void* v, const float* g,
                           const int32_t* cu_seqlens, const float* initial_state,
                           const uint8_t* has_initial, const int32_t* slot_idx,
                           const float* dfinal_state, void* dq, void* dk, void* dv, float* dg,
                           float* dinitial_state, int32_t* status) {
  MixBwdArgs b{};
  b.m.q = q;
  b.m.k = k;
  b.m.v = v;
  b.m.g = g;
  b.m.cu = cu_seqlens;
  b.m.init = initial_state;
  b.m.has_init = has_initial;
  b.m.slot_idx = slot_idx;
  b.m.status = status;
  b.dout = dout;
  b.dfinal = dfinal_state;
  b.dq = dq;
  b.dk = dk;
  b.dv = dv;
  b.dg = dg;
  b.dinit = dinitial_state;
  return b;
}

extern "C" size_t linear_attention_backward_workspace(const rssm_mixer_dims* dims) {
  return mix_backward_bytes(dims, false);
}

extern "C" int linear_attention_backward(const rssm_mixer_dims* dims, const void* dout, const void* q,
                                         const void* k, const void* v, const float* log_decay,
                                         const int32_t* cu_seqlens, const float* initial_state,
                                         const uint8_t* has_initial, const int32_t* slot_idx,
                                         const float* dfinal_state, void* dq, void* dk, void* dv,
                                         float* dlog_decay, float* dinitial_state, void* workspace,
                                         size_t workspace_bytes, int32_t* status, hipStream_t stream) {
  return mix_backward(dims, false,
                      bwd_args(dout, q, k, v, log_decay, cu_seqlens, initial_state, has_initial, slot_idx,
                               dfinal_state, dq, dk, dv, dlog_decay, dinitial_state, status),
                      workspace, workspace_bytes, stream);
}

extern "C" size_t gdn_scan_backward_workspace(const rssm_mixer_dims* dims) {
  return mix_backward_bytes(dims, true);
}

extern "C" int gdn_scan_backward(const rssm_mixer_dims* dims, const void* dout, const void* q, const void* k,
                                 const void* v, const float* log_g, const float* beta,
                                 const int32_t* cu_seqlens, const float* initial_state,
                                 const uint8_t* has_initial, const int32_t* slot_idx,
                                 const float* dfinal_state, void* dq, void* dk, void* dv, float* dlog_g,
                                 float* dbeta, float* dinitial_state, void* workspace,
                                 size_t workspace_bytes, int32_t* status, hipStream_t stream) {
  MixBwdArgs b = bwd_args(dout, q, k, v, log_g, cu_seqlens, initial_state, has_initial, slot_idx,
                          dfinal_state, dq, dk, dv, dlog_g, dinitial_state, status);
  b.m.beta = beta;
  b.dbeta = dbeta;
  return mix_backward(dims, true, b, workspace, workspace_bytes, stream);
}
